// norm_cols.hip -- the layer norm of norm_rows.hip over the channels of [B, E, L], the layout of the conv and the scan.
//
// A workgroup owns LP * 8 consecutive positions of one batch row and all of their channels: LP lanes hold a channel's
// positions, 8 each, and the NT / LP groups of lanes take the channels in turn.  A position's sums go over the groups:
// within a wave by shuffles, over the waves through LDS.  With C > 0 every lane keeps its C channels in registers
// between the passes; with C = 0 they are read again (from the caches, where they fit).
#include "block_device.h"

namespace ssm {

namespace {

// v[k] summed over all lanes of the workgroup that have the same positions; sm: (NT / 64 + 1) * LP * 8 floats
template <int NT, int LP>
__device__ __forceinline__ void sum_groups(float (&v)[8], float* sm) {
  constexpr int T = LP * 8, NW = NT / 64;
#pragma unroll
  for (int m = LP; m < 64; m *= 2)
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += __shfl_xor(v[k], m);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  if (lane < LP) {
#pragma unroll
    for (int k = 0; k < 8; ++k) sm[w * T + lane * 8 + k] = v[k];
  }
  __syncthreads();
  if (threadIdx.x < T) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) s += sm[i * T + threadIdx.x];
    sm[NW * T + threadIdx.x] = s;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = sm[NW * T + (threadIdx.x % LP) * 8 + k];
}

// sum over the LP lanes that hold a channel's positions
template <int LP> __device__ __forceinline__ float sum_positions(float v) {
#pragma unroll
  for (int m = 1; m < LP; m *= 2) v += __shfl_xor(v, m);
  return v;
}

}  // namespace

template <typename XT, typename HT, int NT, int LP, int C>
__global__ __launch_bounds__(NT) void norm_cols_kernel(NormParams p) {
  constexpr int NG = NT / LP, T = LP * 8;
  __shared__ float sm[(NT / 64 + 1) * T];
  const int pl = threadIdx.x % LP, cg = threadIdx.x / LP;
  const int64_t tiles = (p.L + T - 1) / T, blk = block_id();
  const int64_t b = blk / tiles, t = blk % tiles * T + pl * 8;
  if (b >= p.B) return;
  const int n = p.L - t >= 8 ? 8 : p.L - t > 0 ? (int)(p.L - t) : 0;
  const int64_t base = b * p.E * p.L + t;
  const Drop drop(p.drop);
  auto fetch = [&](int64_t e, float (&s)[8]) {  // the sum that is normalised
    const int64_t at = base + e * p.L;
    load_n<XT, 8>(static_cast<const XT*>(p.x) + at, n, s);
    float q[8];
    if (p.residual) load_n<HT, 8>(static_cast<const HT*>(p.residual) + at, n, q);
    if (drop.any()) drop.apply(drop.kept((uint64_t)at), s);
    if (p.residual) {
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] += q[k];
    }
  };
  float m[8], r[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) m[k] = r[k] = 0.0f;
  auto spread = [&](const float (&s)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = s[k] - m[k];
      r[k] = __builtin_fmaf(d, d, r[k]);
    }
  };
  auto means = [&] {
#pragma unroll
    for (int k = 0; k < 8; ++k) m[k] = p.rms ? 0.0f : m[k] * p.inv_e;
  };
  auto factors = [&] {
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = 1.0f / sqrtf(r[k] * p.inv_e + p.eps);
    if (p.stats && cg == 0) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) {
          p.stats[b * p.L + t + k] = m[k];
          p.stats[p.rows + b * p.L + t + k] = r[k];
        }
    }
  };
  auto finish = [&](int64_t e, float (&s)[8]) {
    const float w = p.weight ? p.weight[e] : 1.0f, c = p.bias ? p.bias[e] : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = __builtin_fmaf((s[k] - m[k]) * r[k], w, c);
    store_n<XT, 8>(static_cast<XT*>(p.out) + base + e * p.L, n, s);
  };
  if constexpr (C > 0) {
    float s[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t e = c * NG + cg;
      if (e < p.E) {
        fetch(e, s[c]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) s[c][k] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) m[k] += s[c][k];
    }
    if (p.hidden) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (c * NG + cg < p.E)
          store_n<HT, 8>(static_cast<HT*>(p.hidden) + base + (int64_t)(c * NG + cg) * p.L, n, s[c]);
    }
    if (!p.rms) sum_groups<NT, LP>(m, sm);
    means();
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c * NG + cg < p.E) spread(s[c]);
    sum_groups<NT, LP>(r, sm);
    factors();
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c * NG + cg < p.E) finish(c * NG + cg, s[c]);
  } else {
    float s[8];
    for (int64_t e = cg; e < p.E; e += NG) {
      fetch(e, s);
      if (p.hidden) store_n<HT, 8>(static_cast<HT*>(p.hidden) + base + e * p.L, n, s);
#pragma unroll
      for (int k = 0; k < 8; ++k) m[k] += s[k];
    }
    if (!p.rms) sum_groups<NT, LP>(m, sm);
    means();
    for (int64_t e = cg; e < p.E; e += NG) {
      fetch(e, s);
      spread(s);
    }
    sum_groups<NT, LP>(r, sm);
    factors();
    for (int64_t e = cg; e < p.E; e += NG) {
      fetch(e, s);
      finish(e, s);
    }
  }
}

// Tiles in turn; the lanes that own a channel add its dw and db of every tile to the workgroup's partial sums, which
// no other lane touches.
template <typename XT, typename HT, int NT, int LP, int C>
__global__ __launch_bounds__(NT) void norm_cols_bwd_kernel(NormParams p) {
  constexpr int NG = NT / LP, T = LP * 8;
  __shared__ float sm[(NT / 64 + 1) * T];
  const int pl = threadIdx.x % LP, cg = threadIdx.x / LP;
  const int64_t tiles = (p.L + T - 1) / T;
  const Drop drop(p.drop);
  float* part = p.part ? p.part + (int64_t)block_id() * 2 * p.E : nullptr;
  bool first = true;
  for (int64_t tile = block_id(); tile < p.B * tiles; tile += p.blocks) {
    const int64_t b = tile / tiles, t = tile % tiles * T + pl * 8;
    const int n = p.L - t >= 8 ? 8 : p.L - t > 0 ? (int)(p.L - t) : 0;
    const int64_t base = b * p.E * p.L + t;
    float m[8], r[8], c1[8], c2[8];
    load_n<float, 8>(p.stats + b * p.L + t, n, m);
    load_n<float, 8>(p.stats + p.rows + b * p.L + t, n, r);
#pragma unroll
    for (int k = 0; k < 8; ++k) c1[k] = c2[k] = 0.0f;
    auto fetch = [&](int64_t e, float (&d)[8], float (&h)[8]) {
      const int64_t at = base + e * p.L;
      load_n<XT, 8>(static_cast<const XT*>(p.x) + at, n, d);
      load_n<HT, 8>(static_cast<const HT*>(p.residual) + at, n, h);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[k] = (h[k] - m[k]) * r[k];  // (r is 0 behind the last position)
    };
    auto sums = [&](int64_t e, const float (&d)[8], const float (&h)[8]) {
      const float w = p.weight ? p.weight[e] : 1.0f;
      float dw = 0.0f, db = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dw = __builtin_fmaf(d[k], h[k], dw);
        db += d[k];
        c1[k] = __builtin_fmaf(d[k], w, c1[k]);
        c2[k] = __builtin_fmaf(d[k] * w, h[k], c2[k]);
      }
      if (part) {
        dw = sum_positions<LP>(dw);
        db = sum_positions<LP>(db);
        if (pl == 0) {
          part[e] = first ? dw : part[e] + dw;
          part[p.E + e] = first ? db : part[p.E + e] + db;
        }
      }
    };
    auto finish = [&](int64_t e, float (&d)[8], const float (&h)[8]) {
      const int64_t at = base + e * p.L;
      const float w = p.weight ? p.weight[e] : 1.0f;
      float q[8];
      if (p.dhidden) load_n<HT, 8>(static_cast<const HT*>(p.dhidden) + at, n, q);
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] = r[k] * (d[k] * w - c1[k] - h[k] * c2[k]);
      if (p.dhidden) {
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] += q[k];
      }
      if (p.hidden) store_n<HT, 8>(static_cast<HT*>(p.hidden) + at, n, d);
      if (p.out) {
        if (drop.any()) drop.apply(drop.kept((uint64_t)at), d);
        store_n<XT, 8>(static_cast<XT*>(p.out) + at, n, d);
      }
    };
    auto join = [&] {
      if (!p.rms) sum_groups<NT, LP>(c1, sm);
      sum_groups<NT, LP>(c2, sm);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        c1[k] = p.rms ? 0.0f : c1[k] * p.inv_e;
        c2[k] *= p.inv_e;
      }
    };
    if constexpr (C > 0) {
      float d[C][8], h[C][8];
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (c * NG + cg < p.E) fetch(c * NG + cg, d[c], h[c]);
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (c * NG + cg < p.E) sums(c * NG + cg, d[c], h[c]);
      join();
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (c * NG + cg < p.E) finish(c * NG + cg, d[c], h[c]);
    } else {
      float d[8], h[8];
      for (int64_t e = cg; e < p.E; e += NG) {
        fetch(e, d, h);
        sums(e, d, h);
      }
      join();
      for (int64_t e = cg; e < p.E; e += NG) {
        fetch(e, d, h);
        finish(e, d, h);
      }
    }
    first = false;
  }
}

namespace {

template <typename XT, typename HT, int NT, int LP, int C>
void go(const NormParams& p, hipStream_t s) {
  const int64_t tiles = (p.L + LP * 8 - 1) / (LP * 8);
  hipLaunchKernelGGL((norm_cols_kernel<XT, HT, NT, LP, C>), grid_of(p.B * tiles), dim3(NT), 0, s, p);
}

template <typename XT, typename HT>
void fwd(const NormParams& p, hipStream_t s) {
  if (p.E <= 128) return go<XT, HT, 256, 8, 4>(p, s);
  if (p.E <= 512) return go<XT, HT, 1024, 8, 4>(p, s);
  if (p.E <= 1024) return go<XT, HT, 1024, 8, 8>(p, s);
  go<XT, HT, 1024, 8, 0>(p, s);
}

template <typename XT, typename HT, int NT, int LP, int C>
void go_bwd(const NormParams& p, hipStream_t s) {
  hipLaunchKernelGGL((norm_cols_bwd_kernel<XT, HT, NT, LP, C>), grid_of(p.blocks), dim3(NT), 0, s, p);
}

template <typename XT, typename HT>
void bwd(const NormParams& p, hipStream_t s) {
  if (p.E <= 128) return go_bwd<XT, HT, 256, 8, 4>(p, s);
  if (p.E <= 512) return go_bwd<XT, HT, 1024, 8, 4>(p, s);
  go_bwd<XT, HT, 1024, 8, 0>(p, s);
}

}  // namespace

int64_t norm_cols_bwd_blocks(int64_t B, int64_t L, int64_t, int) {
  const int64_t tiles = B * ((L + 63) / 64);
  return tiles < 1024 ? tiles : 1024;
}

hipError_t launch_norm_cols(const NormParams& p, int kind, hipStream_t s) {
  if (kind == 3) fwd<bf16_t, bf16_t>(p, s);
  else if (kind == 1) fwd<bf16_t, float>(p, s);
  else fwd<float, float>(p, s);
  return hipGetLastError();
}

hipError_t launch_norm_cols_bwd(const NormParams& p, int kind, hipStream_t s) {
  if (kind == 3) bwd<bf16_t, bf16_t>(p, s);
  else if (kind == 1) bwd<bf16_t, float>(p, s);
  else bwd<float, float>(p, s);
  return hipGetLastError();
}

}  // namespace ssm
