// norm_rows.hip -- layer norm and RMS norm of rows, with what comes before them in a residual block, and the gradients.
//
//   s = residual + dropout(x);  m = mean(s) (RMS: 0);  r = 1 / sqrt(mean((s - m)^2) + eps)
//   hidden = s;  out = (s - m) r w + b
//   backward, with xh = (s - m) r and g = dout w:
//   ds = r (g - mean(g) - xh mean(g xh)) + dhidden (RMS: without mean(g));  dresidual = ds;  dx = dropout(ds)
//   dw = sum over rows of dout xh;  db = sum over rows of dout
//
// Bound by HBM: every stream is read once and written once.  LN lanes (16, 64 or a workgroup) hold a row in registers,
// P pieces of 8 elements each, so that the variance is a second pass over registers (about the mean, no cancellation).
// out is made from the unrounded sum; the hidden that is kept for the backward pass is rounded to its type.
// Rows too long for the registers go through memory again for each pass.
#include "block_device.h"

namespace ssm {

namespace {

// sum over the LN lanes of a row's team, in all of them; sm: a float for each wave (LN = 256), used in turn
template <int LN>
__device__ __forceinline__ float sum_team(float v, float* sm) {
  if constexpr (LN <= 64) {
    return sum_lanes<LN>(v);
  } else {
    v = sum_lanes<64>(v);
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
    __syncthreads();
    return (sm[0] + sm[1]) + (sm[2] + sm[3]);
  }
}

template <int N> __device__ __forceinline__ float sum8(const float (&x)[N]) {
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < N; ++e) s += x[e];
  return s;
}

__device__ __forceinline__ int in_piece(int64_t left) { return left >= 8 ? 8 : left > 0 ? (int)left : 0; }

}  // namespace

// One row of LN lanes; P = 0: any number of pieces, read again for every pass.
template <typename XT, typename HT, int LN, int P>
__global__ __launch_bounds__(256) void norm_rows_kernel(NormParams p) {
  constexpr int R = 256 / LN;
  __shared__ float sm[8];
  const int lane = threadIdx.x % LN;
  const int64_t row = (int64_t)block_id() * R + threadIdx.x / LN;
  if (row >= p.rows) return;
  const int64_t base = row * p.E;
  const XT* x = static_cast<const XT*>(p.x) + base;
  const HT* res = p.residual ? static_cast<const HT*>(p.residual) + base : nullptr;
  const Drop drop(p.drop);
  auto fetch = [&](int64_t e, int n, float (&s)[8]) {  // the sum that is normalised
    load_n<XT, 8>(x + e, n, s);
    float q[8];
    if (res) load_n<HT, 8>(res + e, n, q);
    if (drop.any()) drop.apply(drop.kept((uint64_t)(base + e)), s);
    if (res) {
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] += q[k];
    }
  };
  auto finish = [&](int64_t e, int n, float (&s)[8], float m, float r) {
    float w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = (s[k] - m) * r;
    if (p.weight) {
      load_n<float, 8>(p.weight + e, n, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] *= w[k];
    }
    if (p.bias) {
      load_n<float, 8>(p.bias + e, n, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] += w[k];
    }
    store_n<XT, 8>(static_cast<XT*>(p.out) + base + e, n, s);
  };
  auto spread = [&](const float (&s)[8], int n, float m) {  // sum of squares about m
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = k < n ? s[k] - m : 0.0f;
      v = __builtin_fmaf(d, d, v);
    }
    return v;
  };
  float m = 0.0f, v = 0.0f;
  if constexpr (P > 0) {
    float s[P][8];
    int n[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int64_t e = (int64_t)(k * LN + lane) * 8;
      n[k] = in_piece(p.E - e);
      fetch(e, n[k], s[k]);
      m += sum8(s[k]);
    }
    if (p.hidden) {
#pragma unroll
      for (int k = 0; k < P; ++k)
        store_n<HT, 8>(static_cast<HT*>(p.hidden) + base + (int64_t)(k * LN + lane) * 8, n[k], s[k]);
    }
    m = p.rms ? 0.0f : sum_team<LN>(m, sm) * p.inv_e;
#pragma unroll
    for (int k = 0; k < P; ++k) v += spread(s[k], n[k], m);
    v = sum_team<LN>(v, sm + 4) * p.inv_e;
    const float r = 1.0f / sqrtf(v + p.eps);
#pragma unroll
    for (int k = 0; k < P; ++k) finish((int64_t)(k * LN + lane) * 8, n[k], s[k], m, r);
    if (p.stats && lane == 0) {
      p.stats[row] = m;
      p.stats[p.rows + row] = r;
    }
  } else {
    float s[8];
    for (int64_t e = lane * 8; e < p.E; e += LN * 8) {
      const int n = in_piece(p.E - e);
      fetch(e, n, s);
      if (p.hidden) store_n<HT, 8>(static_cast<HT*>(p.hidden) + base + e, n, s);
      m += sum8(s);
    }
    m = p.rms ? 0.0f : sum_team<LN>(m, sm) * p.inv_e;
    for (int64_t e = lane * 8; e < p.E; e += LN * 8) {
      const int n = in_piece(p.E - e);
      fetch(e, n, s);
      v += spread(s, n, m);
    }
    v = sum_team<LN>(v, sm + 4) * p.inv_e;
    const float r = 1.0f / sqrtf(v + p.eps);
    for (int64_t e = lane * 8; e < p.E; e += LN * 8) {
      const int n = in_piece(p.E - e);
      fetch(e, n, s);
      finish(e, n, s, m, r);
    }
    if (p.stats && lane == 0) {
      p.stats[row] = m;
      p.stats[p.rows + row] = r;
    }
  }
}

// Rows in turn (p.blocks workgroups of 256 / LN teams); dw and db of the lane's columns are added up over the team's
// rows in registers, then over the workgroup's teams in LDS, and go to memory as the workgroup's partial sums.
// P = 0: any number of pieces, read twice; dw and db are then summed by norm_sums_kernel.
template <typename XT, typename HT, int LN, int P>
__global__ __launch_bounds__(256) void norm_rows_bwd_kernel(NormParams p) {
  constexpr int R = 256 / LN, PA = P > 0 ? P : 1;
  __shared__ float sm[8];
  __shared__ float acc[P > 0 && R > 1 ? 256 * PA * 8 : 1];
  const int lane = threadIdx.x % LN, team = threadIdx.x / LN;
  const HT* hidden = static_cast<const HT*>(p.residual);
  const Drop drop(p.drop);
  float dw[PA][8], db[PA][8];
#pragma unroll
  for (int k = 0; k < PA; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[k][e] = db[k][e] = 0.0f;
  // one piece: xh and g in place of what was read
  auto fetch = [&](int64_t base, int64_t e, int n, float m, float r, float (&d)[8], float (&h)[8], float (&w)[8]) {
    load_n<XT, 8>(static_cast<const XT*>(p.x) + base + e, n, d);
    load_n<HT, 8>(hidden + base + e, n, h);
    if (p.weight) {
      load_n<float, 8>(p.weight + e, n, w);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = 1.0f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = (h[k] - m) * r;
  };
  auto finish = [&](int64_t base, int64_t e, int n, float r, float c1, float c2, float (&g)[8], const float (&h)[8]) {
    float q[8];
    if (p.dhidden) load_n<HT, 8>(static_cast<const HT*>(p.dhidden) + base + e, n, q);
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = r * (g[k] - c1 - h[k] * c2);
    if (p.dhidden) {
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] += q[k];
    }
    if (p.hidden) store_n<HT, 8>(static_cast<HT*>(p.hidden) + base + e, n, g);
    if (p.out) {
      if (drop.any()) drop.apply(drop.kept((uint64_t)(base + e)), g);
      store_n<XT, 8>(static_cast<XT*>(p.out) + base + e, n, g);
    }
  };
  for (int64_t row0 = (int64_t)block_id() * R; row0 < p.rows; row0 += p.blocks * R) {
    const int64_t row = row0 + team;
    if (LN < 256 && row >= p.rows) break;
    const int64_t base = row * p.E;
    const float m = p.stats[row], r = p.stats[p.rows + row];
    float c1 = 0.0f, c2 = 0.0f;
    if constexpr (P > 0) {
      float g[P][8], h[P][8];
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int64_t e = (int64_t)(k * LN + lane) * 8;
        const int n = in_piece(p.E - e);
        float w[8];
        fetch(base, e, n, m, r, g[k], h[k], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i >= n) g[k][i] = h[k][i] = 0.0f;
          dw[k][i] = __builtin_fmaf(g[k][i], h[k][i], dw[k][i]);
          db[k][i] += g[k][i];
          g[k][i] *= w[i];
          c1 += g[k][i];
          c2 = __builtin_fmaf(g[k][i], h[k][i], c2);
        }
      }
      c1 = p.rms ? 0.0f : sum_team<LN>(c1, sm) * p.inv_e;
      c2 = sum_team<LN>(c2, sm + 4) * p.inv_e;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int64_t e = (int64_t)(k * LN + lane) * 8;
        finish(base, e, in_piece(p.E - e), r, c1, c2, g[k], h[k]);
      }
    } else {
      float g[8], h[8], w[8];
      for (int64_t e = lane * 8; e < p.E; e += LN * 8) {
        const int n = in_piece(p.E - e);
        fetch(base, e, n, m, r, g, h, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i >= n) g[i] = h[i] = 0.0f;
          c1 = __builtin_fmaf(g[i], w[i], c1);
          c2 = __builtin_fmaf(g[i] * w[i], h[i], c2);
        }
      }
      c1 = p.rms ? 0.0f : sum_team<LN>(c1, sm) * p.inv_e;
      c2 = sum_team<LN>(c2, sm + 4) * p.inv_e;
      for (int64_t e = lane * 8; e < p.E; e += LN * 8) {
        const int n = in_piece(p.E - e);
        fetch(base, e, n, m, r, g, h, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= w[i];
        finish(base, e, n, r, c1, c2, g, h);
      }
    }
    if constexpr (LN > 64) __syncthreads();  // sm is written again in the next row
  }
  if constexpr (P > 0) {
    if (!p.part) return;
    float* part = p.part + (int64_t)block_id() * 2 * p.E;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if constexpr (R > 1) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < P; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[(team * P * LN + k * LN + lane) * 8 + i] = which ? db[k][i] : dw[k][i];
        __syncthreads();
        for (int c = threadIdx.x; c < P * LN * 8 && c < p.E; c += 256) {
          float s = 0.0f;
          for (int t = 0; t < R; ++t) s += acc[t * P * LN * 8 + c];
          part[which * p.E + c] = s;
        }
      } else {
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const int64_t e = (int64_t)(k * LN + lane) * 8;
          const int n = in_piece(p.E - e);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < n) part[which * p.E + e + i] = which ? db[k][i] : dw[k][i];
        }
      }
    }
  }
}

// dw and db of rows too long for the registers: 256 columns and every p.blocks-th row per workgroup
template <typename XT, typename HT>
__global__ __launch_bounds__(256) void norm_sums_kernel(NormParams p) {
  const int64_t cols = (p.E + 255) / 256, blk = block_id();
  const int64_t e = blk % cols * 256 + threadIdx.x, first = blk / cols;
  if (e >= p.E || first >= p.blocks) return;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = first; row < p.rows; row += p.blocks) {
    const float d = to_f32(static_cast<const XT*>(p.x)[row * p.E + e]);
    const float h = to_f32(static_cast<const HT*>(p.residual)[row * p.E + e]);
    dw = __builtin_fmaf(d, (h - p.stats[row]) * p.stats[p.rows + row], dw);
    db += d;
  }
  p.part[first * 2 * p.E + e] = dw;
  p.part[first * 2 * p.E + p.E + e] = db;
}

// dw and db from the partial sums: 64 columns per workgroup, the partial sums split over 16 waves, each in order,
// then the waves' sums in order.
__global__ __launch_bounds__(1024) void norm_join_kernel(NormParams p) {
  __shared__ float sm[1024];
  const int64_t cols = (p.E + 63) / 64;
  const int64_t blk = block_id();
  const int64_t which = blk / cols;
  if (which > 1) return;
  const int64_t c = blk % cols * 64 + (threadIdx.x & 63);
  const int64_t per = (p.blocks + 15) / 16;
  const int64_t k0 = (threadIdx.x >> 6) * per, k1 = k0 + per < p.blocks ? k0 + per : p.blocks;
  const float* q = p.part + which * p.E + c;
  float s = 0.0f;
  if (c < p.E) {
    int64_t k = k0;
    for (; k + 8 <= k1; k += 8) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = q[(k + e) * 2 * p.E];
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[e];
    }
    for (; k < k1; ++k) s += q[k * 2 * p.E];
  }
  sm[threadIdx.x] = s;
  __syncthreads();
  float* out = which ? p.dbias : p.dweight;
  if (threadIdx.x < 64 && c < p.E && out) {
    s = 0.0f;
#pragma unroll
    for (int t = 0; t < 16; ++t) s += sm[t * 64 + threadIdx.x];
    out[c] = s;
  }
}

namespace {

template <typename XT, typename HT, int LN, int P>
void go(const NormParams& p, hipStream_t s) {
  hipLaunchKernelGGL((norm_rows_kernel<XT, HT, LN, P>), grid_of((p.rows + 256 / LN - 1) / (256 / LN)), dim3(256), 0, s, p);
}

template <typename XT, typename HT>
void fwd(const NormParams& p, hipStream_t s) {
  const int64_t n = (p.E + 7) / 8;
  if (n <= 128) {
    if (n <= 16) return go<XT, HT, 16, 1>(p, s);
    if (n <= 32) return go<XT, HT, 16, 2>(p, s);
    if (n <= 64) return go<XT, HT, 16, 4>(p, s);
    if (n <= 96) return go<XT, HT, 16, 6>(p, s);
    return go<XT, HT, 16, 8>(p, s);
  }
  if (n <= 512) {
    if (n <= 256) return go<XT, HT, 64, 4>(p, s);
    if (n <= 384) return go<XT, HT, 64, 6>(p, s);
    return go<XT, HT, 64, 8>(p, s);
  }
  if (n <= 2048) {
    if (n <= 1024) return go<XT, HT, 256, 4>(p, s);
    return go<XT, HT, 256, 8>(p, s);
  }
  go<XT, HT, 256, 0>(p, s);
}

// lanes of a row's team in the backward pass, whose sums take a register per column besides; and its pieces
int bwd_lanes(int64_t E) { return E <= 256 ? 16 : E <= 2048 ? 64 : 256; }
constexpr int64_t kBwdLongest = 8192;

template <typename XT, typename HT, int LN, int P>
void go_bwd(const NormParams& p, hipStream_t s) {
  hipLaunchKernelGGL((norm_rows_bwd_kernel<XT, HT, LN, P>), grid_of(p.blocks), dim3(256), 0, s, p);
}

template <typename XT, typename HT>
void bwd(const NormParams& p, hipStream_t s) {
  const int64_t n = (p.E + 7) / 8;
  if (p.E > kBwdLongest) {
    NormParams q = p;
    q.part = nullptr;
    q.blocks = p.rows;
    go_bwd<XT, HT, 256, 0>(q, s);
    if (p.part)
      hipLaunchKernelGGL((norm_sums_kernel<XT, HT>), grid_of((p.E + 255) / 256 * p.blocks), dim3(256), 0, s, p);
    return;
  }
  switch (bwd_lanes(p.E)) {
    case 16: return n <= 16 ? go_bwd<XT, HT, 16, 1>(p, s) : go_bwd<XT, HT, 16, 2>(p, s);
    case 64:
      if (n <= 64) return go_bwd<XT, HT, 64, 1>(p, s);
      if (n <= 128) return go_bwd<XT, HT, 64, 2>(p, s);
      return go_bwd<XT, HT, 64, 4>(p, s);
    default:
      return n <= 512 ? go_bwd<XT, HT, 256, 2>(p, s) : go_bwd<XT, HT, 256, 4>(p, s);
  }
}

}  // namespace

int64_t norm_rows_bwd_blocks(int64_t rows, int64_t E) {
  if (E > kBwdLongest) return rows < 64 ? rows : 64;
  const int64_t R = 256 / bwd_lanes(E), all = (rows + R - 1) / R;
  return all < 768 ? all : 768;
}

hipError_t launch_norm_rows(const NormParams& p, int kind, hipStream_t s) {
  if (kind == 3) fwd<bf16_t, bf16_t>(p, s);
  else if (kind == 1) fwd<bf16_t, float>(p, s);
  else fwd<float, float>(p, s);
  return hipGetLastError();
}

hipError_t launch_norm_rows_bwd(const NormParams& p, int kind, hipStream_t s) {
  if (kind == 3) bwd<bf16_t, bf16_t>(p, s);
  else if (kind == 1) bwd<bf16_t, float>(p, s);
  else bwd<float, float>(p, s);
  return hipGetLastError();
}

hipError_t launch_norm_join(const NormParams& p, hipStream_t s) {
  hipLaunchKernelGGL(norm_join_kernel, grid_of((p.E + 63) / 64 * 2), dim3(1024), 0, s, p);
  return hipGetLastError();
}

}  // namespace ssm
