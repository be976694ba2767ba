// conv_bwd.hip -- gradients of the causal depthwise conv1d + SiLU (conv_kernels.hip).
//
//   a[t] = bias + sum_k w[k] x[t-H+k]             H = K - 1, x extended by the initial state
//   g[t] = dout[t] silu'(a[t]),  silu'(a) = s (1 + a (1 - s)),  s = 1 / (1 + e^-a)
//   dx[t] = sum_k w[k] g[t+H-k];  dw[k] = sum_t g[t] x[t-H+k];  dbias = sum_t g[t]
//
// Bound by HBM: x and dout are read once, dx is written once (6 bytes a step in bf16), and the
// pre-activation is recomputed rather than kept by the forward pass.
//
// Layout: LN lanes (64, or 16 for short rows) own one segment of LN * V * P steps of one row: a lane holds P pieces
// of 16 bytes (V steps each, LN * V steps apart) of x and dout, all in flight before any arithmetic.  A piece needs
// H inputs from its left neighbour and H values of g from its right one; both come by DPP shifts.  The
// pieces are walked from right to left, so a pass finds the g that follows its last lane in the first lane of
// the pass before; the g after the whole segment (the next segment's) is recomputed by the last lane.  Rows may
// begin at any element: the pieces lie at addresses that are multiples of 16 bytes, so the first one of a row may
// begin before it and the last one end behind it.  Each segment's K + 1 sums go to memory and are added by a
// second kernel in a fixed order.
//
// Measured: 8 x 1536 x 2048 in bf16, width 4 (151 MB): 30 us, 5.1 TB/s, and 4 for the sums; 1 x 509 x 262147, width 3,
// with states (801 MB): 150 us, 5.3 TB/s; a copy runs at 5.2.  About 33 instructions a step.  On the way there: 39 and
// 219 us with pieces that begin where the row does; 37 and 150 with aligned ones, 32-bit positions and DPP shifts;
// 30 for the first once whole rows took the initial state's gradient from registers.
#include "../ssm_device.h"
#include "train_device.h"
#include "train_launch.h"

namespace ssm {

namespace {

constexpr int kPasses = 4;  // 2: 47 and 187 us a call for the two sizes above, 8: 77 and 190, where 4 took 43 and 155

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 16 bytes as V = 8 or 4 floats
__device__ __forceinline__ void widen(const u32x4& q, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(q[i] << 16);
    x[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen(const u32x4& q, float (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(q[i]);
}
__device__ __forceinline__ u32x4 narrow(const float (&x)[8]) {
  u32x4 q;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i]) |
           ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i + 1]) << 16);
  return q;
}
__device__ __forceinline__ u32x4 narrow(const float (&x)[4]) {
  return u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
}
__device__ __forceinline__ uint32_t bits_of(bf16_t v) { return v; }
__device__ __forceinline__ uint32_t bits_of(float v) { return __float_as_uint(v); }

// The piece at p; where it is not whole, its elements lo..hi-1 (the others are zero).
template <typename IO>
__device__ __forceinline__ u32x4 load_piece(const IO* p, int lo, int hi) {
  constexpr int V = 16 / (int)sizeof(IO);
  if (lo == 0 && hi == V) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  u32x4 q = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i >= lo && i < hi) {
      if constexpr (V == 8) q[i >> 1] |= bits_of(p[i]) << (16 * (i & 1));
      else q[i] = bits_of(p[i]);
    }
  return q;
}

// The value of the lane to the left (right) in the group of LN lanes; its first (last) lane gets `end`.
template <int LN>
__device__ __forceinline__ uint32_t from_left(uint32_t v, uint32_t end) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)end, (int)v, LN == 64 ? 0x138 : 0x111, 0xf, 0xf, false);
}
template <int LN>
__device__ __forceinline__ float from_right(float v, float end) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)__float_as_uint(end), (int)__float_as_uint(v),
                                                               LN == 64 ? 0x130 : 0x101, 0xf, 0xf, false));
}
// the group's first or last lane's value, in all of its lanes
template <int LN, bool LAST>
__device__ __forceinline__ uint32_t of_lane(uint32_t v) {
  if constexpr (LN == 64) return (uint32_t)__builtin_amdgcn_readlane((int)v, LAST ? 63 : 0);
  else return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, LAST ? 0x15f : 0x150, 0xf, 0xf, true);
}

__device__ __forceinline__ float silu_slope(float a) {
  const float s = rcp_(1.0f + exp2_(-a * kLog2e));
  return s * __builtin_fmaf(a, 1.0f - s, 1.0f);
}

}  // namespace

template <typename IO, int K, int LN>
__global__ __launch_bounds__(256, LN == 64 ? 5 : 4) void conv_bwd_kernel(ConvBwdParams p) {
  constexpr int V = 16 / (int)sizeof(IO);
  constexpr int H = K - 1, HA = H > 0 ? H : 1;
  constexpr int P = kPasses;
  constexpr int W = (H * (int)sizeof(IO) + 3) / 4;  // words that hold a piece's last H steps
  constexpr int SEG = LN * V * P;
  const int lane = threadIdx.x % LN;
  // row segment; their number fits 31 bits, so the divisions take 32
  uint32_t unit = block_id() * (256 / LN) + threadIdx.x / LN;
  if constexpr (LN == 64) unit = (uint32_t)__builtin_amdgcn_readfirstlane((int)unit);  // scalar from here on
  const bool live = unit < p.units;
  unit = live ? unit : 0;
  const uint32_t r32 = unit / (uint32_t)p.S, s32 = unit - r32 * (uint32_t)p.S;
  const uint32_t b32 = r32 / (uint32_t)p.Dm, d32 = r32 - b32 * (uint32_t)p.Dm;
  const int64_t row = r32, seg = s32, d = d32;
  const IO* x = static_cast<const IO*>(p.x) + row * p.L;
  const IO* dout = static_cast<const IO*>(p.dout) + row * p.L;
  const IO* init = p.init && live ? static_cast<const IO*>(p.init) + row * H : nullptr;
  const IO* dfin = p.dfinal && live ? static_cast<const IO*>(p.dfinal) + row * H : nullptr;
  const int64_t L = live ? p.L : 0;
  // the segment's first step: the row's first piece begins up to V - 1 steps before the row
  const int64_t t0 = seg * SEG - (row * p.L) % V;
  const int begin = t0 < 0 ? (int)-t0 : 0;                     // of the row within the segment
  const int end = L - t0 < SEG + 8 ? (int)(L - t0) : SEG + 8;  // where it lies within the segment or close behind
  x += t0;
  dout += t0;

  u32x4 xq[P], gq[P];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int i = (j * LN + lane) * V;
    const int lo = begin - i > 0 ? begin - i : 0, hi = end - i < V ? end - i : V;
    xq[j] = load_piece(x + i, lo, hi);
    gq[j] = load_piece(dout + i, lo, hi);
  }
  float w[K];
#pragma unroll
  for (int k = 0; k < K; ++k) w[k] = p.w[d * K + k];
  const float bias = p.bias ? p.bias[d] : 0.0f;

  // single steps, counted from the segment's first, for its ends
  auto input = [&](int i) -> uint32_t {
    if (t0 + i >= 0) return i < end ? bits_of(x[i]) : 0u;
    return init && t0 + i >= -H ? bits_of(init[H + t0 + i]) : 0u;
  };
  auto value = [](uint32_t v) -> float { return __uint_as_float(sizeof(IO) == 2 ? v << 16 : v); };
  auto gradient = [&](int i, float (&g)[HA]) {  // g of the H steps from i on
    if constexpr (H > 0) {
      float xv[2 * H];
#pragma unroll
      for (int k = 0; k < 2 * H; ++k) xv[k] = value(input(i - H + k));
#pragma unroll
      for (int e = 0; e < H; ++e) {
        float a = bias;
#pragma unroll
        for (int k = 0; k < K; ++k) a = __builtin_fmaf(w[k], xv[e + k], a);
        g[e] = i + e < end ? to_f32(dout[i + e]) * silu_slope(a) : 0.0f;
      }
    }
  };
  auto initial = [&](const float* g) {  // dx at the steps before the row, from the row's first g
    IO* di = static_cast<IO*>(p.dinit) + row * H;
#pragma unroll
    for (int i = 0; i < H; ++i) {  // step i - H
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k <= i; ++k) s = __builtin_fmaf(w[k], g[i - k], s);
      if (dfin && i >= L) s += to_f32(dfin[i - L]);  // L < H: the final state still holds it
      store_io(di + i, s);
    }
  };
  uint32_t before[W > 0 ? W : 1];  // the words before the segment (first lane)
  float after[HA];                 // g behind it (last lane)
#pragma unroll
  for (int k = 0; k < (W > 0 ? W : 1); ++k) before[k] = 0u;
#pragma unroll
  for (int k = 0; k < HA; ++k) after[k] = 0.0f;
  if constexpr (H > 0) {
    if (lane == 0 && (t0 > 0 || init || begin > 0)) {
#pragma unroll
      for (int k = 0; k < W; ++k) {
        if constexpr (V == 8) before[k] = input(-2 * (W - k)) | input(-2 * (W - k) + 1) << 16;
        else before[k] = input(k - W);
      }
      if (begin > 0) {  // the steps before the row in its first piece are the initial state
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (e < begin) {
            if constexpr (V == 8) xq[0][e >> 1] |= input(e) << (16 * (e & 1));
            else xq[0][e] = input(e);
          }
      }
      if (begin > 0 && p.dinit) {  // the row's first g may lie in two lanes
        float g[HA];
        gradient(begin, g);
        initial(g);
      }
    }
    if (lane == LN - 1 && end > SEG) gradient(SEG, after);
  }

  float sw[K], sb = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k) sw[k] = 0.0f;
#pragma unroll
  for (int j = P - 1; j >= 0; --j) {
    float xe[H + V], xv[V], go[V];  // xe: the piece and the H inputs before it
    widen(xq[j], xv);
    widen(gq[j], go);
    if constexpr (H > 0) {
      u32x4 left = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const uint32_t end = j > 0 ? of_lane<LN, true>(xq[j > 0 ? j - 1 : 0][4 - W + k]) : before[k];
        left[4 - W + k] = from_left<LN>(xq[j][4 - W + k], end);
      }
      float lv[V];
      widen(left, lv);
#pragma unroll
      for (int k = 0; k < H; ++k) xe[k] = lv[V - H + k];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) xe[H + e] = xv[e];
    float ge[V + HA];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float a = bias;
#pragma unroll
      for (int k = 0; k < K; ++k) a = __builtin_fmaf(w[k], xe[e + k], a);
      ge[e] = go[e] * silu_slope(a);
      sb += ge[e];
#pragma unroll
      for (int k = 0; k < K; ++k) sw[k] = __builtin_fmaf(ge[e], xe[e + k], sw[k]);
    }
#pragma unroll
    for (int k = 0; k < H; ++k) {
      ge[V + k] = from_right<LN>(ge[k], after[k]);
      after[k] = __uint_as_float(of_lane<LN, false>(__float_as_uint(ge[k])));
    }
    const int i = (j * LN + lane) * V;
    float dxe[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k) s = __builtin_fmaf(w[k], ge[e + H - k], s);
      dxe[e] = s;
    }
    if constexpr (H > 0) {
      if (j == 0 && lane == 0 && seg == 0 && begin == 0 && live && p.dinit) initial(ge);
      if (dfin && i + V > end - H) {  // the last H inputs are the final state
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int q = i + e - (end - H);
          if (q >= 0 && q < H) dxe[e] += to_f32(dfin[q]);
        }
      }
    }
    IO* dx = static_cast<IO*>(p.dx) + row * p.L + t0 + i;
    if (i >= begin && i + V <= end) {
      __builtin_nontemporal_store(narrow(dxe), reinterpret_cast<u32x4*>(dx));
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (i + e >= begin && i + e < end) store_io(dx + e, dxe[e]);
    }
  }

  // the segment's sums over its lanes
  sb = sum_lanes<LN>(sb);
#pragma unroll
  for (int k = 0; k < K; ++k) sw[k] = sum_lanes<LN>(sw[k]);
  if (live && lane == 0) {
    const bool whole = p.Bsz * p.S == 1;  // the only segment of its channel: these are the results
    float* o = whole ? p.dw + d * K : p.part + (((int64_t)b32 * p.S + seg) * p.Dm + d) * (K + 1);
#pragma unroll
    for (int k = 0; k < K; ++k) o[k] = sw[k];
    if (!whole) o[K] = sb;
    else if (p.db) p.db[d] = sb;
  }
}

// dweight and dbias from the partial sums: 64 outputs per workgroup, the partials split over 4 waves,
// each in order, then the waves' sums in order.
__global__ __launch_bounds__(256) void conv_bwd_join_kernel(const float* part, int64_t count, int64_t Dm, int K,
                                                            float* dw, float* db) {
  const int64_t n = Dm * (K + 1);
  const int64_t i = (int64_t)block_id() * 64 + (threadIdx.x & 63);
  const int64_t per = (count + 3) / 4;
  const int64_t k0 = (threadIdx.x >> 6) * per, k1 = k0 + per < count ? k0 + per : count;
  float s = 0.0f;
  if (i < n) {
    int64_t k = k0;
    for (; k + 8 <= k1; k += 8) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = part[(k + e) * n + i];
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[e];
    }
    for (; k < k1; ++k) s += part[k * n + i];
  }
  __shared__ float sm[256];
  sm[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x < 64 && i < n) {
    s = sm[threadIdx.x] + sm[threadIdx.x + 64] + sm[threadIdx.x + 128] + sm[threadIdx.x + 192];
    const int64_t d = i / (K + 1);
    const int k = (int)(i - d * (K + 1));
    if (k < K) dw[d * K + k] = s;
    else if (db) db[d] = s;
  }
}

// Rows of up to 32 pieces take 16 lanes each, so that a wave has 4 of them: with 64 half of its lanes or more
// would be idle.
int64_t conv_bwd_segments(int64_t L, bool bf16, int* lanes) {
  const int64_t V = bf16 ? 8 : 4;
  *lanes = L <= 32 * V ? 16 : 64;
  const int64_t seg = *lanes * V * kPasses;
  return (L + (L % V ? V - 1 : 0) + seg - 1) / seg;  // rows of whole pieces all begin with one
}

namespace {

template <typename IO, int K>
void launch_k(const ConvBwdParams& p, hipStream_t s) {
  if (p.lanes == 16)
    hipLaunchKernelGGL((conv_bwd_kernel<IO, K, 16>), grid_of((p.units + 15) / 16), dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((conv_bwd_kernel<IO, K, 64>), grid_of((p.units + 3) / 4), dim3(256), 0, s, p);
}

template <typename IO>
void launch_io(const ConvBwdParams& p, hipStream_t s) {
  switch (p.K) {
    case 1: return launch_k<IO, 1>(p, s);
    case 2: return launch_k<IO, 2>(p, s);
    case 3: return launch_k<IO, 3>(p, s);
    default: return launch_k<IO, 4>(p, s);
  }
}

}  // namespace

hipError_t launch_conv_bwd(const ConvBwdParams& p, bool bf16, hipStream_t s) {
  if (bf16) launch_io<bf16_t>(p, s);
  else launch_io<float>(p, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.Bsz * p.S == 1) return e;
  hipLaunchKernelGGL(conv_bwd_join_kernel, grid_of((p.Dm * (p.K + 1) + 63) / 64), dim3(256), 0, s, p.part,
                     p.Bsz * p.S, p.Dm, p.K, p.dw, p.db);
  return hipGetLastError();
}

}  // namespace ssm
