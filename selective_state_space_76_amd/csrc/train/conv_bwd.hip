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
// H inputs from its left neighbour and H values of g from its right one; both come by cross-lane
// moves.  The pieces are walked from right to left, so a pass finds the g that follows its last lane
// in the first lane of the pass before; the g after the whole segment (the next segment's) is
// recomputed by the last lane.  Rows may begin at any element: the pieces are loaded at the alignment
// of one element, so odd lengths take the same path.  Each segment's K + 1 sums go to memory and are added
// by a second kernel in a fixed order.
#include "../ssm_device.h"
#include "train_launch.h"

namespace ssm {

namespace {

constexpr int kPasses = 4;

template <typename IO> struct Piece;
template <> struct Piece<float> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4))); };
template <> struct Piece<bf16_t> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2))); };

// V steps from p, of which the first c exist (the others are zero)
template <typename IO, int V>
__device__ __forceinline__ void load_piece(const IO* p, int c, float (&x)[V]) {
  if (c >= V) {
    const auto q = __builtin_nontemporal_load(reinterpret_cast<const typename Piece<IO>::type*>(p));
    if constexpr (V == 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(q[i] << 16);
        x[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(q[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = i < c ? to_f32(p[i]) : 0.0f;
  }
}

template <typename IO, int V>
__device__ __forceinline__ void store_piece(IO* p, int c, const float (&x)[V]) {
  if (c >= V) {
    typename Piece<IO>::type q;
    if constexpr (V == 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        q[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i]) |
               ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i + 1]) << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = __float_as_uint(x[i]);
    }
    __builtin_nontemporal_store(q, reinterpret_cast<typename Piece<IO>::type*>(p));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < c) store_io(p + i, x[i]);
  }
}

__device__ __forceinline__ float silu_slope(float a) {
  const float s = rcp_(1.0f + exp2_(-a * kLog2e));
  return s * __builtin_fmaf(a, 1.0f - s, 1.0f);
}

}  // namespace

template <typename IO, int K, int LN>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvBwdParams p) {
  constexpr int V = 16 / (int)sizeof(IO);
  constexpr int H = K - 1, HA = H > 0 ? H : 1;
  constexpr int P = kPasses;
  const int64_t rows = p.Bsz * p.Dm;
  const int64_t unit = (int64_t)blockIdx.x * (256 / LN) + threadIdx.x / LN;  // row segment
  const int lane = threadIdx.x % LN;
  const bool live = unit < rows * p.S;
  const int64_t row = live ? unit / p.S : 0, seg = live ? unit - row * p.S : 0;
  const int64_t d = row % p.Dm;
  const IO* x = static_cast<const IO*>(p.x) + row * p.L;
  const IO* dout = static_cast<const IO*>(p.dout) + row * p.L;
  IO* dx = static_cast<IO*>(p.dx) + row * p.L;
  const IO* init = p.init ? static_cast<const IO*>(p.init) + row * H : nullptr;
  const IO* dfin = p.dfinal ? static_cast<const IO*>(p.dfinal) + row * H : nullptr;
  const int64_t t0 = seg * (LN * V * P);  // the segment's first step
  const int64_t L = live ? p.L : 0;

  float xs[P][V], go[P][V];
  int cnt[P];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int64_t t = t0 + (j * LN + lane) * V;
    const int64_t left = L - t;
    cnt[j] = left >= V ? V : left > 0 ? (int)left : 0;
    load_piece<IO, V>(x + t, cnt[j], xs[j]);
    load_piece<IO, V>(dout + t, cnt[j], go[j]);
  }
  float w[K];
#pragma unroll
  for (int k = 0; k < K; ++k) w[k] = p.w[d * K + k];
  const float bias = p.bias ? p.bias[d] : 0.0f;

  // the H inputs before the segment (lane 0 uses them), and g of the H steps after it (last lane)
  auto input = [&](int64_t t) -> float {
    if (t >= 0) return t < L ? to_f32(x[t]) : 0.0f;
    return init && live && t >= -H ? to_f32(init[H + t]) : 0.0f;
  };
  float before[HA], after[HA];
#pragma unroll
  for (int k = 0; k < HA; ++k) before[k] = after[k] = 0.0f;
  if constexpr (H > 0) {
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < H; ++k) before[k] = input(t0 - H + k);
    }
    const int64_t te = t0 + LN * V * P;
    if (lane == LN - 1 && te < L) {
      float xv[2 * H];
#pragma unroll
      for (int k = 0; k < 2 * H; ++k) xv[k] = input(te - H + k);
#pragma unroll
      for (int e = 0; e < H; ++e) {
        float a = bias;
#pragma unroll
        for (int k = 0; k < K; ++k) a = __builtin_fmaf(w[k], xv[e + k], a);
        after[e] = te + e < L ? to_f32(dout[te + e]) * silu_slope(a) : 0.0f;
      }
    }
  }

  float sw[K], sb = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k) sw[k] = 0.0f;
#pragma unroll
  for (int j = P - 1; j >= 0; --j) {
    float xe[H + V];  // the piece and the H inputs before it
#pragma unroll
    for (int k = 0; k < H; ++k) {
      float left = __shfl_up(xs[j][V - H + k], 1, LN);
      const float prev = j > 0 ? __shfl(xs[j > 0 ? j - 1 : 0][V - H + k], LN - 1, LN) : before[k];
      xe[k] = lane == 0 ? prev : left;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) xe[H + e] = xs[j][e];
    float ge[V + HA];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float a = bias;
#pragma unroll
      for (int k = 0; k < K; ++k) a = __builtin_fmaf(w[k], xe[e + k], a);
      ge[e] = go[j][e] * silu_slope(a);
      sb += ge[e];
#pragma unroll
      for (int k = 0; k < K; ++k) sw[k] = __builtin_fmaf(ge[e], xe[e + k], sw[k]);
    }
    float first[HA];
#pragma unroll
    for (int k = 0; k < H; ++k) {
      const float right = __shfl_down(ge[k], 1, LN);
      first[k] = __shfl(ge[k], 0, LN);
      ge[V + k] = lane == LN - 1 ? after[k] : right;
    }
#pragma unroll
    for (int k = 0; k < H; ++k) after[k] = first[k];
    const int64_t t = t0 + (j * LN + lane) * V;
    float dxe[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k) s = __builtin_fmaf(w[k], ge[e + H - k], s);
      dxe[e] = s;
    }
    if constexpr (H > 0) {
      if (dfin && t + V > L - H) {  // the last H inputs are the final state
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int64_t q = t + e - (L - H);
          if (q >= 0 && q < H) dxe[e] += to_f32(dfin[q]);
        }
      }
      if (j == 0 && t == 0 && p.dinit && live) {
        IO* di = static_cast<IO*>(p.dinit) + row * H;
#pragma unroll
        for (int i = 0; i < H; ++i) {  // step i - H
          float s = 0.0f;
#pragma unroll
          for (int k = 0; k <= i; ++k) s = __builtin_fmaf(w[k], ge[i - k], s);
          if (dfin && i >= L) s += to_f32(dfin[i - L]);  // L < H: the final state still holds it
          store_io(di + i, s);
        }
      }
    }
    if (cnt[j] > 0) store_piece<IO, V>(dx + t, cnt[j], dxe);
  }

  // the segment's sums over its lanes
#pragma unroll
  for (int o = LN / 2; o > 0; o >>= 1) {
    sb += __shfl_xor(sb, o, LN);
#pragma unroll
    for (int k = 0; k < K; ++k) sw[k] += __shfl_xor(sw[k], o, LN);
  }
  if (live && lane == 0) {
    const int64_t b = row / p.Dm;
    float* o = p.part + ((b * p.S + seg) * p.Dm + d) * (K + 1);
#pragma unroll
    for (int k = 0; k < K; ++k) o[k] = sw[k];
    o[K] = sb;
  }
}

// dweight and dbias from the partial sums: 64 outputs per workgroup, the partials split over 4 waves,
// each in order, then the waves' sums in order.
__global__ __launch_bounds__(256) void conv_bwd_join_kernel(const float* part, int64_t count, int64_t Dm, int K,
                                                            float* dw, float* db) {
  const int64_t n = Dm * (K + 1);
  const int64_t i = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
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

// Short rows take 16 lanes each, so that a wave has 4 of them.
int64_t conv_bwd_segments(int64_t L, bool bf16, int* lanes) {
  const int64_t V = bf16 ? 8 : 4;
  *lanes = L <= 32 * V ? 16 : 64;
  const int64_t seg = *lanes * V * kPasses;
  return (L + seg - 1) / seg;
}

namespace {

template <typename IO, int K>
void launch_k(const ConvBwdParams& p, hipStream_t s) {
  const int64_t units = p.Bsz * p.Dm * p.S;
  if (p.lanes == 16)
    hipLaunchKernelGGL((conv_bwd_kernel<IO, K, 16>), dim3((unsigned)((units + 15) / 16)), dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((conv_bwd_kernel<IO, K, 64>), dim3((unsigned)((units + 3) / 4)), dim3(256), 0, s, p);
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
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(conv_bwd_join_kernel, dim3((unsigned)((p.Dm * (p.K + 1) + 63) / 64)), dim3(256), 0, s, p.part,
                     p.Bsz * p.S, p.Dm, p.K, p.dw, p.db);
  return hipGetLastError();
}

}  // namespace ssm
