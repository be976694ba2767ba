// embed_fwd.hip -- embedding: out[b,t,:] = scale * weight[tokens[b,t],:], zeros for a token outside the table.
//
// Bound by HBM: the output is written once and the named rows are read once (from the caches where they
// come again).
//   * [B,L,E]: a lane owns V output elements (16 bytes) of a row; lanes run over the rows' pieces.
//   * [B,E,L]: a workgroup turns a tile of kT positions x kE columns through LDS: a lane reads 8
//     consecutive columns of two neighbouring positions, writes them as pairs, and later reads
//     consecutive positions of one column, so both sides move whole lines.
#include "../ssm_device.h"
#include "train_device.h"
#include "train_launch.h"

namespace ssm {

template <typename WT, typename IO>
__global__ __launch_bounds__(256) void embed_rows_kernel(EmbedParams p) {
  constexpr int V = 16 / (int)sizeof(IO);
  const int64_t cpr = (p.E + V - 1) / V;  // pieces per row
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.T * cpr) return;
  int64_t t, c;
  if (p.T * cpr <= 0xffffffffll) {
    t = (uint32_t)i / (uint32_t)cpr;
    c = (uint32_t)i - (uint32_t)t * (uint32_t)cpr;
  } else {
    t = i / cpr;
    c = i - t * cpr;
  }
  const int64_t e = c * V;
  const int n = p.E - e < V ? (int)(p.E - e) : V;
  const int64_t row = token_at(p.tokens, p.i64, t, p.V);
  float x[V];
  if (row < p.V) {
    load_n<WT, V>(static_cast<const WT*>(p.table) + row * p.E + e, n, x);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) x[k] = 0.0f;
  }
#pragma unroll
  for (int k = 0; k < V; ++k) x[k] *= p.scale;
  store_n<IO, V>(static_cast<IO*>(p.out) + t * p.E + e, n, x);
}

constexpr int kT = 128, kE = 64;  // positions x columns of a tile

template <typename WT, typename IO>
__global__ __launch_bounds__(256) void embed_cols_kernel(EmbedParams p) {
  constexpr int V = 16 / (int)sizeof(IO);
  constexpr int LD = kT + 16 / (int)sizeof(IO);  // elements between columns in LDS, whole 16-byte pieces
  __shared__ __align__(16) IO sm[kE * LD];
  const int64_t tiles_t = (p.L + kT - 1) / kT, tiles_e = (p.E + kE - 1) / kE;
  const int64_t blk = blockIdx.x;
  const int64_t te = blk % tiles_e, rest = blk / tiles_e;
  const int64_t tt = rest % tiles_t, b = rest / tiles_t;
  const int64_t t0 = tt * kT, e0 = te * kE;
  const int64_t nt = p.L - t0, ne = p.E - e0;
  {
    const int c = (threadIdx.x & 7) * 8;  // first column
    const int n = ne - c >= 8 ? 8 : ne - c > 0 ? (int)(ne - c) : 0;
#pragma unroll
    for (int h = 0; h < kT / 64; ++h) {
      const int r = h * 64 + (threadIdx.x >> 3) * 2;  // first of two positions
      float x[2][8];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        int64_t row = p.V;
        if (r + k < nt) row = token_at(p.tokens, p.i64, b * p.L + t0 + r + k, p.V);
        if (row < p.V) {
          load_n<WT, 8>(static_cast<const WT*>(p.table) + row * p.E + e0 + c, n, x[k]);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) x[k][q] = 0.0f;
        }
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if constexpr (sizeof(IO) == 2) {
          const uint32_t lo = __builtin_bit_cast(uint16_t, (__bf16)(x[0][q] * p.scale));
          const uint32_t hi = __builtin_bit_cast(uint16_t, (__bf16)(x[1][q] * p.scale));
          *reinterpret_cast<uint32_t*>(&sm[(c + q) * LD + r]) = lo | (hi << 16);
        } else {
          *reinterpret_cast<float2*>(&sm[(c + q) * LD + r]) = make_float2(x[0][q] * p.scale, x[1][q] * p.scale);
        }
      }
    }
  }
  __syncthreads();
  constexpr int PPC = kT / V;  // pieces per column
#pragma unroll
  for (int h = 0; h < kE * PPC / 256; ++h) {
    const int i = h * 256 + threadIdx.x;
    const int col = i / PPC, r = (i % PPC) * V;
    if (col >= ne || r >= nt) continue;
    const int n = nt - r < V ? (int)(nt - r) : V;
    IO* o = static_cast<IO*>(p.out) + (b * p.E + e0 + col) * p.L + t0 + r;
    const u32x4a q = *reinterpret_cast<const u32x4a*>(&sm[col * LD + r]);
    if (n == V) {
      __builtin_nontemporal_store((typename Unaligned<IO>::type)q, reinterpret_cast<typename Unaligned<IO>::type*>(o));
    } else {
      for (int k = 0; k < n; ++k) o[k] = sm[col * LD + r + k];
    }
  }
}

namespace {

template <typename WT, typename IO>
hipError_t launch(const EmbedParams& p, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(IO);
  if (p.cf) {
    const int64_t blocks = p.Bsz * ((p.L + kT - 1) / kT) * ((p.E + kE - 1) / kE);
    hipLaunchKernelGGL((embed_cols_kernel<WT, IO>), dim3((unsigned)blocks), dim3(256), 0, s, p);
  } else {
    const int64_t pieces = p.T * ((p.E + V - 1) / V);
    hipLaunchKernelGGL((embed_rows_kernel<WT, IO>), dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed_fwd(const EmbedParams& p, bool table_bf16, bool io_bf16, hipStream_t s) {
  if (table_bf16) return io_bf16 ? launch<bf16_t, bf16_t>(p, s) : launch<bf16_t, float>(p, s);
  return io_bf16 ? launch<float, bf16_t>(p, s) : launch<float, float>(p, s);
}

}  // namespace ssm
