// embed_fwd.hip -- embedding: out[b,t,:] = scale * weight[tokens[b,t],:], zeros for a token outside the table.
//
// Bound by HBM: the output is written once and the named rows are read once (from the caches where they
// come again).  A million letters into 1024 channels of bf16 (2.1 GB): 370 us, 5.8 TB/s (a plain fill of as many
// bytes runs at 6.9; the rows of [B,E,L] lie 2 MB apart, and no other tile, order of tiles or table in LDS came
// below 367).  The stores are marked as not needed again: through the caches it takes 612 us.
//   * [B,L,E]: a lane owns 16 aligned bytes of the output, wherever the rows begin.
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
  const int64_t total = p.T * p.E;
  const int64_t i = ((int64_t)block_id() * 256 + threadIdx.x) * V;  // the piece's first element
  if (i >= total) return;
  int64_t t, e;
  if (total <= 0xffffffffll) {
    t = (uint32_t)i / (uint32_t)p.E;
    e = (uint32_t)i - (uint32_t)t * (uint32_t)p.E;
  } else {
    t = i / p.E;
    e = i - t * p.E;
  }
  const WT* table = static_cast<const WT*>(p.table);
  int64_t row = token_at(p.tokens, p.i64, t, p.V);
  float x[V];
  if (e + V <= p.E) {
    if (row < p.V) {
      load_n<WT, V>(table + row * p.E + e, V, x);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) x[k] = 0.0f;
    }
  } else {  // the piece goes on in the next row (or rows, or ends with the last)
#pragma unroll
    for (int k = 0; k < V; ++k) {
      x[k] = row < p.V && i + k < total ? to_f32(table[row * p.E + e]) : 0.0f;
      if (++e == p.E && i + k + 1 < total) {
        e = 0;
        row = token_at(p.tokens, p.i64, ++t, p.V);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) x[k] *= p.scale;
  store_n<IO, V>(static_cast<IO*>(p.out) + i, total - i >= V ? V : (int)(total - i), x);
}

// Rows that begin at a multiple of 128 bytes (SHIFT false) take tiles of 128 positions x 64 columns.  Others would
// share a line with the next tile at each end of every column; there a column's tile begins up to a line earlier, at
// a multiple of 128 bytes, so that only a row's own ends are partial lines.  262149 letters into 1000 channels of
// bf16: 291 us with tiles where they fall, 251 with tiles at 16 bytes, 131 with these (128 x 32: 149, 512 x 32: 146,
// 256 x 64: 193); at 262144, with the aligned tiles, 102.
template <typename IO, bool SHIFT> struct Tile {
  static constexpr int V = 16 / (int)sizeof(IO);
  static constexpr int line = 128 / (int)sizeof(IO);
  static constexpr int T = SHIFT ? 256 : 128, E = SHIFT ? 32 : 64;  // positions x columns
  static constexpr int before = SHIFT ? line : 0;                 // positions kept before the tile
  static int64_t along(int64_t L) { return (L + (SHIFT ? line - 1 : 0) + T - 1) / T; }
};

template <typename WT, typename IO, bool SHIFT>
__global__ __launch_bounds__(256) void embed_cols_kernel(EmbedParams p) {
  using S = Tile<IO, SHIFT>;
  constexpr int V = S::V, kT = S::T, kE = S::E, EX = S::before;
  constexpr int LD = kT + EX + V;  // elements between columns in LDS, whole 16-byte pieces
  __shared__ __align__(16) IO sm[kE * LD];
  const int64_t tiles_t = p.tiles, tiles_e = (p.E + kE - 1) / kE;
  const int64_t blk = block_id(), te = blk % tiles_e, rest = blk / tiles_e;
  const int64_t tt = rest % tiles_t, b = rest / tiles_t;
  if (b >= p.Bsz) return;
  const int64_t t0 = tt * kT, e0 = te * kE;
  const int64_t ne = p.E - e0;
  constexpr int CPR = kE / 8, RPP = 256 / CPR * 2;  // pieces of 8 columns, positions per pass
  const int c = (threadIdx.x % CPR) * 8;
  const int n = ne - c >= 8 ? 8 : ne - c > 0 ? (int)(ne - c) : 0;
  auto fetch = [&](int r) {  // positions r and r + 1 of LDS
    float x[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t t = t0 - EX + r + k;
      int64_t row = p.V;
      if (t >= 0 && t < p.L) row = token_at(p.tokens, p.i64, b * p.L + t, p.V);
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
  };
#pragma unroll
  for (int h = 0; h < (kT + EX + RPP - 1) / RPP; ++h) {
    const int r = h * RPP + (threadIdx.x / CPR) * 2;
    if ((kT + EX) % RPP == 0 || r < kT + EX) fetch(r);
  }
  __syncthreads();
  constexpr int PPC = kT / V;  // pieces per column
#pragma unroll
  for (int h = 0; h < kE * PPC / 256; ++h) {
    const int i = h * 256 + threadIdx.x;
    const int col = i / PPC;
    if (col >= ne) continue;
    const int64_t first = (b * p.E + e0 + col) * p.L;  // of the row
    const int m = SHIFT ? (int)((first + t0) % S::line) : 0;
    const int r = (i % PPC) * V;
    const int64_t t = t0 - m + r;
    if (t >= p.L || t + V <= 0) continue;
    IO* o = static_cast<IO*>(p.out) + first + t;
    const IO* s = &sm[col * LD + EX - m + r];
    u32x4a q;
    if constexpr (!SHIFT) {
      q = *reinterpret_cast<const u32x4a*>(s);
    } else if constexpr (V == 4) {
#pragma unroll
      for (int w = 0; w < 4; ++w) q[w] = __float_as_uint(s[w]);
    } else {
      const uint32_t* d = reinterpret_cast<const uint32_t*>(s - (m & 1));
#pragma unroll
      for (int w = 0; w < 4; ++w) q[w] = m & 1 ? d[w] >> 16 | d[w + 1] << 16 : d[w];
    }
    if (t >= 0 && t + V <= p.L) {
      __builtin_nontemporal_store(q, reinterpret_cast<u32x4a*>(o));
    } else {
      for (int k = 0; k < V; ++k)
        if (t + k >= 0 && t + k < p.L) o[k] = s[k];
    }
  }
}

namespace {

template <typename WT, typename IO>
hipError_t launch(const EmbedParams& p, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(IO);
  if (p.cf && p.L % Tile<IO, false>::line == 0) {
    EmbedParams q = p;
    q.tiles = Tile<IO, false>::along(p.L);
    const int64_t blocks = p.Bsz * q.tiles * ((p.E + Tile<IO, false>::E - 1) / Tile<IO, false>::E);
    hipLaunchKernelGGL((embed_cols_kernel<WT, IO, false>), grid_of(blocks), dim3(256), 0, s, q);
  } else if (p.cf) {
    EmbedParams q = p;
    q.tiles = Tile<IO, true>::along(p.L);
    const int64_t blocks = p.Bsz * q.tiles * ((p.E + Tile<IO, true>::E - 1) / Tile<IO, true>::E);
    hipLaunchKernelGGL((embed_cols_kernel<WT, IO, true>), grid_of(blocks), dim3(256), 0, s, q);
  } else {
    const int64_t pieces = (p.T * p.E + V - 1) / V;
    hipLaunchKernelGGL((embed_rows_kernel<WT, IO>), grid_of((pieces + 255) / 256), dim3(256), 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed_fwd(const EmbedParams& p, bool table_bf16, bool io_bf16, hipStream_t s) {
  if (table_bf16) return io_bf16 ? launch<bf16_t, bf16_t>(p, s) : launch<bf16_t, float>(p, s);
  return io_bf16 ? launch<float, bf16_t>(p, s) : launch<float, float>(p, s);
}

}  // namespace ssm
