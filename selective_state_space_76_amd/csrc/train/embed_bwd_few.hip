// embed_bwd_few.hip -- gradient of the embedding for a table of few rows (letters), dout in the scan's [B,E,L].
//
// With few rows the sum over the positions of each token is a product: dweight[v,e] = scale * sum_t [token_t = v]
// dout[e,t].  Positions are contiguous in dout, as the matrix cores want the summed index of their right
// operand; the left operand, ones and zeros, is made from the tokens in registers for
// v_mfma_f32_16x16x32_bf16 (16x16x4 in fp32).  Products with one and zero are exact, the sums are fp32.  No
// sort, no transposed copy.
//
// A workgroup owns 64 channels (16 per wave) and `seg` positions of one batch row.  A wave moves a tile of 1 KB of
// each of its 16 channels at a time from memory to registers (a load per channel, 1 KB in one piece), from
// there to its own LDS, and from LDS into the products, while the next tile is on its way; the pieces of 16 bytes
// lie rotated by xor with the channel, so that the products' reads, 16 channels at one position, meet all
// banks.  The segments' sums are added by a second kernel in order.
//
// Bound by HBM: dout is read once.  For a million letters and 1024 channels in bf16 (2.1 GB): 371 us, 5.8 TB/s, at
// the rate of a plain sum over as many bytes (6.0 TB/s).  With the products fed straight from memory (each load
// 64 bytes of 16 channels that lie 2 MB apart) it took 636 us with the loads marked as not needed again, which
// dropped half-used lines, 532 without, 480 and 442 with 512 and 1024 bytes of a channel per step; through LDS
// 502 with 8192 positions per workgroup (one workgroup per CU), 377 with 4096, 371 with 2048, 420 with 1024.
//
// 0 * x is not 0 where x is infinite or NaN.  What lies at positions whose token is outside the table is cleared
// on the way; where a workgroup still meets such a value it adds its segment up again by selection.
#include "../ssm_device.h"
#include "train_device.h"
#include "train_launch.h"

namespace ssm {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

struct FewParams {
  const void* tokens;
  const void* dout;   // [B,E,L]
  void* dweight;
  float* part;        // [segs][V][E]
  int64_t L, V, E, seg, segs_row, segs, groups;
  float scale;
  int i64, add;
};

constexpr int kMaxSeg = 2048;

// 4 words of a channel from element t on; past the row's end zero
template <typename IO>
__device__ __forceinline__ u32x4a words(const IO* row, int64_t t, int64_t L, bool live) {
  constexpr int V = 16 / (int)sizeof(IO);
  if (live && t + V <= L) {
    const auto q = __builtin_nontemporal_load(reinterpret_cast<const typename Unaligned<IO>::type*>(row + t));
    return u32x4a{q[0], q[1], q[2], q[3]};
  }
  u32x4a w = {0u, 0u, 0u, 0u};
  if (live && t < L) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + i < L) {
        if constexpr (sizeof(IO) == 2) w[i >> 1] |= (uint32_t)row[t + i] << (16 * (i & 1));
        else w[i] = __float_as_uint(row[t + i]);
      }
  }
  return w;
}

}  // namespace

template <typename IO, int MT>
__global__ __launch_bounds__(256) void embed_few_kernel(FewParams p) {
  constexpr bool BF = sizeof(IO) == 2;
  constexpr int V = 16 / (int)sizeof(IO);
  constexpr int STEP = 64 * V;  // positions at a time: 1 KB of each channel
  __shared__ __align__(16) uint16_t tok[kMaxSeg];   // 0xffff: no row
  __shared__ __align__(16) u32x4a tile[4][16][64];  // per wave: 16 channels; piece c of channel k lies at c ^ k
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 15, g = lane >> 4;
  const int64_t grp = block_id() % p.groups, seg = block_id() / p.groups;
  if (seg >= p.segs) return;
  const int64_t b = seg / p.segs_row, t0 = (seg - b * p.segs_row) * p.seg;
  const int64_t e0 = grp * 64;
  const IO* base = static_cast<const IO*>(p.dout) + (b * p.E + e0) * p.L;
  for (int i = threadIdx.x; i < p.seg; i += 256) {
    const int64_t k = t0 + i < p.L ? token_at(p.tokens, p.i64, b * p.L + t0 + i, p.V) : p.V;
    tok[i] = k < p.V ? (uint16_t)k : 0xffffu;
  }
  f32x4 acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  u16x2 big16 = {0, 0};
  uint32_t big32 = 0;
  u32x4a next[16];
  const IO* mine = base + wave * 16 * p.L;
  auto fetch = [&](int i) {
    const int64_t t = t0 + i + lane * V;
#pragma unroll
    for (int k = 0; k < 16; ++k)
      next[k] = words<IO>(mine + k * p.L, t, p.L, e0 + wave * 16 + k < p.E);
  };
  const int64_t here = p.L - t0 < p.seg ? p.L - t0 : p.seg;
  fetch(0);
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < here; i += STEP) {
#pragma unroll
    for (int k = 0; k < 16; ++k) tile[wave][k][lane ^ k] = next[k];
    wave_sync();
    if (i + STEP < here) fetch(i + STEP);
#pragma unroll
    for (int s = 0; s < 16; ++s) {
      const int c = s * 4 + g;  // the lane's piece: V positions of channel n
      const u32x4a x = tile[wave][n][c ^ n];
      if constexpr (BF) {
        const u32x4a tk = *reinterpret_cast<const u32x4a*>(&tok[i + c * 8]);  // 8 tokens
        u32x4a y;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
          const uint32_t two = tk[w];  // (a bit cast of tk[w] itself would read tk[0])
          const i16x2 neg = __builtin_bit_cast(i16x2, two) >> 15;  // ones where the token has no row
          y[w] = x[w] & ~__builtin_bit_cast(uint32_t, neg);
          big16 = __builtin_elementwise_max(big16, __builtin_bit_cast(u16x2, y[w] & 0x7fff7fffu));
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          u32x4a a;
          const uint32_t row = (uint32_t)(m * 16 + n) * 0x10001u;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const u16x2 d = __builtin_elementwise_min(__builtin_bit_cast(u16x2, tk[w] ^ row), u16x2{1, 1});
            a[w] = (__builtin_bit_cast(uint32_t, d) ^ 0x10001u) * 0x3f80u;  // 1.0 in bf16 where they agree
          }
          acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, y),
                                                           acc[m], 0, 0, 0);
        }
      } else {
        const uint2 tk = *reinterpret_cast<const uint2*>(&tok[i + c * 4]);  // 4 tokens
        const uint32_t t4[4] = {tk.x & 0xffffu, tk.x >> 16, tk.y & 0xffffu, tk.y >> 16};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t y = t4[j] == 0xffffu ? 0u : x[j], a = y & 0x7fffffffu;
          big32 = big32 > a ? big32 : a;
#pragma unroll
          for (int m = 0; m < MT; ++m)
            acc[m] = __builtin_amdgcn_mfma_f32_16x16x4f32(t4[j] == (uint32_t)(m * 16 + n) ? 1.0f : 0.0f,
                                                          __uint_as_float(y), acc[m], 0, 0, 0);
        }
      }
    }
    wave_sync();  // the tile has been read
  }
  const int bad = BF ? (big16[0] >= 0x7f80u || big16[1] >= 0x7f80u) : big32 >= 0x7f800000u;
  float* out = p.part + seg * p.V * p.E;
  if (__syncthreads_or(bad)) {  // by selection: every token's sum sees its own values only
    const int64_t e = e0 + lane;
    if (e >= p.E) return;
    const int64_t m = p.L - t0 < p.seg ? p.L - t0 : p.seg;
    for (int v = wave; v < p.V; v += 4) {
      float s = 0.0f;
      for (int64_t i = 0; i < m; ++i)
        if (tok[i] == v) s += to_f32(base[lane * p.L + t0 + i]);
      out[v * p.E + e] = s;
    }
    return;
  }
  // lane: rows 4 g + i of a tile, channel n
  const int64_t e = e0 + wave * 16 + n;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int v = m * 16 + g * 4 + i;
      if (v < p.V && e < p.E) out[v * p.E + e] = acc[m][i];
    }
}

// dweight from the segments' sums: 64 elements per workgroup, the segments split over 4 waves, each in order,
// then the waves' sums in order.
template <typename OT>
__global__ __launch_bounds__(256) void embed_few_join_kernel(FewParams p) {
  const int64_t n = p.V * p.E;
  const int64_t i = (int64_t)block_id() * 64 + (threadIdx.x & 63);
  const int64_t per = (p.segs + 3) / 4;
  const int64_t k0 = (threadIdx.x >> 6) * per, k1 = k0 + per < p.segs ? k0 + per : p.segs;
  float s = 0.0f;
  if (i < n) {
    int64_t k = k0;
    for (; k + 16 <= k1; k += 16) {
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = p.part[(k + e) * n + i];
#pragma unroll
      for (int e = 0; e < 16; ++e) s += v[e];
    }
    for (; k < k1; ++k) s += p.part[k * n + i];
  }
  __shared__ float sm[256];
  sm[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x < 64 && i < n) {
    s = (sm[threadIdx.x] + sm[threadIdx.x + 64] + sm[threadIdx.x + 128] + sm[threadIdx.x + 192]) * p.scale;
    OT* o = static_cast<OT*>(p.dweight) + i;
    // Adding nothing leaves the element alone: the rows of tokens that do not occur (an exact zero) are not written.
    if (!p.add) store_io(o, s);
    else if (s != 0.0f) store_io(o, to_f32(*o) + s);
  }
}

void plan_embed_few(int64_t Bsz, int64_t L, int64_t V, int64_t E, EmbedBwdPlan* pl) {
  const int64_t groups = (E + 63) / 64;
  int64_t seg = (Bsz * L * groups / 2048 + 511) / 512 * 512;  // whole tiles; 2048 workgroups or more
  if (seg > kMaxSeg) seg = kMaxSeg;
  if (seg < 512) seg = 512;
  pl->few = true;
  pl->run = seg;
  pl->chunks = Bsz * ((L + seg - 1) / seg);
  pl->total = (size_t)pl->chunks * V * E * 4;
}

// Where the products pay.  The matrix cores keep up with HBM through 64 rows in bf16 and 32 in fp32 (4 and 2 products
// per piece of dout).  A workgroup covers 512 positions of one batch row at least and writes V sums of each of its
// channels, so short batch rows would be mostly idle work and sums: they are turned and sorted instead.  Calls in bf16
// with 4 / 16 / 64 rows by products, and sorted: 8192 x 16 positions, 1024 channels: 1.5 / 1.6 / 3.1 ms and 0.52 (at 64
// rows with 2.1 GB of sums for 0.27 GB of dout); 4096 x 64: 0.82 / 0.84 / 1.6 ms and 0.36; 1024 x 256: 222 / 229 / 386 us
// and 309; 256 x 640: 92 / 96 / 180 and 202; 64 x 512: 20 / 21 / 34 and 58.  Few workgroups and sums cost little,
// whatever they cover: 64 x 64: 16 / 17 / 30 us and 31 / 28 / 27; 64 x 16: 17 / 17 / 31 and 23 / 19 / 16.
bool embed_few_pays(int64_t Bsz, int64_t L, int64_t V, int64_t E, bool io_bf16) {
  if (V > (io_bf16 ? 64 : 32)) return false;
  EmbedBwdPlan pl;
  plan_embed_few(Bsz, L, V, E, &pl);
  if (pl.chunks * ((E + 63) / 64) <= 1024 && pl.total <= (size_t(4) << 20)) return true;
  return L >= 256 && 2 * pl.chunks * V * 4 < Bsz * L * (io_bf16 ? 2 : 4);
}

namespace {

template <typename IO>
hipError_t launch_few(const FewParams& p, bool table_bf16, hipStream_t s) {
  const dim3 grid = grid_of(p.segs * p.groups);
  if (p.V <= 16) hipLaunchKernelGGL((embed_few_kernel<IO, 1>), grid, dim3(256), 0, s, p);
  else if (p.V <= 32) hipLaunchKernelGGL((embed_few_kernel<IO, 2>), grid, dim3(256), 0, s, p);
  else if constexpr (sizeof(IO) == 2) hipLaunchKernelGGL((embed_few_kernel<IO, 4>), grid, dim3(256), 0, s, p);
  const dim3 jgrid = grid_of((p.V * p.E + 63) / 64);
  if (table_bf16) hipLaunchKernelGGL(embed_few_join_kernel<bf16_t>, jgrid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL(embed_few_join_kernel<float>, jgrid, dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed_few(const EmbedParams& e, const EmbedBwdPlan& pl, bool table_bf16, bool io_bf16, void* ws,
                            hipStream_t s) {
  FewParams p{};
  p.tokens = e.tokens; p.dout = e.dout; p.dweight = e.out; p.part = static_cast<float*>(ws);
  p.L = e.L; p.V = e.V; p.E = e.E; p.seg = pl.run; p.segs = pl.chunks; p.segs_row = (e.L + pl.run - 1) / pl.run;
  p.groups = (e.E + 63) / 64;
  p.scale = e.scale; p.i64 = e.i64; p.add = e.add;
  return io_bf16 ? launch_few<bf16_t>(p, table_bf16, s) : launch_few<float>(p, table_bf16, s);
}

}  // namespace ssm
