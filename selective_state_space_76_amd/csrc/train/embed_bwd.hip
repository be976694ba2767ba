// embed_bwd.hip -- gradient of the embedding: dweight[v,:] = scale * sum of dout over the positions whose token is v.
//
// The positions are sorted by token, equal tokens in order of position, and each token's rows are summed in
// that order: no atomics on the sums, so the result is the same bits on every run.
//   1. Sort: a stable radix sort of (token, position), digits of up to 8 bits, the lowest first.  Per digit a
//      counting pass and a moving pass; in the latter every workgroup adds up the counts of the tiles
//      before its own.  A wave ranks 64 keys at a time by ballots over the digit's bits.
//   2. Sums: the sorted list is cut into chunks of `run` rows.  A wave owns a chunk and 64 * VC columns; it
//      keeps 8 rows in flight and adds them to the running token's sum.  Sums of tokens that lie within
//      the chunk go to dweight; one that reaches over an end goes to memory as a partial sum.
//   3. Join: where a token's rows begin in a chunk and go on in the next, its partial sums are added, in order.
//   4. Rows of tokens that do not occur are set to zero (not when the gradient is added to).
// Bound by HBM: dout is read once in whole rows, dweight is written once.
// Tokens outside the table sort as V, behind all others, and are left out.
#include "../ssm_device.h"
#include "embed_device.h"
#include "train_launch.h"

namespace ssm {

namespace {

constexpr int kRounds = 8;  // keys per lane of a sort tile

struct SortParams {
  const void* tokens;     // first pass: the keys are the tokens; else null
  const uint32_t* key_in;
  const uint32_t* pos_in;
  uint32_t* key_out;
  uint32_t* pos_out;
  uint32_t* hist;         // [tiles][digits], or null for a single tile
  int64_t n, V, tiles;
  int i64, shift, bits;
};

__device__ __forceinline__ uint32_t key_at(const SortParams& p, int64_t i) {
  return p.tokens ? (uint32_t)token_at(p.tokens, p.i64, i, p.V) : p.key_in[i];
}

template <int NW>
__global__ __launch_bounds__(NW * 64) void sort_count_kernel(SortParams p) {
  __shared__ uint32_t cnt[256];
  const int digits = 1 << p.bits;
  for (int i = threadIdx.x; i < digits; i += NW * 64) cnt[i] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * (NW * 64 * kRounds);
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * (NW * 64) + threadIdx.x;
    if (i < p.n) atomicAdd(&cnt[(key_at(p, i) >> p.shift) & (digits - 1)], 1u);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < digits; i += NW * 64) p.hist[blockIdx.x * digits + i] = cnt[i];
}

template <int NW>
__global__ __launch_bounds__(NW * 64) void sort_move_kernel(SortParams p) {
  __shared__ uint32_t at[NW][256];  // next place of a digit's keys, per wave
  __shared__ uint32_t tot[256], pre[256];
  const int digits = 1 << p.bits;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < NW * 256; i += NW * 64) (&at[0][0])[i] = 0;
  __syncthreads();
  // a wave's keys: 64 * kRounds consecutive ones
  const int64_t base = ((int64_t)blockIdx.x * NW + wave) * (64 * kRounds);
  uint32_t key[kRounds], pos[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * 64 + lane;
    key[r] = pos[r] = 0;
    if (i < p.n) {
      key[r] = key_at(p, i);
      pos[r] = p.tokens ? (uint32_t)i : p.pos_in[i];
    }
  }
#pragma unroll
  for (int r = 0; r < kRounds; ++r)
    if (base + r * 64 + lane < p.n) atomicAdd(&at[wave][(key[r] >> p.shift) & (digits - 1)], 1u);
  if (tid < digits) {  // a digit's keys in all tiles, and in those before this one
    uint32_t all = 0, mine = 0;
    if (p.hist) {
      int64_t j = 0;
      for (; j + 8 <= p.tiles; j += 8) {
        uint32_t c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = p.hist[(j + e) * digits + tid];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          all += c[e];
          if (j + e < blockIdx.x) mine += c[e];
        }
      }
      for (; j < p.tiles; ++j) {
        const uint32_t c = p.hist[j * digits + tid];
        all += c;
        if (j < blockIdx.x) mine += c;
      }
    }
    tot[tid] = all;
    pre[tid] = mine;
  }
  __syncthreads();
  if (!p.hist && tid < digits) {
    uint32_t all = 0;
    for (int w = 0; w < NW; ++w) all += at[w][tid];
    tot[tid] = all;
  }
  __syncthreads();
  // exclusive sum of the totals over the digits, by one wave (4 digits per lane)
  if (wave == 0) {
    uint32_t v[4], s = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = s;
      if (lane * 4 + e < digits) s += tot[lane * 4 + e];
    }
    uint32_t inc = s;
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t up = __shfl_up(inc, o, 64);
      if (lane >= o) inc += up;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (lane * 4 + e < digits) tot[lane * 4 + e] = inc - s + v[e];
  }
  __syncthreads();
  if (tid < digits) {
    uint32_t a = tot[tid] + pre[tid];
    for (int w = 0; w < NW; ++w) {
      const uint32_t c = at[w][tid];
      at[w][tid] = a;
      a += c;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int r = 0; r < kRounds; ++r) {
    uint32_t k = 0, q = 0;
#pragma unroll
    for (int e = 0; e < kRounds; ++e)
      if (e == r) { k = key[e]; q = pos[e]; }
    const bool valid = base + r * 64 + lane < p.n;
    const uint32_t d = (k >> p.shift) & (digits - 1);
    uint64_t same = __ballot(valid);
    for (int b = 0; b < p.bits; ++b) {
      const uint64_t set = __ballot((d >> b) & 1u);
      same &= (d >> b) & 1u ? set : ~set;
    }
    const uint64_t below = same & ((1ull << lane) - 1);
    uint32_t dst = 0;
    if (valid) dst = at[wave][d] + (uint32_t)__popcll(below);
    wave_sync();  // every lane has read its place before the digit's first lane moves it on
    if (valid && below == 0) at[wave][d] = dst + (uint32_t)__popcll(same);
    wave_sync();
    if (valid) {
      p.key_out[dst] = k;
      p.pos_out[dst] = q;
    }
  }
}

struct SumParams {
  const uint32_t* key;   // sorted
  const uint32_t* pos;
  const void* dout;      // [T,E]
  void* dweight;
  float* part;           // [chunks][2][E]: a sum that comes from the previous chunk, one that goes on in the next
  int64_t n, V, E, run, chunks, col_tiles;
  float scale;
  int add;
};

template <typename OT, int VC>
__device__ __forceinline__ void put_row(const SumParams& p, uint32_t k, int64_t col, int nc, const float (&acc)[VC]) {
  OT* o = static_cast<OT*>(p.dweight) + (int64_t)k * p.E + col;
  float x[VC];
  if (p.add) {
    load_n<OT, VC>(o, nc, x);
#pragma unroll
    for (int e = 0; e < VC; ++e) x[e] += acc[e] * p.scale;
  } else {
#pragma unroll
    for (int e = 0; e < VC; ++e) x[e] = acc[e] * p.scale;
  }
  store_n<OT, VC>(o, nc, x);
}

template <typename IO, typename OT, int VC>
__global__ __launch_bounds__(256) void embed_sum_kernel(SumParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t chunk = unit / p.col_tiles, ct = unit - chunk * p.col_tiles;
  if (chunk >= p.chunks) return;
  const int64_t i0 = chunk * p.run, i1 = i0 + p.run < p.n ? i0 + p.run : p.n;
  const int64_t col = (ct * 64 + lane) * VC;
  const int nc = p.E - col >= VC ? VC : p.E - col > 0 ? (int)(p.E - col) : 0;
  const IO* rows = static_cast<const IO*>(p.dout) + col;
  const uint32_t V = (uint32_t)p.V;
  const uint32_t prev = i0 > 0 ? p.key[i0 - 1] : V, next = i1 < p.n ? p.key[i1] : V;

  float acc[VC];
#pragma unroll
  for (int e = 0; e < VC; ++e) acc[e] = 0.0f;
  uint32_t cur = V;     // token whose rows are being added; V: none yet
  bool head = true;     // its rows began with the chunk
  auto flush = [&](bool at_end) {
    if (cur == V) return;
    if (head && prev == cur) store_n<float, VC>(p.part + (chunk * 2) * p.E + col, nc, acc);
    else if (at_end && next == cur) store_n<float, VC>(p.part + (chunk * 2 + 1) * p.E + col, nc, acc);
    else put_row<OT, VC>(p, cur, col, nc, acc);
  };
  for (int64_t s = i0; s < i1; s += 64) {
    const int m = i1 - s < 64 ? (int)(i1 - s) : 64;
    uint32_t kv = V, pv = 0;
    if (lane < m) {
      kv = p.key[s + lane];
      pv = p.pos[s + lane];
    }
    for (int r = 0; r < m; r += 8) {
      float x[8][VC];
      uint32_t k[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        k[q] = r + q < m ? (uint32_t)__builtin_amdgcn_readlane((int)kv, r + q) : V;
        const uint32_t t = (uint32_t)__builtin_amdgcn_readlane((int)pv, r + q < m ? r + q : 0);
        if (k[q] != V) load_n<IO, VC, true>(rows + (int64_t)t * p.E, nc, x[q]);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (k[q] == V) continue;  // past the chunk, or outside the table: all that follow are, too
        if (k[q] != cur) {
          flush(false);
          head = s + r + q == i0;
          cur = k[q];
#pragma unroll
          for (int e = 0; e < VC; ++e) acc[e] = x[q][e];
        } else {
#pragma unroll
          for (int e = 0; e < VC; ++e) acc[e] += x[q][e];
        }
      }
    }
  }
  flush(true);
}

// A workgroup per chunk and column tile: where a token begins in the chunk and goes on, the sums of the chunks
// that follow are added by 4 waves, a run of chunks each, and these in order.
template <typename OT, int VC>
__global__ __launch_bounds__(256) void embed_join_kernel(SumParams p) {
  const int64_t chunk = blockIdx.x / p.col_tiles, ct = blockIdx.x - chunk * p.col_tiles;
  const int64_t i0 = chunk * p.run, i1 = i0 + p.run;
  if (i1 >= p.n) return;
  const uint32_t k = p.key[i1 - 1];
  if (k == (uint32_t)p.V || p.key[i1] != k) return;
  if (i0 > 0 && p.key[i0] == k && p.key[i0 - 1] == k) return;  // it begins in an earlier chunk
  int64_t lo = i1 + 1, hi = p.n;  // the first place behind the token's rows
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (p.key[mid] <= k) lo = mid + 1;
    else hi = mid;
  }
  const int64_t last = (lo - 1) / p.run;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (ct * 64 + lane) * VC;
  const int nc = p.E - col >= VC ? VC : p.E - col > 0 ? (int)(p.E - col) : 0;
  const int64_t per = (last - chunk + 3) / 4;
  int64_t c = chunk + 1 + wave * per;
  const int64_t c1 = c + per < last + 1 ? c + per : last + 1;
  float acc[VC];
#pragma unroll
  for (int e = 0; e < VC; ++e) acc[e] = 0.0f;
  if (wave == 0) load_n<float, VC>(p.part + (chunk * 2 + 1) * p.E + col, nc, acc);
  for (; c + 8 <= c1; c += 8) {
    float x[8][VC];
#pragma unroll
    for (int q = 0; q < 8; ++q) load_n<float, VC>(p.part + (c + q) * 2 * p.E + col, nc, x[q]);
#pragma unroll
    for (int q = 0; q < 8; ++q)
#pragma unroll
      for (int e = 0; e < VC; ++e) acc[e] += x[q][e];
  }
  for (; c < c1; ++c) {
    float x[VC];
    load_n<float, VC>(p.part + c * 2 * p.E + col, nc, x);
#pragma unroll
    for (int e = 0; e < VC; ++e) acc[e] += x[e];
  }
  __shared__ float sm[4][VC][64];
#pragma unroll
  for (int e = 0; e < VC; ++e) sm[wave][e][lane] = acc[e];
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int e = 0; e < VC; ++e) acc[e] += sm[1][e][lane] + (sm[2][e][lane] + sm[3][e][lane]);
    put_row<OT, VC>(p, k, col, nc, acc);
  }
}

// A wave looks 16 rows of the table up in the sorted tokens and clears those that are not there.
template <typename OT>
__global__ __launch_bounds__(256) void embed_zero_kernel(SumParams p) {
  constexpr int VO = 16 / (int)sizeof(OT);
  const int lane = threadIdx.x & 63;
  const int64_t v0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * 16;
  const int64_t v = v0 + (lane & 15);
  bool absent = false;
  if (lane < 16 && v < p.V) {
    int64_t lo = 0, hi = p.n;
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (p.key[mid] < (uint32_t)v) lo = mid + 1;
      else hi = mid;
    }
    absent = lo == p.n || p.key[lo] != (uint32_t)v;
  }
  uint64_t todo = __ballot(absent);
  float zero[VO];
#pragma unroll
  for (int e = 0; e < VO; ++e) zero[e] = 0.0f;
  while (todo) {
    const int b = __builtin_ctzll(todo);
    todo &= todo - 1;
    OT* o = static_cast<OT*>(p.dweight) + (v0 + b) * p.E;
    for (int64_t c = lane * VO; c < p.E; c += 64 * VO)
      store_n<OT, VO>(o + c, p.E - c >= VO ? VO : (int)(p.E - c), zero);
  }
}

// [B,E,L] to [B,L,E]: a tile of 64 columns x 128 positions through LDS, in pairs of neighbouring columns
template <typename IO>
__global__ __launch_bounds__(256) void embed_turn_kernel(const IO* in, IO* out, int64_t E, int64_t L) {
  constexpr int V = 16 / (int)sizeof(IO);
  constexpr int TT = 128, TE = 64;
  constexpr int LD = TE + V;  // elements between positions in LDS
  __shared__ __align__(16) IO sm[TT * LD];
  const int64_t tiles_t = (L + TT - 1) / TT, tiles_e = (E + TE - 1) / TE;
  const int64_t blk = blockIdx.x;
  const int64_t te = blk % tiles_e, rest = blk / tiles_e;
  const int64_t tt = rest % tiles_t, b = rest / tiles_t;
  const int64_t t0 = tt * TT, e0 = te * TE;
  const int64_t nt = L - t0, ne = E - e0;
  constexpr int PPR = TT / 8;  // 8 positions per lane
#pragma unroll
  for (int h = 0; h < (TE / 2) * PPR / 256; ++h) {
    const int i = h * 256 + threadIdx.x;
    const int r = (i % PPR) * 8, c = (i / PPR) * 2;
    const int n = nt - r >= 8 ? 8 : nt - r > 0 ? (int)(nt - r) : 0;
    float x[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) load_n<IO, 8, true>(in + (b * E + e0 + c + k) * L + t0 + r, c + k < ne ? n : 0, x[k]);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if constexpr (sizeof(IO) == 2)
        *reinterpret_cast<uint32_t*>(&sm[(r + q) * LD + c]) =
            (__float_as_uint(x[0][q]) >> 16) | (__float_as_uint(x[1][q]) & 0xffff0000u);
      else
        *reinterpret_cast<float2*>(&sm[(r + q) * LD + c]) = make_float2(x[0][q], x[1][q]);
    }
  }
  __syncthreads();
  constexpr int PPC = TE / V;
#pragma unroll
  for (int h = 0; h < TT * PPC / 256; ++h) {
    const int i = h * 256 + threadIdx.x;
    const int r = i / PPC, c = (i % PPC) * V;
    if (r >= nt || c >= ne) continue;
    const int n = ne - c < V ? (int)(ne - c) : V;
    IO* o = out + (b * L + t0 + r) * E + e0 + c;
    const u32x4a q = *reinterpret_cast<const u32x4a*>(&sm[r * LD + c]);
    if (n == V) *reinterpret_cast<typename Unaligned<IO>::type*>(o) = (typename Unaligned<IO>::type)q;
    else
      for (int k = 0; k < n; ++k) o[k] = sm[r * LD + c + k];
  }
}

template <typename IO, typename OT, int VC>
hipError_t launch_sums(SumParams p, hipStream_t s) {
  p.col_tiles = (p.E + 64 * VC - 1) / (64 * VC);
  const int64_t units = p.chunks * p.col_tiles;
  hipLaunchKernelGGL((embed_sum_kernel<IO, OT, VC>), dim3((unsigned)((units + 3) / 4)), dim3(256), 0, s, p);
  if (p.chunks > 1) hipLaunchKernelGGL((embed_join_kernel<OT, VC>), dim3((unsigned)units), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename IO, typename OT>
hipError_t launch_io(const EmbedParams& e, const EmbedBwdPlan& pl, SumParams p, char* ws, hipStream_t s) {
  if (pl.transpose) {
    const int64_t blocks = e.Bsz * ((e.L + 127) / 128) * ((e.E + 63) / 64);
    IO* rows = reinterpret_cast<IO*>(ws + pl.rows);
    hipLaunchKernelGGL((embed_turn_kernel<IO>), dim3((unsigned)blocks), dim3(256), 0, s,
                       static_cast<const IO*>(e.dout), rows, e.E, e.L);
    p.dout = rows;
  }
  if (!e.add)
    hipLaunchKernelGGL((embed_zero_kernel<OT>), dim3((unsigned)((e.V + 63) / 64)), dim3(256), 0, s, p);
  // 8 columns per lane where that covers the row with no more idle lanes than 4
  if (sizeof(IO) == 2 && (e.E + 511) / 512 * 2 == (e.E + 255) / 256) return launch_sums<IO, OT, 8>(p, s);
  return launch_sums<IO, OT, 4>(p, s);
}

template <int NW>
hipError_t launch_sort(SortParams sp, hipStream_t s) {
  if (sp.tiles > 1)
    hipLaunchKernelGGL((sort_count_kernel<NW>), dim3((unsigned)sp.tiles), dim3(NW * 64), 0, s, sp);
  else
    sp.hist = nullptr;
  hipLaunchKernelGGL((sort_move_kernel<NW>), dim3((unsigned)sp.tiles), dim3(NW * 64), 0, s, sp);
  return hipGetLastError();
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

void plan_embed_bwd(int64_t Bsz, int64_t L, int64_t V, int64_t E, bool io_bf16, bool cf, EmbedBwdPlan* pl) {
  const int64_t n = Bsz * L;
  pl->bits = 1;
  while ((V >> pl->bits) != 0) ++pl->bits;  // keys 0 .. V
  pl->passes = (pl->bits + 7) / 8;
  pl->digit_bits = (pl->bits + pl->passes - 1) / pl->passes;
  pl->tile = n <= 8192 || n > 262144 ? 16 * 64 * kRounds : 4 * 64 * kRounds;
  pl->tiles = (n + pl->tile - 1) / pl->tile;
  pl->run = n <= 65536 ? 32 : n <= 524288 ? 64 : 256;
  pl->chunks = (n + pl->run - 1) / pl->run;
  pl->transpose = cf && L > 1;
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t o = off; off += round256(bytes); return o; };
  if (pl->transpose) pl->rows = take((size_t)n * E * (io_bf16 ? 2 : 4));
  for (int i = 0; i < 2; ++i) {
    pl->key[i] = take((size_t)n * 4);
    pl->pos[i] = take((size_t)n * 4);
  }
  pl->hist[0] = take((size_t)pl->tiles * 4 << pl->digit_bits);
  pl->part = take((size_t)pl->chunks * 2 * E * 4);
  pl->total = off;
}

hipError_t launch_embed_bwd(const EmbedParams& e, const EmbedBwdPlan& pl, bool table_bf16, bool io_bf16, void* ws,
                            hipStream_t s) {
  char* w = static_cast<char*>(ws);
  SortParams sp{};
  sp.tokens = e.tokens;
  sp.hist = reinterpret_cast<uint32_t*>(w + pl.hist[0]);
  sp.n = e.T; sp.V = e.V; sp.tiles = pl.tiles; sp.i64 = e.i64; sp.bits = pl.digit_bits;
  int to = 0;
  for (int k = 0; k < pl.passes; ++k) {
    sp.key_out = reinterpret_cast<uint32_t*>(w + pl.key[to]);
    sp.pos_out = reinterpret_cast<uint32_t*>(w + pl.pos[to]);
    sp.shift = k * pl.digit_bits;
    const hipError_t rc = pl.tile == 4 * 64 * kRounds ? launch_sort<4>(sp, s) : launch_sort<16>(sp, s);
    if (rc != hipSuccess) return rc;
    sp.tokens = nullptr;
    sp.key_in = sp.key_out;
    sp.pos_in = sp.pos_out;
    to ^= 1;
  }
  SumParams p{};
  p.key = sp.key_out; p.pos = sp.pos_out; p.dout = e.dout; p.dweight = e.out;
  p.part = reinterpret_cast<float*>(w + pl.part);
  p.n = e.T; p.V = e.V; p.E = e.E; p.run = pl.run; p.chunks = pl.chunks;
  p.scale = e.scale; p.add = e.add;
  if (io_bf16)
    return table_bf16 ? launch_io<bf16_t, bf16_t>(e, pl, p, w, s) : launch_io<bf16_t, float>(e, pl, p, w, s);
  return table_bf16 ? launch_io<float, bf16_t>(e, pl, p, w, s) : launch_io<float, float>(e, pl, p, w, s);
}

}  // namespace ssm
