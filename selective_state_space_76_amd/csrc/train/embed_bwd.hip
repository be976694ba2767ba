// embed_bwd.hip -- gradient of the embedding: dweight[v,:] = scale * sum of dout over the positions whose token is v.
//
// The positions are sorted by token, equal tokens in order of position, and each token's rows are summed in
// that order: no atomics on the sums, so the result is the same bits on every run.
//   1. Sort: a stable radix sort of (token, position), digits of up to 8 bits, the lowest first.  Up to 4096
//      positions are sorted by one workgroup in LDS (whole calls of width 4: 22 us, where the launches below
//      take 25; 8192 would take 30 against 26); more of them take, per digit, a counting pass and a moving pass,
//      in which every workgroup adds up the counts of the tiles before its own.  A wave ranks 64 keys at a
//      time by ballots over the digit's bits, without a wait between them (4096: 26 -> 22 us per call).  The
//      sort is short and narrow: the other workgroups of its launches clear dweight meanwhile (not when the
//      gradient is added to).
//   2. Sums: the sorted list is cut into chunks of `run` rows.  A wave owns a chunk and 64 * VC columns; it
//      keeps 8 rows in flight and adds them to the running token's sum.  Sums of tokens that lie within
//      the chunk go to dweight; one that reaches over an end goes to memory as a partial sum.
//   3. Join: where a token's rows begin in a chunk and go on in the next, its partial sums are added, in order.
// Up to 2048 positions take all three in one launch where there is little to clear (embed_once_kernel).
// dout in [B,E,L] is first brought to [B,L,E], unless the table has few rows and the batch rows are not too short for
// products (embed_bwd_few.hip).
// Tokens outside the table sort as V, behind all others, and are left out.
//
// Bound by HBM, which the launches reach in part: 8 x 2048 tokens of width 768 into 50000 rows (25 MB read, 154 MB
// cleared or written) take 47 us, of which 30 are the sort's four launches with the clearing (5.1 TB/s), 11 the sums
// and 6 the join.  262144 x 1024 in bf16: 148 us (sort 33, sums 105 at 5.1 TB/s, join 10).
#include "../ssm_device.h"
#include "train_device.h"
#include "train_launch.h"

namespace ssm {

namespace {

struct SortParams {
  const void* tokens;     // first pass: the keys are the tokens; else null
  const uint32_t* key_in;
  const uint32_t* pos_in;
  uint32_t* key_out;
  uint32_t* pos_out;
  uint32_t* hist;         // [tiles][digits]
  char* fill;             // bytes to clear meanwhile (the sort leaves most of the chip idle)
  int64_t fill_bytes, fill_blocks;
  int64_t n, V, tiles;
  int i64, shift, bits, passes;
};

__device__ __forceinline__ uint32_t key_at(const SortParams& p, int64_t i) {
  return p.tokens ? (uint32_t)token_at(p.tokens, p.i64, i, p.V) : p.key_in[i];
}

constexpr int64_t kFill = 16384;                       // bytes per workgroup,
constexpr int64_t kFillBlocks = int64_t(1) << 20;  // up to 16 GiB; then again that far on

// clears piece `block` of the bytes to fill
__device__ __forceinline__ void fill_piece(const SortParams& p, int64_t block, int threads) {
  for (int64_t lo = block * kFill; lo < p.fill_bytes; lo += p.fill_blocks * kFill) {
    const int64_t hi = lo + kFill < p.fill_bytes ? lo + kFill : p.fill_bytes;
    int64_t i = lo + threadIdx.x * 16;
    for (; i + 16 <= hi; i += threads * 16)
      __builtin_nontemporal_store(u32x4a{0u, 0u, 0u, 0u}, reinterpret_cast<u32x4a*>(p.fill + i));
    if (i < hi)  // the last elements, fewer than 16 bytes
      for (; i < hi; i += 2) *reinterpret_cast<uint16_t*>(p.fill + i) = 0;
  }
}

// Exclusive sum over up to 256 digits, by one wave: 4 per lane.
__device__ __forceinline__ void scan_digits(uint32_t* tot, int digits, int lane) {
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

// Where the wave's keys go: count[] (zero before, in LDS) gets the wave's number of each digit, rank[r] the number
// of keys with the same digit before key r of this lane, in rounds of 64 keys.  A round's lanes find their equals
// by ballots over the digit's 8 bits, read the count, and the first of them moves it on.  The LDS serves a wave in
// order, so that nothing waits between the rounds.
template <int R>
__device__ __forceinline__ void rank_keys(uint32_t* count, const uint32_t (&key)[R], int shift, uint32_t mask,
                                          int64_t base, int64_t n, int rounds, uint32_t (&rank)[R]) {
  uint32_t below[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    rank[r] = below[r] = 0;
    if (r >= rounds) continue;
    const bool valid = base + r * 64 < n;
    const uint32_t d = (key[r] >> shift) & mask;
    const uint64_t in = __ballot(valid);
    uint32_t lo = (uint32_t)in, hi = (uint32_t)(in >> 32);  // lanes with the same digit
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const int32_t bit = (int32_t)(d << (31 - b)) >> 31;
      const uint64_t set = __ballot(bit < 0);
      lo &= ~((uint32_t)set ^ (uint32_t)bit);
      hi &= ~((uint32_t)(set >> 32) ^ (uint32_t)bit);
    }
    below[r] = __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0u));
    rank[r] = __hip_atomic_load(&count[d], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    __builtin_amdgcn_wave_barrier();
    if (valid && below[r] == 0)
      __hip_atomic_fetch_add(&count[d], (uint32_t)(__popc(lo) + __popc(hi)), __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_WORKGROUP);
    __builtin_amdgcn_wave_barrier();
  }
#pragma unroll
  for (int r = 0; r < R; ++r) rank[r] += below[r];
}

// Up to 1024 R keys sorted by one workgroup of 1024, all digits: the tokens, or (LISTED) what is in sm.key and sm.pos.
// Keys and positions move through LDS and stay there.
template <int R>
struct SortLds {
  uint32_t at[16][256];  // a wave's keys of a digit; then where they go
  uint32_t tot[256];
  uint32_t key[1024 * R];
  uint16_t pos[1024 * R];
};

template <int R, bool LISTED>
__device__ __forceinline__ void sort_lds(const SortParams& p, int n, SortLds<R>& sm) {
  const int digits = 1 << p.bits;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int rounds = (n + 1023) / 1024;
  const int base = wave * (64 * rounds) + lane;
  uint32_t key[R], pos[R], rank[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    pos[r] = base + r * 64;
    key[r] = !LISTED && r < rounds && (int)pos[r] < n ? key_at(p, pos[r]) : 0u;
  }
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    for (int i = tid; i < 16 * 256; i += 1024) (&sm.at[0][0])[i] = 0;
    __syncthreads();
    if (LISTED || pass > 0) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r < rounds && base + r * 64 < n) {
          pos[r] = sm.pos[base + r * 64];
          key[r] = sm.key[base + r * 64];
        }
    }
    rank_keys<R>(sm.at[wave], key, shift, (uint32_t)digits - 1, base, n, rounds, rank);
    __syncthreads();
    uint32_t c[16];
    if (tid < digits) {
      uint32_t all = 0;
#pragma unroll
      for (int w = 0; w < 16; ++w) {
        c[w] = all;
        all += sm.at[w][tid];
      }
      sm.tot[tid] = all;
    }
    __syncthreads();
    if (wave == 0) scan_digits(sm.tot, digits, lane);
    __syncthreads();
    if (tid < digits) {
      const uint32_t a = sm.tot[tid];
#pragma unroll
      for (int w = 0; w < 16; ++w) sm.at[w][tid] = a + c[w];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= rounds || base + r * 64 >= n) continue;
      const uint32_t dst = sm.at[wave][(key[r] >> shift) & (digits - 1)] + rank[r];
      sm.key[dst] = key[r];
      sm.pos[dst] = (uint16_t)pos[r];
    }
    __syncthreads();
  }
}

// The sort in a launch of its own.  The lists leave in order: stores by rank would cost a line each (4096: 24 -> 22 us
// per call).  The other workgroups fill.
template <int R>
__global__ __launch_bounds__(1024) void sort_small_kernel(SortParams p) {
  if (blockIdx.x > 0) return fill_piece(p, blockIdx.x - 1, 1024);
  __shared__ SortLds<R> sm;
  sort_lds<R, false>(p, (int)p.n, sm);
  for (int i = threadIdx.x; i < (int)p.n; i += 1024) {
    p.key_out[i] = sm.key[i];
    p.pos_out[i] = sm.pos[i];
  }
}

template <int NW, int R>
__global__ __launch_bounds__(NW * 64) void sort_count_kernel(SortParams p) {
  if (blockIdx.x >= p.tiles) return fill_piece(p, blockIdx.x - p.tiles, NW * 64);
  __shared__ uint32_t cnt[256];
  const int digits = 1 << p.bits;
  for (int i = threadIdx.x; i < digits; i += NW * 64) cnt[i] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * (NW * 64 * R);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t i = base + r * (NW * 64) + threadIdx.x;
    if (i < p.n) atomicAdd(&cnt[(key_at(p, i) >> p.shift) & (digits - 1)], 1u);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < digits; i += NW * 64) p.hist[blockIdx.x * digits + i] = cnt[i];
}

template <int NW, int R>
__global__ __launch_bounds__(NW * 64) void sort_move_kernel(SortParams p) {
  if (blockIdx.x >= p.tiles) return fill_piece(p, blockIdx.x - p.tiles, NW * 64);
  __shared__ uint32_t at[NW][256];  // next place of a digit's keys, per wave
  __shared__ uint32_t tot[256];
  const int digits = 1 << p.bits;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < NW * 256; i += NW * 64) (&at[0][0])[i] = 0;
  __syncthreads();
  // a wave's keys: 64 R consecutive ones
  const int64_t base = ((int64_t)blockIdx.x * NW + wave) * (64 * R) + lane;
  uint32_t key[R], pos[R], rank[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t i = base + r * 64;
    key[r] = pos[r] = 0;
    if (i < p.n) {
      key[r] = key_at(p, i);
      pos[r] = p.tokens ? (uint32_t)i : p.pos_in[i];
    }
  }
  uint32_t mine = 0;  // a digit's keys in the tiles before this one
  if (tid < digits) {
    uint32_t all = 0;
    int64_t j = 0;
    for (; j + 16 <= p.tiles; j += 16) {
      uint32_t c[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) c[e] = p.hist[(j + e) * digits + tid];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        all += c[e];
        if (j + e < blockIdx.x) mine += c[e];
      }
    }
    for (; j < p.tiles; ++j) {
      const uint32_t c = p.hist[j * digits + tid];
      all += c;
      if (j < blockIdx.x) mine += c;
    }
    tot[tid] = all;
  }
  rank_keys<R>(at[wave], key, p.shift, (uint32_t)digits - 1, base, p.n, R, rank);
  __syncthreads();
  if (wave == 0) scan_digits(tot, digits, lane);
  __syncthreads();
  if (tid < digits) {
    uint32_t a = tot[tid] + mine;
    for (int w = 0; w < NW; ++w) {
      const uint32_t c = at[w][tid];
      at[w][tid] = a;
      a += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (base + r * 64 >= p.n) continue;
    const uint32_t dst = at[wave][(key[r] >> p.shift) & (digits - 1)] + rank[r];
    p.key_out[dst] = key[r];
    p.pos_out[dst] = pos[r];
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
__device__ __forceinline__ OT* row_at(const SumParams& p, uint32_t k, int64_t col) {
  return static_cast<OT*>(p.dweight) + (int64_t)k * p.E + col;
}

// The sums of rows i0 .. i1 - 1 of the sorted list; prev and next: the keys beside them (V: none).  Sums of tokens
// within go to dweight, others to partial(0, ..) where the token's rows began before i0, partial(1, ..) where they
// go on at i1.
// With ADD the rows of dweight that a group of 8 will add to are loaded with the group, not one by one as the
// tokens change: one wait for memory per group and not per token (509 tokens of width 768 into a table of 50000
// rows: 18 -> 7 us, with chunks of 8 rows and not 32).
// NT: dout is too large to be found in the Infinity Cache (256 MB), where a backward pass has just left it, and
// is read as not needed again (16384 x 768: 53 -> 49 us per call without; 262144 x 1024: 165 -> 153 us with).
template <typename IO, typename OT, int VC, bool ADD, bool NT, typename Key, typename Pos, typename Partial>
__device__ __forceinline__ void sum_rows(const SumParams& p, int64_t i0, int64_t i1, uint32_t prev, uint32_t next,
                                         int64_t col, int nc, int lane, Key key, Pos pos, Partial partial) {
  const IO* rows = static_cast<const IO*>(p.dout) + col;
  const uint32_t V = (uint32_t)p.V;
  float acc[VC];
#pragma unroll
  for (int e = 0; e < VC; ++e) acc[e] = 0.0f;
  uint32_t cur = V;     // token whose rows are being added; V: none yet
  bool head = true;     // its rows began with the chunk
  for (int64_t s = i0; s < i1; s += 64) {
    const int m = i1 - s < 64 ? (int)(i1 - s) : 64;
    uint32_t kv = V, pv = 0;
    if (lane < m) {
      kv = key(s + lane);
      pv = pos(s + lane);
    }
    const uint32_t after = s + 64 < i1 ? key(s + 64) : next;  // the key behind these
    for (int r = 0; r < m; r += 8) {
      Raw<IO, VC, NT> x[8];
      Raw<OT, VC> old[ADD ? 8 : 1];
      uint32_t k[9];
#pragma unroll
      for (int q = 0; q < 9; ++q)
        k[q] = r + q < m    ? (uint32_t)__builtin_amdgcn_readlane((int)kv, r + q < 64 ? r + q : 63)
               : r + q == m ? after
                            : V;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (r + q >= m || k[q] == V) continue;  // past the chunk, or outside the table as all that follow
        const uint32_t t = (uint32_t)__builtin_amdgcn_readlane((int)pv, r + q);
        x[q].load(rows + (int64_t)t * p.E, nc);
        if constexpr (ADD)
          if (k[q] != k[q + 1]) old[q].load(row_at<OT, VC>(p, k[q], col), nc);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (r + q >= m || k[q] == V) continue;
        if (k[q] != cur) {
          head = s + r + q == i0;
          cur = k[q];
#pragma unroll
          for (int e = 0; e < VC; ++e) acc[e] = x[q].at(e);
        } else {
#pragma unroll
          for (int e = 0; e < VC; ++e) acc[e] += x[q].at(e);
        }
        const bool end = s + r + q + 1 == i1;
        if (!end && k[q] == k[q + 1]) continue;
        if (head && prev == cur) {
          partial(0, acc);
        } else if (end && next == cur) {
          partial(1, acc);
        } else {
          float y[VC];
#pragma unroll
          for (int e = 0; e < VC; ++e) y[e] = ADD ? old[ADD ? q : 0].at(e) + acc[e] * p.scale : acc[e] * p.scale;
          store_n<OT, VC>(row_at<OT, VC>(p, cur, col), nc, y);
        }
      }
    }
  }
}

template <typename IO, typename OT, int VC, bool ADD, bool NT>
__global__ __launch_bounds__(256) void embed_sum_kernel(SumParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t chunk = unit / p.col_tiles, ct = unit - chunk * p.col_tiles;
  if (chunk >= p.chunks) return;
  const int64_t i0 = chunk * p.run, i1 = i0 + p.run < p.n ? i0 + p.run : p.n;
  const int64_t col = (ct * 64 + lane) * VC;
  const int nc = p.E - col >= VC ? VC : p.E - col > 0 ? (int)(p.E - col) : 0;
  const uint32_t prev = i0 > 0 ? p.key[i0 - 1] : (uint32_t)p.V, next = i1 < p.n ? p.key[i1] : (uint32_t)p.V;
  sum_rows<IO, OT, VC, ADD, NT>(
      p, i0, i1, prev, next, col, nc, lane, [&](int64_t i) { return p.key[i]; }, [&](int64_t i) { return p.pos[i]; },
      [&](int which, const float(&acc)[VC]) { store_n<float, VC>(p.part + (chunk * 2 + which) * p.E + col, nc, acc); });
}

// All steps in one launch, for up to 1024 R positions: a workgroup takes the tokens v with v % groups == its own number
// and a tile of 64 * VC columns.  It lists their positions in order, sorts the list, short as a rule, by
// counting for each entry those that come before it, and by radix where it is long.  Its 16 waves share the list's
// rows, and sums that reach over a wave's end meet in LDS.  Without ADD it also clears its rows that no token names.
// (509 x 768, added: 8.9 us per call; 10.7 where every workgroup sorted all positions for itself, 13.8 with a launch
// for each step.)
constexpr int kPairs = 128;  // longest list sorted by counting

template <typename IO, typename OT, int VC, int R, bool ADD>
__global__ __launch_bounds__(1024) void embed_once_kernel(SortParams sp, SumParams p) {
  __shared__ SortLds<R> sm;
  __shared__ float part[16][2][VC][64];
  __shared__ uint32_t listed[16];
  const uint32_t groups = (uint32_t)p.chunks, group = blockIdx.x / (uint32_t)p.col_tiles;
  const int64_t ct = blockIdx.x - group * (uint32_t)p.col_tiles;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t col = (ct * 64 + lane) * VC;
  const int nc = p.E - col >= VC ? VC : p.E - col > 0 ? (int)(p.E - col) : 0;
  const uint32_t V = (uint32_t)p.V;
  const int base = wave * (64 * R) + lane;
  uint32_t mine[R];
  uint64_t ins[R];
  uint32_t count = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) mine[r] = base + r * 64 < (int)p.n ? key_at(sp, base + r * 64) : V;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    ins[r] = __ballot(mine[r] != V && mine[r] % groups == group);
    count += (uint32_t)__popcll(ins[r]);
  }
  if (lane == 0) listed[wave] = count;
  __syncthreads();
  int z = 0, at = 0;  // entries of the list, and of the waves before this one
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    if (w == wave) at = z;
    z += (int)listed[w];
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int to = at + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(ins[r] >> 32),
                                                       __builtin_amdgcn_mbcnt_lo((uint32_t)ins[r], 0u));
    if (ins[r] >> lane & 1) {
      sm.key[to] = mine[r];
      sm.pos[to] = (uint16_t)(base + r * 64);
    }
    at += (int)__popcll(ins[r]);
  }
  __syncthreads();
  if (z <= kPairs) {
    uint32_t key = 0, pos = 0;
    int rank = 0;
    if (tid < z) {
      key = sm.key[tid];
      pos = sm.pos[tid];
#pragma unroll 8
      for (int j = 0; j < z; ++j) {
        const uint32_t other = sm.key[j];
        rank += other < key || (other == key && j < tid);
      }
    }
    __syncthreads();
    if (tid < z) {
      sm.key[rank] = key;
      sm.pos[rank] = (uint16_t)pos;
    }
    __syncthreads();
  } else {
    sort_lds<R, true>(sp, z, sm);
  }
  const int per = (z + 15) / 16;
  const int i0 = wave * per < z ? wave * per : z, i1 = i0 + per < z ? i0 + per : z;
  const uint32_t prev = i0 > 0 ? sm.key[i0 - 1] : V, next = i1 < z ? sm.key[i1] : V;
  sum_rows<IO, OT, VC, ADD, false>(
      p, i0, i1, prev, next, col, nc, lane, [&](int64_t i) { return sm.key[i]; },
      [&](int64_t i) { return (uint32_t)sm.pos[i]; },
      [&](int which, const float(&acc)[VC]) {
#pragma unroll
        for (int e = 0; e < VC; ++e) part[wave][which][e][lane] = acc[e];
      });
  __syncthreads();
  if (i0 < i1) {
    const uint32_t k = sm.key[i1 - 1];
    if (next == k && !(sm.key[i0] == k && prev == k)) {  // begins here and goes on
      float acc[VC], old[VC];
#pragma unroll
      for (int e = 0; e < VC; ++e) acc[e] = part[wave][1][e][lane];
      if (ADD) load_n<OT, VC>(row_at<OT, VC>(p, k, col), nc, old);
      for (int w = wave + 1, j = i1; j < z && sm.key[j] == k; ++w, j += per)
#pragma unroll
        for (int e = 0; e < VC; ++e) acc[e] += part[w][0][e][lane];
#pragma unroll
      for (int e = 0; e < VC; ++e) acc[e] = ADD ? old[e] + acc[e] * p.scale : acc[e] * p.scale;
      store_n<OT, VC>(row_at<OT, VC>(p, k, col), nc, acc);
    }
  }
  if (ADD) return;
  // the group's rows are v = group + groups * r; a wave clears those of r0 <= r < r1
  const int64_t rows = group < V ? (p.V - group + groups - 1) / groups : 0, share = (rows + 15) / 16;
  const int64_t r0 = wave * share, r1 = r0 + share < rows ? r0 + share : rows;
  float zero[VC];
#pragma unroll
  for (int e = 0; e < VC; ++e) zero[e] = 0.0f;
  auto first_from = [&](uint32_t v) {  // the list's first entry that is not before row v
    int lo = 0, hi = z;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (sm.key[mid] < v) lo = mid + 1;
      else hi = mid;
    }
    return lo;
  };
  int i = r0 < r1 ? first_from(group + groups * (uint32_t)r0) : z;
  uint32_t named = i < z ? sm.key[i] : V;  // the next row that is not to be cleared
  for (int64_t r = r0; r < r1; ++r) {
    const uint32_t v = group + groups * (uint32_t)r;
    if (v == named) {
      i = first_from(v + 1);
      named = i < z ? sm.key[i] : V;
    } else {
      store_n<OT, VC>(row_at<OT, VC>(p, v, col), nc, zero);
    }
  }
}

// A workgroup per chunk and column tile: where a token begins in the chunk and goes on, the sums of the chunks
// that follow are added by 4 waves, a run of chunks each, and these in order.
template <typename OT, int VC>
__global__ __launch_bounds__(256) void embed_join_kernel(SumParams p) {
  const int64_t chunk = blockIdx.x / p.col_tiles, ct = blockIdx.x - chunk * p.col_tiles;
  const int64_t i0 = chunk * p.run, i1 = i0 + p.run;
  if (i1 >= p.n) return;
  const uint32_t k = p.key[i1 - 1], first = p.key[i0], before = i0 > 0 ? p.key[i0 - 1] : (uint32_t)p.V;
  if (k == (uint32_t)p.V || p.key[i1] != k) return;
  if (first == k && before == k) return;  // it begins in an earlier chunk
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t last = chunk + 1;  // the chunk that the token's rows end in: the next one begins with another
  for (;;) {
    const int64_t i = (last + 1 + lane) * p.run;
    const uint64_t goes_on = __ballot(i < p.n && p.key[i < p.n ? i : 0] == k);
    if (~goes_on) {
      last += __builtin_ctzll(~goes_on);
      break;
    }
    last += 64;
  }
  const int64_t col = (ct * 64 + lane) * VC;
  const int nc = p.E - col >= VC ? VC : p.E - col > 0 ? (int)(p.E - col) : 0;
  const int64_t per = (last - chunk + 3) / 4;
  int64_t c = chunk + 1 + wave * per;
  const int64_t c1 = c + per < last + 1 ? c + per : last + 1;
  float acc[VC], old[VC];
#pragma unroll
  for (int e = 0; e < VC; ++e) acc[e] = old[e] = 0.0f;
  if (wave == 0) {
    load_n<float, VC>(p.part + (chunk * 2 + 1) * p.E + col, nc, acc);
    if (p.add) load_n<OT, VC>(row_at<OT, VC>(p, k, col), nc, old);
  }
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
    for (int e = 0; e < VC; ++e) {
      acc[e] = (acc[e] + (sm[1][e][lane] + (sm[2][e][lane] + sm[3][e][lane]))) * p.scale;
      if (p.add) acc[e] += old[e];
    }
    store_n<OT, VC>(row_at<OT, VC>(p, k, col), nc, acc);
  }
}

// [B,E,L] to [B,L,E]: a tile of 64 columns x 128 positions through LDS, in pairs of neighbouring columns
template <typename IO>
__global__ __launch_bounds__(256) void embed_turn_kernel(const IO* in, IO* out, int64_t Bsz, int64_t E, int64_t L) {
  constexpr int V = 16 / (int)sizeof(IO);
  constexpr int TT = 128, TE = 64;
  constexpr int LD = TE + V;  // elements between positions in LDS
  __shared__ __align__(16) IO sm[TT * LD];
  const int64_t tiles_t = (L + TT - 1) / TT, tiles_e = (E + TE - 1) / TE;
  const int64_t blk = block_id();
  const int64_t te = blk % tiles_e, rest = blk / tiles_e;
  const int64_t tt = rest % tiles_t, b = rest / tiles_t;
  if (b >= Bsz) return;
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

// Columns per lane of the sums: 8 (16 bytes) where that covers a row with no more idle lanes than 4
// (262144 x 1024: 153 us with 8, 159 with 4; 262144 x 1000: 189 and 247).
int columns(int64_t E, bool io_bf16) { return io_bf16 && (E + 511) / 512 * 2 == (E + 255) / 256 ? 8 : 4; }

template <typename IO, typename OT, int VC>
hipError_t launch_sums(SumParams p, hipStream_t s) {
  p.col_tiles = (p.E + 64 * VC - 1) / (64 * VC);
  const int64_t units = p.chunks * p.col_tiles;
  const dim3 grid((unsigned)((units + 3) / 4));
  const bool nt = p.n * p.E * (int64_t)sizeof(IO) > (int64_t(128) << 20);
  auto go = [&](auto fn) { hipLaunchKernelGGL(fn, grid, dim3(256), 0, s, p); };
  if (p.add) nt ? go(embed_sum_kernel<IO, OT, VC, true, true>) : go(embed_sum_kernel<IO, OT, VC, true, false>);
  else nt ? go(embed_sum_kernel<IO, OT, VC, false, true>) : go(embed_sum_kernel<IO, OT, VC, false, false>);
  if (p.chunks > 1) hipLaunchKernelGGL((embed_join_kernel<OT, VC>), dim3((unsigned)units), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename IO, typename OT>
hipError_t launch_once(const SortParams& sp, SumParams p, hipStream_t s) {
  p.col_tiles = (p.E + 255) / 256;
  const dim3 grid((unsigned)(p.chunks * p.col_tiles)), block(1024);
  auto go = [&](auto fn) { hipLaunchKernelGGL(fn, grid, block, 0, s, sp, p); };
  if (p.n <= 1024) p.add ? go(embed_once_kernel<IO, OT, 4, 1, true>) : go(embed_once_kernel<IO, OT, 4, 1, false>);
  else p.add ? go(embed_once_kernel<IO, OT, 4, 2, true>) : go(embed_once_kernel<IO, OT, 4, 2, false>);
  return hipGetLastError();
}

template <typename IO, typename OT>
hipError_t launch_io(const EmbedParams& e, const EmbedBwdPlan& pl, const SortParams& sp, SumParams p, char* ws,
                     hipStream_t s) {
  if (pl.transpose) {
    const int64_t blocks = e.Bsz * ((e.L + 127) / 128) * ((e.E + 63) / 64);
    IO* rows = reinterpret_cast<IO*>(ws + pl.rows);
    hipLaunchKernelGGL((embed_turn_kernel<IO>), grid_of(blocks), dim3(256), 0, s,
                       static_cast<const IO*>(e.dout), rows, e.Bsz, e.E, e.L);
    p.dout = rows;
  }
  if (pl.once) return launch_once<IO, OT>(sp, p, s);
  if constexpr (sizeof(IO) == 2)
    if (columns(e.E, true) == 8) return launch_sums<IO, OT, 8>(p, s);
  return launch_sums<IO, OT, 4>(p, s);
}

// A launch of a sort kernel whose workgroups behind the sort's clear `share` of the bytes left to fill.
template <typename F>
hipError_t with_fill(SortParams& sp, int64_t* left, double share, F&& go) {
  int64_t bytes = (int64_t)(*left * share) / kFill * kFill;
  if (share >= 1.0) bytes = *left;
  sp.fill_bytes = bytes;
  sp.fill_blocks = (bytes + kFill - 1) / kFill;
  if (sp.fill_blocks > kFillBlocks) sp.fill_blocks = kFillBlocks;
  go((unsigned)sp.fill_blocks);
  sp.fill += bytes;
  *left -= bytes;
  return hipGetLastError();
}

template <int NW, int R>
hipError_t launch_pass(SortParams& sp, int64_t* left, int passes_left, hipStream_t s) {
  const unsigned tiles = (unsigned)sp.tiles;
  hipError_t e = with_fill(sp, left, 1.0 / (2 * passes_left), [&](unsigned more) {
    hipLaunchKernelGGL((sort_count_kernel<NW, R>), dim3(tiles + more), dim3(NW * 64), 0, s, sp);
  });
  if (e != hipSuccess) return e;
  return with_fill(sp, left, 1.0 / (2 * passes_left - 1), [&](unsigned more) {
    hipLaunchKernelGGL((sort_move_kernel<NW, R>), dim3(tiles + more), dim3(NW * 64), 0, s, sp);
  });
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

void plan_embed_bwd(int64_t Bsz, int64_t L, int64_t V, int64_t E, int64_t table_size, bool io_bf16, bool cf, bool add,
                    EmbedBwdPlan* pl) {
  if (cf && embed_few_pays(Bsz, L, V, E, io_bf16)) return plan_embed_few(Bsz, L, V, E, pl);
  const int64_t n = Bsz * L;
  pl->bits = 1;
  while ((V >> pl->bits) != 0) ++pl->bits;  // keys 0 .. V
  pl->passes = (pl->bits + 7) / 8;
  pl->digit_bits = (pl->bits + pl->passes - 1) / pl->passes;
  pl->transpose = cf;
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t o = off; off += round256(bytes); return o; };
  if (pl->transpose) pl->rows = take((size_t)n * E * (io_bf16 ? 2 : 4));
  // All in one launch: up to 2048 positions, at most a workgroup per CU (a row per wave, or up to 4) and with little or
  // nothing to clear.  Calls of 509 x 768, added: 8.9 us, 13.8 with three launches; 2048 x 768: 8.7 and 17.4; 1024 x
  // 8192 (512 workgroups): 27 and 24.  What a single token names is one workgroup's work: 1024 and 2048 x 768 on one
  // token 30 and 53 us, 18 and 23 with three launches, and 98 and 34 for 4096 (else 13 and 22).  Not added: 509 x 768
  // into 2500 / 10000 / 20000 rows 9.4 / 10.4 / 15.1 and 13.7 / 15.6 / 18.5; 1 x 1000 into 70000 (280 MB): 79 and 54.
  const int64_t tiles = (E + 255) / 256;
  int64_t run = 16;
  while (run < 64 && (n + run - 1) / run * tiles > 256) run *= 2;
  int64_t chunks = (n + run - 1) / run;
  pl->once = n <= 2048 && chunks * tiles <= 256 && (add || V * E * table_size <= (int64_t(64) << 20));
  if (!add) {  // rows to clear: up to a workgroup per CU, where each wave has one
    const int64_t all = 256 / tiles < V / 16 ? 256 / tiles : V / 16;
    if (chunks < all) chunks = all;
  }
  if (pl->once) {
    pl->run = run;
    pl->chunks = chunks;
    if (!pl->transpose) take(1);  // (no size of 0 for a call that can be made)
    pl->total = off;
    return;
  }
  // Small tiles spread a short list over the chip; but each adds up the counts of all tiles, so long lists take
  // larger ones.  Whole calls of width 4 with tiles of 512 / 4096 / 8192: 29 / 38 / 46 us for 16384 positions,
  // 52 / 56 / 68 for 65536, 76 / 71 / 78 for 131072, 603 / 322 / 320 for 2^20, 6.0 / 0.96 / 0.90 ms for 2^22.
  pl->tile = n <= 4096 ? 4096 : n <= 65536 ? 512 : n <= 524288 ? 4096 : 8192;
  pl->tiles = (n + pl->tile - 1) / pl->tile;
  // Rows per chunk of the sums: about 4096 waves, so that short lists spread over the chip and long ones leave few
  // partial sums (16384 x 768: 52.1 us with 4096, 53.2 with 8192, 56.6 with 2048; 262144 x 1024: 153 with 128 rows,
  // 163 with 64, 176 with 32).
  const int64_t tiles_e = (E + 64 * columns(E, io_bf16) - 1) / (64 * columns(E, io_bf16));
  pl->run = 8;
  while (pl->run < 256 && n * tiles_e > pl->run * 4096) pl->run *= 2;
  pl->chunks = (n + pl->run - 1) / pl->run;
  for (int i = 0; i < (pl->tiles > 1 ? 2 : 1); ++i) {
    pl->key[i] = take((size_t)n * 4);
    pl->pos[i] = take((size_t)n * 4);
  }
  if (pl->tiles > 1) pl->hist = take((size_t)pl->tiles * 4 << pl->digit_bits);
  pl->part = take((size_t)pl->chunks * 2 * E * 4);
  pl->total = off;
}

hipError_t launch_embed_bwd(const EmbedParams& e, const EmbedBwdPlan& pl, bool table_bf16, bool io_bf16, void* ws,
                            hipStream_t s) {
  if (pl.few) return launch_embed_few(e, pl, table_bf16, io_bf16, ws, s);
  char* w = static_cast<char*>(ws);
  SortParams sp{};
  sp.tokens = e.tokens;
  sp.hist = reinterpret_cast<uint32_t*>(w + pl.hist);
  sp.n = e.T; sp.V = e.V; sp.tiles = pl.tiles; sp.i64 = e.i64; sp.bits = pl.digit_bits; sp.passes = pl.passes;
  sp.fill = static_cast<char*>(e.out);
  int64_t left = e.add ? 0 : e.V * e.E * (table_bf16 ? 2 : 4);
  hipError_t rc = hipSuccess;
  if (pl.tiles == 1 && !pl.once) {
    sp.key_out = reinterpret_cast<uint32_t*>(w + pl.key[0]);
    sp.pos_out = reinterpret_cast<uint32_t*>(w + pl.pos[0]);
    rc = with_fill(sp, &left, 1.0, [&](unsigned more) {
      const dim3 grid(1 + more), block(1024);
      if (e.T <= 1024) hipLaunchKernelGGL(sort_small_kernel<1>, grid, block, 0, s, sp);
      else hipLaunchKernelGGL(sort_small_kernel<4>, grid, block, 0, s, sp);
    });
    if (rc != hipSuccess) return rc;
  }
  for (int k = 0; pl.tiles > 1 && k < pl.passes; ++k) {
    sp.key_out = reinterpret_cast<uint32_t*>(w + pl.key[k & 1]);
    sp.pos_out = reinterpret_cast<uint32_t*>(w + pl.pos[k & 1]);
    sp.shift = k * pl.digit_bits;
    rc = pl.tile == 512    ? launch_pass<4, 2>(sp, &left, pl.passes - k, s)
         : pl.tile == 4096 ? launch_pass<8, 8>(sp, &left, pl.passes - k, s)
                           : launch_pass<16, 8>(sp, &left, pl.passes - k, s);
    if (rc != hipSuccess) return rc;
    sp.tokens = nullptr;
    sp.key_in = sp.key_out;
    sp.pos_in = sp.pos_out;
  }
  SumParams p{};
  p.key = sp.key_out; p.pos = sp.pos_out; p.dout = e.dout; p.dweight = e.out;
  p.part = reinterpret_cast<float*>(w + pl.part);
  p.n = e.T; p.V = e.V; p.E = e.E; p.run = pl.run; p.chunks = pl.chunks;
  p.scale = e.scale; p.add = e.add;
  if (io_bf16)
    return table_bf16 ? launch_io<bf16_t, bf16_t>(e, pl, sp, p, w, s) : launch_io<bf16_t, float>(e, pl, sp, p, w, s);
  return table_bf16 ? launch_io<float, bf16_t>(e, pl, sp, p, w, s) : launch_io<float, float>(e, pl, sp, p, w, s);
}

}  // namespace ssm
