// norm_rows.hip -- layer norm and RMS norm of rows, with what comes before them in a residual block, and the gradients.
//
//   s = residual + dropout(x);  m = mean(s) (RMS: 0);  r = 1 / sqrt(mean((s - m)^2) + eps)
//   hidden = s;  out = (s - m) r w + b
//   backward, with xh = (s - m) r and g = dout w:
//   ds = r (g - mean(g) - xh mean(g xh)) + dhidden (RMS: without mean(g));  dresidual = ds;  dx = dropout(ds)
//   dw = sum over rows of dout xh;  db = sum over rows of dout
//
// Bound by HBM: every stream is read once and written once.  A row's team (16, 32 or 64 lanes, or a workgroup of as many
// waves as it takes) holds the row in registers, 8 elements a lane, so that the variance is a second pass over registers
// (about the mean, no cancellation).  out is made from the unrounded sum; the hidden that is kept for the backward
// pass is rounded to its type.  Where E is no multiple of 8 a row's pieces begin up to 7 elements before it, at a
// multiple of 16 bytes (16384 x 767 in bf16 with a residual: 27.7 us; with pieces that begin where the row does 38.7).
// Rows that a workgroup does not hold (forward more than 16384 elements, backward more than 8192, one piece a lane; 16377
// and 8185 where E is no multiple of 8) go through memory again for each pass.
//
// A lane holds one piece, two above 4096 elements: a row's loads are then all in flight at once, few instructions stand
// between them and the stores, and what a call of few rows takes is one pass through a short kernel (256 x 2560: 3.5 us;
// 6 pieces a lane, one wave a row: 12).  16384 x 768 in bf16 into a stream in fp32, with dropout (151 MB): 31 us, 4.9
// TB/s (16 lanes a row, 6 pieces each: 39; two pieces 33); 16384 x 2048, bf16 with a residual: 45.6 us, 5.9 TB/s; 16384 x
// 8176: 110 us, 4.9 TB/s (one piece a lane 131).  Rows in turn with the next one's loads under way take twice the
// registers and gave 33, 49 and 141.
//
// Backward: 16384 x 768 as above, with the stream's own gradient (201 MB): 39 us, 5.3 TB/s, and 6 for the join of the sums.
// Odd widths over 512 keep up to 12 registers in scratch memory, the other forms none.
#include "block_device.h"

namespace ssm {

namespace {

// Lanes of a row's team with `each` pieces a lane; 0: rows that no team holds.
int team_of(int64_t E, int each = 1) {
  const int64_t n = (E + (E % 8 ? 7 : 0) + 7) / 8;
  if (n <= 64) return n <= 16 ? 16 : n <= 32 ? 32 : 64;
  const int64_t lanes = (n + each * 64 - 1) / (each * 64) * 64;
  return lanes <= 1024 ? (int)lanes : 0;
}
constexpr int64_t kTwo = 4096;  // elements from which on a lane holds two pieces (forward)
constexpr int kLong = 1024;     // lanes of a row that no team holds (16 x 200000: 84 us, 250 with 256)
constexpr int kTurns = 256;     // rows in turn of a team in the backward pass

// (a, b) summed over the team's lanes, in all of them; TEAM 0: the workgroup; sm: two floats for each of 16 waves
template <int TEAM>
__device__ __forceinline__ void sum_team(float& a, float& b, float (*sm)[2]) {
  if constexpr (TEAM == 16 || TEAM == 64) {
    a = sum_lanes<TEAM>(a);
    b = sum_lanes<TEAM>(b);
  } else if constexpr (TEAM == 32) {
    a = sum_lanes<16>(a);
    b = sum_lanes<16>(b);
    a += __shfl_xor(a, 16);
    b += __shfl_xor(b, 16);
  } else {
    a = sum_lanes<64>(a);
    b = sum_lanes<64>(b);
    if ((threadIdx.x & 63) == 0) {
      sm[threadIdx.x >> 6][0] = a;
      sm[threadIdx.x >> 6][1] = b;
    }
    __syncthreads();
    const int k = threadIdx.x & 15;
    const bool wave = k < (int)(blockDim.x >> 6);
    a = sum_lanes<16>(wave ? sm[k][0] : 0.0f);
    b = sum_lanes<16>(wave ? sm[k][1] : 0.0f);
  }
}
template <int TEAM> __device__ __forceinline__ float sum_team(float a, float (*sm)[2]) {
  float none = 0.0f;
  sum_team<TEAM>(a, none, sm);
  return a;
}

}  // namespace

// A row each, P pieces a lane.  ODD: E is no multiple of 8.
template <typename XT, typename HT, int TEAM, int P, bool ODD>
__global__ __launch_bounds__(TEAM ? 256 : 1024) void norm_rows_kernel(NormParams p) {
  constexpr int R = TEAM ? 256 / (TEAM ? TEAM : 1) : 1;
  __shared__ float sm[2][16][2];
  const int LN = TEAM ? TEAM : blockDim.x;
  const int lane = TEAM ? threadIdx.x % (TEAM ? TEAM : 1) : threadIdx.x, team = TEAM ? threadIdx.x / (TEAM ? TEAM : 1) : 0;
  const int64_t row = (int64_t)block_id() * R + team;
  if (row >= p.rows) return;
  const int64_t E = p.E, total = p.rows * E, base = row * E;
  const Drop drop(p.drop);
  const int before = ODD ? (int)(base % 8) : 0;
  auto at = [&](int k) { return (int64_t)((k * LN + lane) * 8 - before); };
  auto held = [&](int k) {
    Part n(at(k), E);
    if (!ODD) n.hi = n.hi ? 8 : 0, n.lo = 0;
    return n;
  };
  Piece<XT> a[P];
  Piece<HT> b[P];
  Piece<float> w[P], c[P];  // the columns' weights and biases
#pragma unroll
  for (int k = 0; k < P; ++k) {
    const int64_t e = at(k);
    const bool may = held(k).any() && (!ODD || base + e + 8 <= total);
    a[k].full(static_cast<const XT*>(p.x) + base + e, may);
    if (p.residual) b[k].full(static_cast<const HT*>(p.residual) + base + e, may);
  }
#pragma unroll
  for (int k = 0; k < P; ++k) {
    const Part n = held(k);
    if (p.weight) w[k].full(p.weight + at(k), n.whole());
    if (p.bias) c[k].full(p.bias + at(k), n.whole());
  }
  float s[P][8], m = 0.0f, v = 0.0f;  // what is normalised (zeros outside the row)
#pragma unroll
  for (int k = 0; k < P; ++k) {
    if constexpr (ODD) {
      const Part n = held(k);
      const int64_t e = at(k);
      if (n.any() && !n.whole()) {
        if (p.weight) w[k].part(p.weight + e, n);
        if (p.bias) c[k].part(p.bias + e, n);
        if (base + e + 8 > total) {  // the tensor's end
          a[k].part(static_cast<const XT*>(p.x) + base + e, n);
          if (p.residual) b[k].part(static_cast<const HT*>(p.residual) + base + e, n);
        }
        a[k].cut(n);
        if (p.residual) b[k].cut(n);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s[k][i] = a[k].at(i);
    if (drop.any()) drop.apply(drop.kept((uint64_t)(base + at(k))), s[k]);
    if (p.residual) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[k][i] += b[k].at(i);
    }
    if (p.hidden) store_part(static_cast<HT*>(p.hidden) + base + at(k), held(k), s[k]);
  }
  if (!p.rms) {
#pragma unroll
    for (int k = 0; k < P; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) m += s[k][i];
    m = sum_team<TEAM>(m, sm[0]) * p.inv_e;
  }
#pragma unroll
  for (int k = 0; k < P; ++k) {
    const Part n = held(k);
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float d = s[k][i] - m;
      if (ODD) d = n.has(i) ? d : 0.0f;
      q = __builtin_fmaf(d, d, q);
    }
    v += n.any() ? q : 0.0f;
  }
  const float r = 1.0f / sqrtf(sum_team<TEAM>(v, sm[1]) * p.inv_e + p.eps);
#pragma unroll
  for (int k = 0; k < P; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s[k][i] = (s[k][i] - m) * r;
    if (p.weight) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[k][i] *= w[k].at(i);
    }
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[k][i] += c[k].at(i);
    }
    store_part(static_cast<XT*>(p.out) + base + at(k), held(k), s[k]);
  }
  if (p.stats && lane == 0) {
    p.stats[row] = m;
    p.stats[p.rows + row] = r;
  }
}

// A row of any length by a workgroup, 8 elements a lane at a time, read again for every pass.  A lane's share is up to 2^20
// elements: each piece is summed by itself, the pieces' sums are compensated (constant rows of 2^24: (s - m) r was 0.06).
template <typename XT, typename HT>
__global__ __launch_bounds__(kLong) void norm_long_kernel(NormParams p) {
  __shared__ float sm[2][16][2];
  const int64_t row = block_id(), E = p.E, base = row * E;
  if (row >= p.rows) return;
  const XT* x = static_cast<const XT*>(p.x) + base;
  const HT* res = p.residual ? static_cast<const HT*>(p.residual) + base : nullptr;
  const Drop drop(p.drop);
  float s[8];
  LongSum sum, squares;
  auto take = [&](int64_t e, const Part& n) {
    Piece<XT> a;
    Piece<HT> b;
    a.full(x + e, n.whole());
    if (res) b.full(res + e, n.whole());
    if (!n.whole()) {
      a.part(x + e, n);
      a.cut(n);
      if (res) {
        b.part(res + e, n);
        b.cut(n);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = a.at(k);
    if (drop.any()) drop.apply(drop.kept((uint64_t)(base + e)), s);
    if (res) {
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] += b.at(k);
    }
  };
  const int64_t e0 = threadIdx.x * 8;
  for (int64_t e = e0; e < E; e += kLong * 8) {
    const Part n(e, E);
    take(e, n);
    if (p.hidden) store_part(static_cast<HT*>(p.hidden) + base + e, n, s);
    sum.add(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])));
  }
  const float m = p.rms ? 0.0f : sum_team<0>(sum.value(), sm[0]) * p.inv_e;
  for (int64_t e = e0; e < E; e += kLong * 8) {
    const Part n(e, E);
    take(e, n);
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = n.has(k) ? s[k] - m : 0.0f;
      v = __builtin_fmaf(d, d, v);
    }
    squares.add(v);
  }
  const float r = 1.0f / sqrtf(sum_team<0>(squares.value(), sm[1]) * p.inv_e + p.eps);
  for (int64_t e = e0; e < E; e += kLong * 8) {
    const Part n(e, E);
    take(e, n);
    float w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = (s[k] - m) * r;
    if (p.weight) {
      load_n<float, 8>(p.weight + e, n.hi, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] *= w[k];
    }
    if (p.bias) {
      load_n<float, 8>(p.bias + e, n.hi, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] += w[k];
    }
    store_part(static_cast<XT*>(p.out) + base + e, n, s);
  }
  if (p.stats && threadIdx.x == 0) {
    p.stats[row] = m;
    p.stats[p.rows + row] = r;
  }
}

// Rows p.from .. p.to - 1 in turn (p.blocks workgroups); dw and db of the lane's columns are added up over the team's rows in
// registers, then over the workgroup's teams in LDS, and go to memory as the workgroup's partial sums.  ODD: a team's
// rows are 8 k apart, so that they all begin alike and a lane keeps its columns.
template <typename XT, typename HT, int TEAM, bool ODD>
__global__ __launch_bounds__(TEAM ? 256 : 1024) void norm_rows_bwd_kernel(NormParams p) {
  constexpr int R = TEAM ? 256 / (TEAM ? TEAM : 1) : 1;
  __shared__ float sm[2][16][2];
  __shared__ float acc[R > 1 ? 256 * 8 : 1];
  const int lane = TEAM ? threadIdx.x % (TEAM ? TEAM : 1) : threadIdx.x, team = TEAM ? threadIdx.x / (TEAM ? TEAM : 1) : 0;
  const int64_t E = p.E, total = p.rows * E;
  const XT* dout = static_cast<const XT*>(p.x);
  const HT* hidden = static_cast<const HT*>(p.residual);
  const HT* dhidden = static_cast<const HT*>(p.dhidden);
  const Drop drop(p.drop);
  const int64_t first = p.from + (int64_t)block_id() * R + team;
  const int64_t e = lane * 8 - (ODD ? (int)(first * E % 8) : 0);
  Part n(e, E);
  if (!ODD) n.hi = n.hi ? 8 : 0, n.lo = 0;
  Piece<float> w;
  if (p.weight) {
    w.full(p.weight + e, n.whole());
    if (ODD && n.any() && !n.whole()) w.part(p.weight + e, n);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) w.w[k >> 2][k & 3] = 0x3f800000u;
  }
  float dw[8], db[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) dw[k] = db[k] = 0.0f;
  int turn = 0;
  for (int64_t row = first; row < p.to; row += p.blocks * R, turn ^= 1) {
    const int64_t at = row * E + e;
    const bool end = ODD && at + 8 > total, may = n.any() && !end;
    Piece<XT> a;
    Piece<HT> b, q;
    a.full(dout + at, may);
    b.full(hidden + at, may);
    if (dhidden) q.full(dhidden + at, may);
    const float m = p.stats[row], r = p.stats[p.rows + row];
    if constexpr (ODD) {
      if (n.any() && !n.whole()) {
        if (end) {
          a.part(dout + at, n);
          b.part(hidden + at, n);
          if (dhidden) q.part(dhidden + at, n);
        }
        a.cut(n);
        b.cut(n);
      }
    }
    float g[8], h[8], c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = a.at(k);  // (zero outside the row)
      h[k] = (b.at(k) - m) * r;
      dw[k] = __builtin_fmaf(d, h[k], dw[k]);
      db[k] += d;
      g[k] = d * w.at(k);
      c1 += g[k];
      c2 = __builtin_fmaf(g[k], h[k], c2);
    }
    sum_team<TEAM>(c1, c2, sm[turn]);  // (the other half may still be read)
    c1 = p.rms ? 0.0f : c1 * p.inv_e;
    c2 *= p.inv_e;
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = r * (g[k] - c1 - h[k] * c2);
    if (dhidden) {
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] += q.at(k);
    }
    if (p.hidden) store_part(static_cast<HT*>(p.hidden) + at, n, g);
    if (p.out) {
      if (drop.any()) drop.apply(drop.kept((uint64_t)at), g);
      store_part(static_cast<XT*>(p.out) + at, n, g);
    }
  }
  if (!p.part) return;
  float* part = p.part + (int64_t)block_id() * 2 * E;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if constexpr (R > 1) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[threadIdx.x * 8 + k] = which ? db[k] : dw[k];
      __syncthreads();
      for (int c = threadIdx.x; c < E; c += 256) {
        float s = 0.0f;
#pragma unroll
        for (int t = 0; t < R; ++t)
          s += acc[t * TEAM * 8 + c + (ODD ? (int)((p.from + (int64_t)block_id() * R + t) * E % 8) : 0)];
        part[which * E + c] = s;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (n.has(k)) part[which * E + e + k] = which ? db[k] : dw[k];
    }
  }
}

// The gradients of a row of any length by a workgroup, read twice; dw and db are summed by norm_sums_kernel.
template <typename XT, typename HT>
__global__ __launch_bounds__(kLong) void norm_long_bwd_kernel(NormParams p) {
  __shared__ float sm[16][2];
  const int64_t row = block_id(), E = p.E, base = row * E;
  if (row >= p.rows) return;
  const Drop drop(p.drop);
  const float m = p.stats[row], r = p.stats[p.rows + row];
  float g[8], h[8];
  Piece<HT> q;
  auto take = [&](int64_t e, const Part& n) {
    Piece<XT> a;
    Piece<HT> b;
    const int64_t at = base + e;
    a.full(static_cast<const XT*>(p.x) + at, n.whole());
    b.full(static_cast<const HT*>(p.residual) + at, n.whole());
    if (p.dhidden) q.full(static_cast<const HT*>(p.dhidden) + at, n.whole());
    if (!n.whole()) {
      a.part(static_cast<const XT*>(p.x) + at, n);
      b.part(static_cast<const HT*>(p.residual) + at, n);
      if (p.dhidden) q.part(static_cast<const HT*>(p.dhidden) + at, n);
      a.cut(n);
    }
    if (p.weight) {
      load_n<float, 8>(p.weight + e, n.hi, g);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] = 1.0f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      h[k] = (b.at(k) - m) * r;
      g[k] *= a.at(k);
    }
  };
  LongSum s1, s2;
  for (int64_t e = threadIdx.x * 8; e < E; e += kLong * 8) {
    const Part n(e, E);
    take(e, n);
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      a += g[k];
      b = n.has(k) ? __builtin_fmaf(g[k], h[k], b) : b;
    }
    s1.add(a);
    s2.add(b);
  }
  float c1 = s1.value(), c2 = s2.value();
  sum_team<0>(c1, c2, sm);
  c1 = p.rms ? 0.0f : c1 * p.inv_e;
  c2 *= p.inv_e;
  for (int64_t e = threadIdx.x * 8; e < E; e += kLong * 8) {
    const Part n(e, E);
    take(e, n);
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = r * (g[k] - c1 - h[k] * c2) + (p.dhidden ? q.at(k) : 0.0f);
    if (p.hidden) store_part(static_cast<HT*>(p.hidden) + base + e, n, g);
    if (p.out) {
      if (drop.any()) drop.apply(drop.kept((uint64_t)(base + e)), g);
      store_part(static_cast<XT*>(p.out) + base + e, n, g);
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

namespace {

template <typename XT, typename HT, int TEAM, int P>
void go(const NormParams& p, int lanes, hipStream_t s) {
  constexpr int R = TEAM ? 256 / (TEAM ? TEAM : 1) : 1;
  const dim3 grid = grid_of((p.rows + R - 1) / R), block(TEAM ? 256 : lanes);
  if (p.E % 8) hipLaunchKernelGGL((norm_rows_kernel<XT, HT, TEAM, P, true>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((norm_rows_kernel<XT, HT, TEAM, P, false>), grid, block, 0, s, p);
}

template <typename XT, typename HT>
void fwd(const NormParams& p, hipStream_t s) {
  const int lanes = team_of(p.E, p.E > kTwo ? 2 : 1);
  switch (lanes) {
    case 0:
      hipLaunchKernelGGL((norm_long_kernel<XT, HT>), grid_of(p.rows), dim3(kLong), 0, s, p);
      return;
    case 16: return go<XT, HT, 16, 1>(p, lanes, s);
    case 32: return go<XT, HT, 32, 1>(p, lanes, s);
    case 64: return go<XT, HT, 64, 1>(p, lanes, s);
    default: return p.E > kTwo ? go<XT, HT, 0, 2>(p, lanes, s) : go<XT, HT, 0, 1>(p, lanes, s);
  }
}

// Workgroups of the backward pass, each of which leaves a partial sum of dw and db: about 16 waves a compute unit, the
// same number on each (16384 x 5000, 10 waves a row: 84 us with 512, 117 and 100 with 256 and 768), and where the
// rows are fewer, up to 12 rows in turn rather than more sums (16384 x 768: 39 us with 1366, 41.6 with 2048, 51 with
// 4096), but 512 at least.  A multiple of 8 where E is none.  A plain sum over rows in turn is off by up to their number of
// half steps: of very many rows, each launch takes kTurns (2^20 x 768: 1.19 ms; more workgroups instead, of which not all
// are resident at once, take a tenth more).  Rows that no team holds: groups of rows in one launch.
struct BwdPlan {
  int64_t groups, launches;
};
BwdPlan bwd_plan(int64_t rows, int64_t E) {
  const int lanes = team_of(E);
  if (!lanes) return {rows < 64 ? rows : rows <= 64 * kTurns ? 64 : (rows + kTurns - 1) / kTurns, 1};
  const int64_t waves = lanes <= 64 ? 4 : lanes / 64, R = lanes <= 64 ? 256 / lanes : 1;
  const int64_t each = (16 + waves - 1) / waves < 24 / waves ? (16 + waves - 1) / waves : 24 / waves;
  const int64_t all = (rows + R - 1) / R, most = 256 * each;
  int64_t turns = (all + 511) / 512 < 12 ? (all + 511) / 512 : 12;
  if (turns < (all + most - 1) / most) turns = (all + most - 1) / most;
  const int64_t n = (all + turns - 1) / turns;
  return {E % 8 ? (n + 7) / 8 * 8 : n, (turns + kTurns - 1) / kTurns};
}

template <typename XT, typename HT, int TEAM>
void go_bwd(const NormParams& p, int lanes, hipStream_t s) {
  const BwdPlan plan = bwd_plan(p.rows, p.E);
  const dim3 grid = grid_of(plan.groups), block(TEAM ? 256 : lanes);
  const int64_t step = kTurns * plan.groups * (TEAM ? 256 / (TEAM ? TEAM : 1) : 1);
  NormParams q = p;
  q.blocks = plan.groups;
  for (int64_t k = 0; k < plan.launches; ++k) {
    q.from = k * step;
    q.to = q.from + step < p.rows ? q.from + step : p.rows;
    q.part = p.part ? p.part + k * plan.groups * 2 * p.E : nullptr;
    if (p.E % 8) hipLaunchKernelGGL((norm_rows_bwd_kernel<XT, HT, TEAM, true>), grid, block, 0, s, q);
    else hipLaunchKernelGGL((norm_rows_bwd_kernel<XT, HT, TEAM, false>), grid, block, 0, s, q);
  }
}

template <typename XT, typename HT>
void bwd(const NormParams& p, hipStream_t s) {
  const int lanes = team_of(p.E);
  switch (lanes) {
    case 0:
      hipLaunchKernelGGL((norm_long_bwd_kernel<XT, HT>), grid_of(p.rows), dim3(kLong), 0, s, p);
      if (p.part)
        hipLaunchKernelGGL((norm_sums_kernel<XT, HT>), grid_of((p.E + 255) / 256 * p.blocks), dim3(256), 0, s, p);
      return;
    case 16: return go_bwd<XT, HT, 16>(p, lanes, s);
    case 32: return go_bwd<XT, HT, 32>(p, lanes, s);
    case 64: return go_bwd<XT, HT, 64>(p, lanes, s);
    default: return go_bwd<XT, HT, 0>(p, lanes, s);
  }
}

}  // namespace

int64_t norm_rows_bwd_blocks(int64_t rows, int64_t E) {
  const BwdPlan plan = bwd_plan(rows, E);
  return plan.groups * plan.launches;
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

}  // namespace ssm
