// recur_fwd.hip -- the gated linear recurrence over a sequence, and one step of it.
//
// Bound by HBM: x, r, i (and z) are read once, out is written once (8 or 10 bytes a step in bf16).  A step is an affine
// map of the state; a lane composes those of its V steps, the wave those of its lanes (DPP), and the state that enters
// the wave's 64 pieces then gives all states.  Rows are walked in turns of W * 64 pieces by a team of W waves, whose
// maps go through LDS, so that the sequence is read once however long it is; the next turn's pieces are loaded before
// the present one's arithmetic.  Where there are too few rows even for that, a row is cut into S segments and the first
// launch makes each segment's map (reading x, r and i once more).
//
// 8 x 1536 x 2048 in bf16 with a gate, a wave a row: 56 us a call, 4.5 TB/s; 1 x 1024 x 2^20, 8
// waves a row: 1.75 ms, 4.9 TB/s.
#include "recur_device.h"

namespace ssm {

namespace {

// The map of all of the team's lanes before this one's piece (A, B: the lane's own map before, the map of the lanes of
// its wave before it after), and the state that enters the wave; carry: the state that enters the team, then leaves it.
template <int LN, int W>
__device__ __forceinline__ float enter_up(float& A, float& B, float& carry, float (*sm)[2], int w) {
  scan_up<LN>(A, B);
  const float ta = end_lane<LN, true>(A), tb = end_lane<LN, true>(B);
  A = lane_before<LN>(A, 1.0f);
  B = lane_before<LN>(B, 0.0f);
  float in = carry;
  if constexpr (W == 1) {
    carry = __builtin_fmaf(ta, carry, tb);
  } else {
    if ((threadIdx.x & 63) == 0) {
      sm[w][0] = ta;
      sm[w][1] = tb;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < W; ++k) {
      if (k == w) in = carry;
      carry = __builtin_fmaf(sm[k][0], carry, sm[k][1]);
    }
  }
  return in;
}

}  // namespace

// Z: there is a gate.  MAPS: the segments' maps instead of the outputs.
template <typename IO, int LN, int W, bool REV, bool Z, bool MAPS>
__global__ __launch_bounds__(W > 4 ? W * 64 : 256) void recur_fwd_kernel(RecurParams p) {
  constexpr int V = 16 / (int)sizeof(IO);
  constexpr int UNITS = W > 4 ? 1 : 256 / (LN * W);  // row segments per workgroup
  constexpr int TURN = LN * W * V;       // slots
  __shared__ float sm[2][W][2];
  const int lane = threadIdx.x % LN, w = W > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / 64) : 0;
  const int64_t S = MAPS ? p.plan.S - 1 : p.plan.S;
  const int64_t rows = p.B * p.D, total = rows * p.L;
  int64_t unit = (int64_t)block_id() * UNITS + (W > 1 ? 0 : threadIdx.x / LN);
  const bool live = unit < rows * S;
  if (W > 1 || LN == 64) {
    if (!live) return;
    unit = __builtin_amdgcn_readfirstlane((int)unit);
  } else if (!live) {
    return;
  }
  const int64_t row = unit / S, seg = unit - row * S, d = row % p.D;
  const Row<IO, REV> line(row, p.L);
  const Channel ch(p.decay, p.rb, p.ib, d);
  const int64_t k0 = seg * p.plan.per, k1 = k0 + p.plan.per < p.plan.tiles ? k0 + p.plan.per : p.plan.tiles;

  float carry = 0.0f, whole = 1.0f;
  if (!MAPS) {
    carry = p.init ? p.init[row] : 0.0f;
    if (p.plan.S > 1) {  // the segments before, one a lane
      const int l = threadIdx.x & 63;
      float A = 1.0f, B = 0.0f;
      if (l < seg) {
        A = p.seg[(l * rows + row) * 2];
        B = p.seg[(l * rows + row) * 2 + 1];
      }
      scan_up<64>(A, B);
      carry = __builtin_fmaf(lane_of(A, 63), carry, lane_of(B, 63));
    }
  }

  const u32x4a none = {0u, 0u, 0u, 0u};
  u32x4a xn = none, rn = none, in = none, zn = none;
  const bool gate = Z && !MAPS && p.out;
  auto load = [&](int64_t tile) {
    const int64_t s = tile * TURN + (w * LN + lane) * V, at = line.at(s);
    const int lo = line.lo(s), hi = line.hi(s);
    const bool edge = line.edge(tile * TURN, TURN);
    xn = load_slots<IO, REV>(p.x, at, lo, hi, edge, total);
    rn = load_slots<IO, REV>(p.r, at, lo, hi, edge, total);
    in = load_slots<IO, REV>(p.i, at, lo, hi, edge, total);
    if (gate) zn = load_slots<IO, REV>(p.z, at, lo, hi, edge, total);
  };
  if (k0 < k1) load(k0);
  for (int64_t tile = k0; tile < k1; ++tile) {
    const u32x4a xq = xn, rq = rn, iq = in, zq = zn;
    if (LN == 64 && tile + 1 < k1) load(tile + 1);
    const int64_t s = tile * TURN + (w * LN + lane) * V;
    const int lo = line.lo(s), hi = line.hi(s);
    const bool edge = line.edge(tile * TURN, TURN);
    float a[V], v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const Gates g(slot<IO, REV>(rq, e), slot<IO, REV>(iq, e), ch);
      a[e] = g.a;
      v[e] = g.q * g.si * slot<IO, REV>(xq, e);
    }
    if (edge) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        a[e] = e < lo || e >= hi ? 1.0f : a[e];
        v[e] = e < lo || e >= hi ? 0.0f : v[e];
      }
    }
    float A = a[0], B = v[0];
#pragma unroll
    for (int e = 1; e < V; ++e) {
      A *= a[e];
      B = __builtin_fmaf(a[e], B, v[e]);
    }
    if (MAPS) {  // (the team's map, built up in `whole` and `carry`)
      scan_up<LN>(A, B);
      const float ta = end_lane<LN, true>(A), tb = end_lane<LN, true>(B);
      if constexpr (W == 1) {
        carry = __builtin_fmaf(ta, carry, tb);
        whole *= ta;
      } else {
        float (*q)[2] = sm[tile & 1];
        if ((threadIdx.x & 63) == 0) {
          q[w][0] = ta;
          q[w][1] = tb;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < W; ++k) {
          carry = __builtin_fmaf(q[k][0], carry, q[k][1]);
          whole *= q[k][0];
        }
      }
      continue;
    }
    const float enter = enter_up<LN, W>(A, B, carry, sm[tile & 1], w);
    const int64_t block = tile * W + w;
    if (p.ckpt && lane == 0 && block < p.plan.blocks) p.ckpt[row * p.plan.blocks + block] = enter;
    if (!p.out) continue;
    float h = __builtin_fmaf(A, enter, B), o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      h = __builtin_fmaf(a[e], h, v[e]);
      o[e] = Z ? h * silu_(slot<IO, REV>(zq, e)) : h;
    }
    store_slots<IO, REV>(p.out, line.at(s), lo, hi, edge, o);
    if (LN < 64) break;  // (rows of fewer lanes are one turn)
  }
  if (MAPS) {
    if (lane == 0 && w == 0) {
      p.seg[(seg * rows + row) * 2] = whole;
      p.seg[(seg * rows + row) * 2 + 1] = carry;
    }
  } else if (p.last && seg == S - 1 && lane == 0 && w == 0) {
    p.last[row] = carry;
  }
}

// One step: the same gates, the state updated in place.  A lane owns 4 consecutive elements of [B, D].  EVEN: they are of
// one row, so that the channels' numbers come in one piece each (256 x 5120: 12.9 us with a load for each).
template <typename IO, bool EVEN>
__global__ __launch_bounds__(256) void recur_step_kernel(RecurStepParams p) {
  const int64_t at = ((int64_t)block_id() * 256 + threadIdx.x) * 4;
  if (at >= p.n) return;
  const int n = EVEN || p.n - at >= 4 ? 4 : (int)(p.n - at);
  float x[4], r[4], i[4], z[4], h[4], o[4], c[3][4];
  load_n<IO, 4>(static_cast<const IO*>(p.r) + at, n, r);
  load_n<IO, 4>(static_cast<const IO*>(p.i) + at, n, i);
  load_n<IO, 4>(static_cast<const IO*>(p.x) + at, n, x);
  if (p.z) load_n<IO, 4>(static_cast<const IO*>(p.z) + at, n, z);
  load_n<float, 4>(p.state + at, n, h);
  int64_t d = p.n <= 0xffffffffll ? (uint32_t)at % (uint32_t)p.D : at % p.D;
  if (EVEN) {
    const float* const of[] = {p.decay, p.rb, p.ib};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (of[k]) {
        load_n<float, 4>(of[k] + d, 4, c[k]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) c[k][e] = 0.0f;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[0][e] = p.decay[d];
      c[1][e] = p.rb ? p.rb[d] : 0.0f;
      c[2][e] = p.ib ? p.ib[d] : 0.0f;
      if (++d == p.D) d = 0;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const Gates g(r[e], i[e], Channel(c[0][e], c[1][e], c[2][e]));
    h[e] = __builtin_fmaf(g.a, h[e], g.q * g.si * x[e]);
    o[e] = p.z ? h[e] * silu_(z[e]) : h[e];
  }
  store_n<float, 4>(p.state + at, n, h);
  store_n<IO, 4>(static_cast<IO*>(p.out) + at, n, o);
}

// Short rows take the 1, 4, 16 or 32 lanes that hold all of their pieces (256 x 2560 x 8 in bf16: 15 us, 214 with 16
// lanes; 64 x 1536 x 256: 62, 77 with 16 lanes twice), longer ones a wave: a row at a time costs least where there are rows
// for every SIMD (8 x 1536 x 2048: 57 us, 77 with four waves a row).  Fewer rows take four or eight waves each, if they are
// long enough for several turns (1 x 2048 x 65536: 264 us, 248 with four, 228 with eight; 2 x 1536 x 8192: 54, 63, 83)
// or there is no other way to fill the card; and where that is still too few, segments, up to 64 (a lane each for their
// maps), of two turns and more.
RecurPlan recur_plan(int64_t B, int64_t D, int64_t L, bool bf16) {
  const int64_t V = bf16 ? 8 : 4, rows = B * D;
  RecurPlan pl;
  pl.blocks = (L + V - 1 + 64 * V - 1) / (64 * V);
  const int64_t most = L % V ? (L + 2 * V - 2) / V : L / V;  // pieces of a row that begins anywhere
  if (most <= 32) pl.lanes = most <= 1 ? 1 : most <= 4 ? 4 : most <= 16 ? 16 : 32;
  else if (rows < 256) pl.waves = pl.blocks >= 4 ? 4 : 1;
  else if ((rows < 1024 && pl.blocks >= 8) || (rows <= 2048 && pl.blocks >= 64)) pl.waves = 8;
  else if ((rows < 2048 && pl.blocks >= 4) || (rows < 4096 && pl.blocks >= 32)) pl.waves = 4;
  const int64_t turn = pl.lanes * pl.waves * V;
  pl.tiles = pl.lanes < 64 ? 1 : (L + V - 1 + turn - 1) / turn;
  pl.per = pl.tiles;
  if (pl.waves == 4 && rows < 256) {
    int64_t S = (1023 + rows) / rows;
    if (S > pl.tiles / 2) S = pl.tiles / 2;
    if (S > 64) S = 64;
    if (S > 1) {
      pl.per = (pl.tiles + S - 1) / S;
      pl.S = (pl.tiles + pl.per - 1) / pl.per;
    }
  }
  // 64 to 127 turns a partial sum
  pl.parts = pl.per < 128 ? 1 : (int)(pl.per / 64);
  pl.chain = (int)((pl.per + pl.parts - 1) / pl.parts);
  return pl;
}

namespace {

template <typename IO, bool REV, bool Z>
void go(const RecurParams& p, hipStream_t s) {
  const int64_t rows = p.B * p.D;
  auto few = [&](auto lanes) {
    constexpr int LN = decltype(lanes)::value, ROWS = 256 / LN;
    hipLaunchKernelGGL((recur_fwd_kernel<IO, LN, 1, REV, Z, false>), grid_of((rows + ROWS - 1) / ROWS), dim3(256), 0, s, p);
  };
  if (p.plan.lanes < 64) {
    p.plan.lanes == 1 ? few(IC<1>()) : p.plan.lanes == 4 ? few(IC<4>()) : p.plan.lanes == 16 ? few(IC<16>()) : few(IC<32>());
  } else if (p.plan.waves == 1) {
    hipLaunchKernelGGL((recur_fwd_kernel<IO, 64, 1, REV, Z, false>), grid_of((rows + 3) / 4), dim3(256), 0, s, p);
  } else if (p.plan.waves == 8) {
    hipLaunchKernelGGL((recur_fwd_kernel<IO, 64, 8, REV, Z, false>), grid_of(rows), dim3(512), 0, s, p);
  } else {
    if (p.plan.S > 1)
      hipLaunchKernelGGL((recur_fwd_kernel<IO, 64, 4, REV, false, true>), grid_of(rows * (p.plan.S - 1)), dim3(256), 0, s, p);
    hipLaunchKernelGGL((recur_fwd_kernel<IO, 64, 4, REV, Z, false>), grid_of(rows * p.plan.S), dim3(256), 0, s, p);
  }
}

template <typename IO>
void any(const RecurParams& p, bool reverse, hipStream_t s) {
  if (reverse) p.z ? go<IO, true, true>(p, s) : go<IO, true, false>(p, s);
  else p.z ? go<IO, false, true>(p, s) : go<IO, false, false>(p, s);
}

template <typename IO>
void step(const RecurStepParams& p, hipStream_t s) {
  const dim3 grid = grid_of(((p.n + 3) / 4 + 255) / 256);
  if (p.D % 4) hipLaunchKernelGGL((recur_step_kernel<IO, false>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((recur_step_kernel<IO, true>), grid, dim3(256), 0, s, p);
}

}  // namespace

hipError_t launch_recur_fwd(const RecurParams& p, bool bf16, bool reverse, hipStream_t s) {
  bf16 ? any<bf16_t>(p, reverse, s) : any<float>(p, reverse, s);
  return hipGetLastError();
}

hipError_t launch_recur_step(const RecurStepParams& p, bool bf16, hipStream_t s) {
  bf16 ? step<bf16_t>(p, s) : step<float>(p, s);
  return hipGetLastError();
}

}  // namespace ssm
