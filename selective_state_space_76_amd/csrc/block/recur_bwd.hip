// recur_bwd.hip -- gradients of the gated linear recurrence (recur_fwd.hip).
//
//   G[t] = dout silu(z) + F[t+1],  F[t] = a[t] G[t]  (F behind the last step: the final state's gradient)
//   dx = G q sig(i);  di = G q x sig(i) (1 - sig(i));  dz = dout h silu'(z);  d(initial state) = F[0]
//   dla = G (a h[t-1] - sig(i) x a^2 / q);  dr = -decay dla sig(r) (1 - sig(r));  ddecay = -sum dla sig(r)
//   drb = sum dr;  dib = sum di
//
// Bound by HBM: x, r, i, dout (and z) are read once, their gradients written once (14 or 18 bytes a step in bf16).  The
// states are made again from the checkpoints of the forward pass, one for every 64 pieces, so that a wave needs no
// other's; the adjoint F is an affine recurrence against time, walked as the forward pass walks the states (teams of
// waves through LDS, segments for few rows).  ddecay and the biases' gradients are summed per wave and joined in a fixed
// order (join.hip), or at once where a channel is one team's (1 x 509 x 262147: 401 -> 391 us).
// 8 x 1536 x 2048: 98 us a call, 18 bytes a step, 4.6 TB/s; workgroups of 8 waves instead of 4 take 112, and 123 where
// they are the rows of a channel, whose sums then need no second kernel.
#include "recur_device.h"

namespace ssm {

// Z: there is a gate.  MAPS: the segments' maps of the adjoint.  PARTS: a segment leaves several partial sums, of turns that
// are summed by themselves (apart from the others for its registers: 1 x 509 x 262147 394 us, 405 with it; 1 x 100 x 200000
// in reverse 136 and 147).
template <typename IO, int LN, int W, bool REV, bool Z, bool MAPS, bool PARTS = false>
__global__ __launch_bounds__(W > 4 ? W * 64 : 256, Z || (REV && PARTS) || LN < 64 ? 3 : 4)
void recur_bwd_kernel(RecurParams p) {
  constexpr int V = 16 / (int)sizeof(IO);
  constexpr int UNITS = W > 4 ? 1 : 256 / (LN * W);
  constexpr int TURN = LN * W * V;
  __shared__ float sm[2][W][2];
  const int lane = threadIdx.x % LN, w = W > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / 64) : 0;
  const int64_t S = MAPS ? p.plan.S - 1 : p.plan.S;
  const int64_t rows = p.B * p.D, total = rows * p.L;
  int64_t unit = (int64_t)block_id() * UNITS + (W > 1 ? 0 : threadIdx.x / LN);
  if (unit >= rows * S) return;
  if (W > 1 || LN == 64) unit = __builtin_amdgcn_readfirstlane((int)unit);
  const int64_t row = unit / S, seg = unit - row * S + (MAPS ? 1 : 0);  // (the first segment's map is not needed)
  const int64_t b = row / p.D, d = row - b * p.D;
  const Row<IO, REV> line(row, p.L);
  const Channel ch(p.decay, p.rb, p.ib, d);
  const float decay = p.decay[d];
  const int64_t k0 = seg * p.plan.per, k1 = k0 + p.plan.per < p.plan.tiles ? k0 + p.plan.per : p.plan.tiles;

  float carry = 0.0f, whole = 1.0f;
  if (!MAPS) {
    carry = p.dlast ? p.dlast[row] : 0.0f;
    if (p.plan.S > 1) {  // the segments behind, one a lane
      const int l = threadIdx.x & 63;
      float A = 1.0f, B = 0.0f;
      if (l > seg && l < p.plan.S) {
        A = p.seg[(l * rows + row) * 2];
        B = p.seg[(l * rows + row) * 2 + 1];
      }
      scan_down<64>(A, B);
      carry = __builtin_fmaf(lane_of(A, 0), carry, lane_of(B, 0));
    }
  }

  const u32x4a none = {0u, 0u, 0u, 0u};
  u32x4a xn = none, rn = none, in = none, zn = none, gn = none;
  float hn = 0.0f;
  auto load = [&](int64_t tile) {
    const int64_t s = tile * TURN + (w * LN + lane) * V, at = line.at(s);
    const int lo = line.lo(s), hi = line.hi(s);
    const bool edge = line.edge(tile * TURN, TURN);
    rn = load_slots<IO, REV>(p.r, at, lo, hi, edge, total);
    gn = load_slots<IO, REV>(p.dout, at, lo, hi, edge, total);
    if (Z) zn = load_slots<IO, REV>(p.z, at, lo, hi, edge, total);
    if (!MAPS) {
      xn = load_slots<IO, REV>(p.x, at, lo, hi, edge, total);
      in = load_slots<IO, REV>(p.i, at, lo, hi, edge, total);
      const int64_t block = tile * W + w;
      hn = p.ckpt[row * p.plan.blocks + (block < p.plan.blocks ? block : p.plan.blocks - 1)];
    }
  };
  // The lane's sums, of p.plan.chain turns (127 at the most): then they become a partial sum.  (A plain chain of 2^14 terms
  // of one sign was off by 5e-5; compensated in registers or LDS the sums cost long rows up to 9 and 28%.)
  float sd = 0.0f, sr = 0.0f, si = 0.0f;
  int left = p.plan.chain, parts = 0;
  auto part = [&] { return p.part + (((b * p.plan.S + seg) * W + w) * (PARTS ? p.plan.parts : 1) + parts) * 3 * p.D + d; };
  float state = 0.0f;
  if (k0 < k1) load(k1 - 1);
  for (int64_t tile = k1 - 1; tile >= k0; --tile) {
    const u32x4a xq = xn, rq = rn, uq = in, zq = zn, gq = gn;
    state = hn;
    if (LN == 64 && tile > k0) load(tile - 1);
    const int64_t s = tile * TURN + (w * LN + lane) * V;
    const int lo = line.lo(s), hi = line.hi(s);
    const bool edge = line.edge(tile * TURN, TURN);
    float a[V], v[V], g[V], sig[V], sgi[V], q[V], iq[V], sz[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const Gates k(slot<IO, REV>(rq, e), slot<IO, REV>(uq, e), ch);
      a[e] = k.a;
      sig[e] = k.sr;
      sgi[e] = k.si;
      q[e] = k.q;
      iq[e] = k.iq;
      v[e] = k.q * k.si * slot<IO, REV>(xq, e);
      g[e] = slot<IO, REV>(gq, e);
      if (Z) {
        const float z = slot<IO, REV>(zq, e);
        sz[e] = sigmoid_(z);
        g[e] *= z * sz[e];
      }
    }
    if (edge) {  // the identity where there is no step, and nothing that would add to the sums
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const bool step = e >= lo && e < hi;
        a[e] = step ? a[e] : 1.0f;
        v[e] = step ? v[e] : 0.0f;
        g[e] = step ? g[e] : 0.0f;
      }
    }
    float A = a[0], B = v[0], FA = 1.0f, FB = 0.0f;
#pragma unroll
    for (int e = 1; e < V; ++e) {
      A *= a[e];
      B = __builtin_fmaf(a[e], B, v[e]);
    }
#pragma unroll
    for (int e = V - 1; e >= 0; --e) FB = a[e] * (g[e] + FB);
    FA = A;
    scan_down<LN>(FA, FB);
    const float ta = end_lane<LN, false>(FA), tb = end_lane<LN, false>(FB);
    float behind = carry;
    if constexpr (W == 1) {
      carry = __builtin_fmaf(ta, carry, tb);
      whole *= ta;
    } else {
      float (*to)[2] = sm[tile & 1];
      if ((threadIdx.x & 63) == 0) {
        to[w][0] = ta;
        to[w][1] = tb;
      }
      __syncthreads();
#pragma unroll
      for (int k = W - 1; k >= 0; --k) {
        if (k == w) behind = carry;
        carry = __builtin_fmaf(to[k][0], carry, to[k][1]);
        whole *= to[k][0];
      }
    }
    if (MAPS) continue;

    // the states: hb before each step
    scan_up<LN>(A, B);
    float h = __builtin_fmaf(lane_before<LN>(A, 1.0f), state, lane_before<LN>(B, 0.0f));
    const int64_t at = line.at(s);
    float hb[V], o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      hb[e] = h;
      h = __builtin_fmaf(a[e], h, v[e]);
      if (Z) {
        const float z = slot<IO, REV>(zq, e);
        o[e] = slot<IO, REV>(gq, e) * h * (sz[e] * __builtin_fmaf(z, 1.0f - sz[e], 1.0f));
      }
    }
    if (Z) store_slots<IO, REV>(p.dz, at, lo, hi, edge, o);
    // the adjoint: G in g's place
    float F = __builtin_fmaf(lane_behind<LN>(FA, 1.0f), behind, lane_behind<LN>(FB, 0.0f));
#pragma unroll
    for (int e = V - 1; e >= 0; --e) {
      g[e] += F;
      F = a[e] * g[e];
    }
    if (edge) {
#pragma unroll
      for (int e = 0; e < V; ++e) g[e] = e >= lo && e < hi ? g[e] : 0.0f;
    }
    // (gradients with respect to what the sigmoids take; where a is 1 to the last bit, with sig(r) under 2^-100 / decay,
    // what 1 / q meets is zero)
    float td = PARTS ? 0.0f : sd, tr = PARTS ? 0.0f : sr, ti = PARTS ? 0.0f : si;  // the turn's
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float gs = g[e] * sgi[e], x = slot<IO, REV>(xq, e);
      const float dla = __builtin_fmaf(g[e] * a[e], hb[e], -gs * x * (a[e] * a[e] * iq[e]));
      const float dls = -dla * sig[e];
      td += dls;
      hb[e] = dls * decay * (1.0f - sig[e]);
      tr += hb[e];
      o[e] = gs * q[e];
      g[e] = o[e] * x * (1.0f - sgi[e]);
      ti += g[e];
    }
    sd = PARTS ? sd + td : td;
    sr = PARTS ? sr + tr : tr;
    si = PARTS ? si + ti : ti;
    store_slots<IO, REV>(p.dx, at, lo, hi, edge, o);
    store_slots<IO, REV>(p.dr, at, lo, hi, edge, hb);
    store_slots<IO, REV>(p.di, at, lo, hi, edge, g);
    if (LN < 64) break;  // (rows of fewer lanes are one turn)
    if (PARTS && --left == 0 && tile > k0) {
      sd = sum_group<LN>(sd);
      sr = sum_group<LN>(sr);
      si = sum_group<LN>(si);
      if (lane == 0) {
        float* o = part();
        o[0] = sd;
        o[p.D] = sr;
        o[2 * p.D] = si;
      }
      sd = sr = si = 0.0f;
      left = p.plan.chain;
      ++parts;
    }
  }
  if (MAPS) {
    if (lane == 0 && w == 0) {
      p.seg[(seg * rows + row) * 2] = whole;
      p.seg[(seg * rows + row) * 2 + 1] = carry;
    }
    return;
  }
  if (p.dinit && seg == 0 && lane == 0 && w == 0) p.dinit[row] = carry;
  sd = sum_group<LN>(sd);
  sr = sum_group<LN>(sr);
  si = sum_group<LN>(si);
  if (p.whole) {
    if constexpr (W > 1) {
      __shared__ float all[W][3];
      if (lane == 0) {
        all[w][0] = sd;
        all[w][1] = sr;
        all[w][2] = si;
      }
      __syncthreads();
      if (w) return;
      sd = sr = si = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        sd += all[k][0];
        sr += all[k][1];
        si += all[k][2];
      }
    }
    if (lane == 0) {
      if (p.ddecay) p.ddecay[d] = sd;
      if (p.drb) p.drb[d] = sr;
      if (p.dib) p.dib[d] = si;
    }
  } else if (lane == 0) {
    for (; parts < (PARTS ? p.plan.parts : 1); ++parts) {  // (a last segment may have fewer turns)
      float* o = part();
      o[0] = sd;
      o[p.D] = sr;
      o[2 * p.D] = si;
      sd = sr = si = 0.0f;
    }
  }
}

namespace {

template <typename IO, bool REV, bool Z, bool PARTS>
void waves(const RecurParams& p, hipStream_t s) {
  const int64_t rows = p.B * p.D;
  if (p.plan.waves == 1)
    hipLaunchKernelGGL((recur_bwd_kernel<IO, 64, 1, REV, Z, false, PARTS>), grid_of((rows + 3) / 4), dim3(256), 0, s, p);
  else if (p.plan.waves == 8)
    hipLaunchKernelGGL((recur_bwd_kernel<IO, 64, 8, REV, Z, false, PARTS>), grid_of(rows), dim3(512), 0, s, p);
  else
    hipLaunchKernelGGL((recur_bwd_kernel<IO, 64, 4, REV, Z, false, PARTS>), grid_of(rows * p.plan.S), dim3(256), 0, s, p);
}

template <typename IO, bool REV, bool Z>
void go(const RecurParams& p, hipStream_t s) {
  const int64_t rows = p.B * p.D;
  auto few = [&](auto lanes) {
    constexpr int LN = decltype(lanes)::value, ROWS = 256 / LN;
    hipLaunchKernelGGL((recur_bwd_kernel<IO, LN, 1, REV, Z, false>), grid_of((rows + ROWS - 1) / ROWS), dim3(256), 0, s, p);
  };
  if (p.plan.lanes < 64) {
    p.plan.lanes == 1 ? few(IC<1>()) : p.plan.lanes == 4 ? few(IC<4>()) : p.plan.lanes == 16 ? few(IC<16>()) : few(IC<32>());
  } else {
    if (p.plan.S > 1)
      hipLaunchKernelGGL((recur_bwd_kernel<IO, 64, 4, REV, Z, true>), grid_of(rows * (p.plan.S - 1)), dim3(256), 0, s, p);
    p.plan.parts > 1 ? waves<IO, REV, Z, true>(p, s) : waves<IO, REV, Z, false>(p, s);
  }
}

template <typename IO>
void any(const RecurParams& p, bool reverse, hipStream_t s) {
  if (reverse) p.z ? go<IO, true, true>(p, s) : go<IO, true, false>(p, s);
  else p.z ? go<IO, false, true>(p, s) : go<IO, false, false>(p, s);
}

}  // namespace

hipError_t launch_recur_bwd(const RecurParams& q, bool bf16, bool reverse, hipStream_t s) {
  RecurParams p = q;
  p.whole = p.B == 1 && p.plan.S == 1 && p.plan.parts == 1;
  bf16 ? any<bf16_t>(p, reverse, s) : any<float>(p, reverse, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.whole) return e;
  return launch_join({p.part, p.B * p.plan.S * p.plan.waves * p.plan.parts, p.D, 3, {p.ddecay, p.drb, p.dib}}, s);
}

}  // namespace ssm
