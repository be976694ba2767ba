// recur_device.h -- the gated linear recurrence: its gates, its layout in pieces, scans of affine maps over lanes.
//
//   a = exp(-decay sig(r + rb));  q = sqrt(1 - a^2);  v = q sig(i + ib) x;  h[t] = a[t] h[t-1] + v[t]
//   out = h, or h silu(z)
//
// Pieces.  A lane holds V = 16 / sizeof(IO) steps at a time, the 16 bytes at an address that is a multiple of 16, whatever
// element the row begins at: the row's steps are slots m .. m + L - 1 of its pieces, where m is what the row begins
// behind such an address.  In reverse, slots count from the row's end, and a piece's elements are turned round.  Slots
// that are no steps are the identity (a = 1, v = 0).  64 pieces are a block, whose first slot has a checkpoint.
#pragma once
#include "block_device.h"

namespace ssm {

// ---------------------------------------------------------------- affine maps f(h) = A h + B, composed over lanes

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or(float v, float other) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)__float_as_uint(other), (int)__float_as_uint(v), CTRL,
                                                               ROWS, 0xf, false));
}
__device__ __forceinline__ float lane_of(float v, int l) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), l));
}

// Groups of LN = 1, 4, 16, 32 or 64 lanes.

// the value of the lane that CTRL names, or `other` where that lane is not of the group
template <int CTRL>
__device__ __forceinline__ float quad_or(float v, float other, bool has) {
  const float q = __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
  return has ? q : other;
}

// The lane's map after those of the lanes before it.
template <int LN>
__device__ __forceinline__ void scan_up(float& A, float& B) {
  if constexpr (LN == 1) return;
  if constexpr (LN == 4) {
    auto quad = [&](auto ctrl, int by) {
      const bool has = (int)(threadIdx.x & 3) >= by;
      const float a = quad_or<decltype(ctrl)::value>(A, 1.0f, has), b = quad_or<decltype(ctrl)::value>(B, 0.0f, has);
      B = __builtin_fmaf(A, b, B);
      A *= a;
    };
    quad(IC<0x90>{}, 1);  // [0,0,1,2]
    quad(IC<0x40>{}, 2);  // [0,0,0,1]
    return;
  }
  auto step = [&](auto ctrl, auto rows) {
    const float a = dpp_or<decltype(ctrl)::value, decltype(rows)::value>(A, 1.0f);
    const float b = dpp_or<decltype(ctrl)::value, decltype(rows)::value>(B, 0.0f);
    B = __builtin_fmaf(A, b, B);
    A *= a;
  };
  step(IC<0x111>{}, IC<0xf>{});  // row_shr:1, 2, 4, 8
  step(IC<0x112>{}, IC<0xf>{});
  step(IC<0x114>{}, IC<0xf>{});
  step(IC<0x118>{}, IC<0xf>{});
  if constexpr (LN >= 32) step(IC<0x142>{}, IC<0xa>{});  // row_bcast:15 into rows 1 and 3
  if constexpr (LN == 64) step(IC<0x143>{}, IC<0xc>{});  // row_bcast:31 into rows 2 and 3
}

// The lane's map after those of the lanes behind it.
template <int LN>
__device__ __forceinline__ void scan_down(float& A, float& B) {
  if constexpr (LN == 1) return;
  if constexpr (LN == 4) {
    auto quad = [&](auto ctrl, int by) {
      const bool has = (int)(threadIdx.x & 3) + by < 4;
      const float a = quad_or<decltype(ctrl)::value>(A, 1.0f, has), b = quad_or<decltype(ctrl)::value>(B, 0.0f, has);
      B = __builtin_fmaf(A, b, B);
      A *= a;
    };
    quad(IC<0xf9>{}, 1);  // [1,2,3,3]
    quad(IC<0xfe>{}, 2);  // [2,3,3,3]
    return;
  }
  auto step = [&](auto ctrl) {
    const float a = dpp_or<decltype(ctrl)::value, 0xf>(A, 1.0f);
    const float b = dpp_or<decltype(ctrl)::value, 0xf>(B, 0.0f);
    B = __builtin_fmaf(A, b, B);
    A *= a;
  };
  step(IC<0x101>{});  // row_shl:1, 2, 4, 8
  step(IC<0x102>{});
  step(IC<0x104>{});
  step(IC<0x108>{});
  if constexpr (LN == 32) {  // the row behind: its first lane holds its whole map
    const float a3 = lane_of(A, 48), b3 = lane_of(B, 48), a1 = lane_of(A, 16), b1 = lane_of(B, 16);
    const int row = (threadIdx.x & 63) >> 4;
    const float a = row == 0 ? a1 : row == 2 ? a3 : 1.0f, b = row == 0 ? b1 : row == 2 ? b3 : 0.0f;
    B = __builtin_fmaf(A, b, B);
    A *= a;
  }
  if constexpr (LN == 64) {  // the rows behind
    const float a3 = lane_of(A, 48), b3 = lane_of(B, 48);
    const float a2 = lane_of(A, 32), b2 = lane_of(B, 32);
    const float a1 = lane_of(A, 16), b1 = lane_of(B, 16);
    const float a23 = a2 * a3, b23 = __builtin_fmaf(a2, b3, b2);
    const float a123 = a1 * a23, b123 = __builtin_fmaf(a1, b23, b1);
    const int row = (threadIdx.x & 63) >> 4;
    const float a = row == 0 ? a123 : row == 1 ? a23 : row == 2 ? a3 : 1.0f;
    const float b = row == 0 ? b123 : row == 1 ? b23 : row == 2 ? b3 : 0.0f;
    B = __builtin_fmaf(A, b, B);
    A *= a;
  }
}

// the value of the lane before (behind) in the group of LN; the first (last) gets `end`
template <int LN> __device__ __forceinline__ float lane_before(float v, float end) {
  if constexpr (LN == 1) return end;
  else if constexpr (LN == 4) return quad_or<0x90>(v, end, threadIdx.x & 3);
  else if constexpr (LN == 16) return dpp_or<0x111, 0xf>(v, end);
  else {
    const float q = dpp_or<0x138, 0xf>(v, end);
    return LN == 64 || (threadIdx.x & 31) ? q : end;
  }
}
template <int LN> __device__ __forceinline__ float lane_behind(float v, float end) {
  if constexpr (LN == 1) return end;
  else if constexpr (LN == 4) return quad_or<0xf9>(v, end, (threadIdx.x & 3) < 3);
  else if constexpr (LN == 16) return dpp_or<0x101, 0xf>(v, end);
  else {
    const float q = dpp_or<0x130, 0xf>(v, end);
    return LN == 64 || (threadIdx.x & 31) < 31 ? q : end;
  }
}
// the group's first or last lane's value, in all of its lanes
template <int LN, bool LAST> __device__ __forceinline__ float end_lane(float v) {
  if constexpr (LN == 1) return v;
  else if constexpr (LN == 4) return quad_or<LAST ? 0xff : 0x00>(v, 0.0f, true);
  else if constexpr (LN == 16) return quad_or<LAST ? 0x15f : 0x150>(v, 0.0f, true);  // (row_newbcast)
  else if constexpr (LN == 32) {
    const float a = lane_of(v, LAST ? 31 : 0), b = lane_of(v, LAST ? 63 : 32);
    return threadIdx.x & 32 ? b : a;
  }
  else return lane_of(v, LAST ? 63 : 0);
}
// summed over the group, in its first lane
template <int LN> __device__ __forceinline__ float sum_group(float v) {
  if constexpr (LN == 1) return v;
  else if constexpr (LN == 4) {
    v += quad_or<0xb1>(v, 0.0f, true);
    return v + quad_or<0x4e>(v, 0.0f, true);
  }
  else if constexpr (LN == 32) {
    v = sum_lanes<16>(v);
    return v + __shfl_xor(v, 16);
  }
  else return sum_lanes<LN>(v);
}

// ---------------------------------------------------------------- pieces

// one row's pieces
template <typename IO, bool REV>
struct Row {
  static constexpr int V = 16 / (int)sizeof(IO);
  int64_t m;       // slots before the first step
  int64_t slots;   // m + L
  int64_t origin;  // the first slot's element number in the tensor (REV: the one behind it)
  __device__ __forceinline__ Row(int64_t row, int64_t L) {
    const int64_t at = row * L, past = at + L;
    m = REV ? (V - past % V) % V : at % V;
    slots = m + L;
    origin = REV ? past + m : at - m;
  }
  // element number of the piece that begins at slot s (a multiple of V)
  __device__ __forceinline__ int64_t at(int64_t s) const { return REV ? origin - s - V : origin + s; }
  // whether slots s .. s + n - 1 are not all steps
  __device__ __forceinline__ bool edge(int64_t s, int64_t n) const { return s < m || s + n > slots; }
  // its slots that are steps: lo .. hi - 1
  __device__ __forceinline__ int lo(int64_t s) const { return s >= m ? 0 : (int)(m - s < V ? m - s : V); }
  __device__ __forceinline__ int hi(int64_t s) const { return slots - s >= V ? V : slots > s ? (int)(slots - s) : 0; }
};

// 16 bytes of which the slots lo .. hi - 1 are read, the others zero.  edge: there are others in this turn of the team
// (the same in all its lanes).  What lies there belongs to the neighbouring rows, or to nothing behind the tensor's end
// (total), and only there the elements are read one by one (8 x 1536 x 2047: 63 us, 78 with
// every such piece read so; its gradients 120 and 157).
template <typename IO, bool REV>
__device__ __forceinline__ u32x4a load_slots(const void* p, int64_t at, int lo, int hi, bool edge, int64_t total) {
  constexpr int V = 16 / (int)sizeof(IO);
  const IO* q = static_cast<const IO*>(p) + at;
  if (!edge) return __builtin_nontemporal_load(reinterpret_cast<const u32x4a*>(q));
  u32x4a w = {0u, 0u, 0u, 0u};
  if (lo >= hi) return w;
  const int first = REV ? V - hi : lo, last = REV ? V - lo : hi;  // in the order of memory
  if (at + V <= total) {
    w = *reinterpret_cast<const u32x4a*>(q);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (V == 8)
        w[k] &= (2 * k >= first && 2 * k < last ? 0xffffu : 0u) | (2 * k + 1 >= first && 2 * k + 1 < last ? 0xffff0000u : 0u);
      else w[k] = k >= first && k < last ? w[k] : 0u;
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (k >= first && k < last) {
        if constexpr (V == 8) w[k >> 1] |= (uint32_t)q[k] << (16 * (k & 1));
        else w[k] = __float_as_uint(q[k]);
      }
    }
  }
  return w;
}

template <typename IO, bool REV>
__device__ __forceinline__ float slot(const u32x4a& w, int s) {
  constexpr int V = 16 / (int)sizeof(IO);
  const int k = REV ? V - 1 - s : s;
  if constexpr (V == 8) return __uint_as_float(k & 1 ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16);
  else return __uint_as_float(w[k]);
}

template <typename IO, bool REV, int V>
__device__ __forceinline__ void store_slots(void* p, int64_t at, int lo, int hi, bool edge, const float (&x)[V]) {
  IO* q = static_cast<IO*>(p) + at;
  if (!edge || (lo == 0 && hi == V)) {
    u32x4a w;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (V == 8) {
        const float a = x[REV ? 7 - 2 * k : 2 * k], b = x[REV ? 6 - 2 * k : 2 * k + 1];
        w[k] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)a) | (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)b) << 16;
      } else {
        w[k] = __float_as_uint(x[REV ? 3 - k : k]);
      }
    }
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4a*>(q));
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int s = REV ? V - 1 - k : k;
      if (s >= lo && s < hi) store_io(q + k, x[s]);
    }
  }
}

// ---------------------------------------------------------------- gates

__device__ __forceinline__ float sigmoid_(float x) { return rcp_(1.0f + exp2_(-x * kLog2e)); }

// a channel's numbers: -log2(e) of the decay (NaN for a negative one) and the biases
struct Channel {
  float nd, rb, ib;
  __device__ __forceinline__ Channel(float decay, float r_bias, float i_bias)
      : nd(decay >= 0.0f ? -kLog2e * decay : __builtin_nanf("")), rb(-kLog2e * r_bias), ib(-kLog2e * i_bias) {}
  __device__ __forceinline__ Channel(const float* decay, const float* r_bias, const float* i_bias, int64_t d)
      : Channel(decay[d], r_bias ? r_bias[d] : 0.0f, i_bias ? i_bias[d] : 0.0f) {}
};

// a step's gates; q = sqrt(1 - a^2), iq = 1 / q (of 2^-100 where 1 - a^2 is less)
struct Gates {
  float sr, si, a, q, iq;
  // 1 - a^2 = 1 - e^-t with t = 2 decay sr: up to t = 1/4 from the series to t^6 (the next term is under 5e-8 of it), where
  // a^2 is near 1 and the difference would lose its bits; above it the difference, off by under 6e-7 of itself.
  __device__ __forceinline__ Gates(float r, float i, const Channel& c) {
    sr = rcp_(1.0f + exp2_(__builtin_fmaf(r, -kLog2e, c.rb)));
    si = rcp_(1.0f + exp2_(__builtin_fmaf(i, -kLog2e, c.ib)));
    const float y = sr * c.nd;  // log2 of a
    a = exp2_(y);
    const float t = y * (-2.0f * kLn2);
    float s = __builtin_fmaf(t, -1.0f / 720, 1.0f / 120);
    s = __builtin_fmaf(t, s, -1.0f / 24);
    s = __builtin_fmaf(t, s, 1.0f / 6);
    s = __builtin_fmaf(t, s, -0.5f);
    s = __builtin_fmaf(t, s, 1.0f);
    const float w = t < 0.25f ? t * s : __builtin_fmaf(-a, a, 1.0f);
    iq = __builtin_amdgcn_rsqf(fmaxf(w, 7.888609e-31f));
    q = w * iq;
  }
};

}  // namespace ssm
