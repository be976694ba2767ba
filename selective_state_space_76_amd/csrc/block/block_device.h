// block_device.h -- what the residual block's kernels share: the dropout mask, masked pieces.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../ssm_device.h"
#include "../train/train_device.h"
#include "block_launch.h"

namespace ssm {

// The mask of elements 8 j .. 8 j + 7 (numbered in memory order) are the four words of Philox4x32 with ten rounds
// (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3; SC 2011) for the counter (j, call) and the
// key `seed`, 16 bits an element: about 15 instructions an element, under the 30 that an element of a bf16 stream
// may take at the rate of the memory; with 32 bits an element it would be the other way round.
struct Drop {
  uint32_t key[2], call[2], below;
  float scale;
  __device__ __forceinline__ Drop(const DropParams& p) {
    uint64_t seed = p.seed;
    if (p.below && p.device_seed) seed = (uint64_t)*p.device_seed;
    key[0] = (uint32_t)seed;
    key[1] = (uint32_t)(seed >> 32);
    call[0] = (uint32_t)p.call;
    call[1] = (uint32_t)(p.call >> 32);
    below = p.below;
    scale = p.scale;
  }
  __device__ __forceinline__ bool any() const { return below != 0; }

  __device__ __forceinline__ void words(uint64_t j, uint32_t (&w)[4]) const {
    uint32_t c0 = (uint32_t)j, c1 = (uint32_t)(j >> 32), c2 = call[0], c3 = call[1], k0 = key[0], k1 = key[1];
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
      c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
      c1 = (uint32_t)b;
      c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
      c3 = (uint32_t)a;
      k0 += 0x9E3779B9u;
      k1 += 0xBB67AE85u;
    }
    w[0] = c0;
    w[1] = c1;
    w[2] = c2;
    w[3] = c3;
  }

  // bit e: element i + e is kept; i is any element's number
  __device__ __forceinline__ uint32_t kept(uint64_t i) const {
    const int at = (int)(i & 7);
    uint32_t w[4];
    words(i >> 3, w);
    if (at) {
      uint32_t v[8], next[4];
      words((i >> 3) + 1, next);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = w[k];
        v[4 + k] = next[k];
      }
      // moved down by `at` halves: by masks, so that the words stay in registers
      const uint32_t four = at & 4 ? ~0u : 0u, two = at & 2 ? ~0u : 0u, one = at & 1 ? ~0u : 0u;
#pragma unroll
      for (int k = 0; k < 6; ++k) v[k] = (v[k + 2] & four) | (v[k] & ~four);  // (v[6], v[7]: not looked at from here on)
#pragma unroll
      for (int k = 0; k < 5; ++k) v[k] = (v[k + 1] & two) | (v[k] & ~two);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = ((v[k] >> 16 | v[k + 1] << 16) & one) | (v[k] & ~one);
    }
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m |= ((e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu) >= below ? 1u : 0u) << e;
    return m;
  }
  // A dropped element is zero whatever it was, infinities and NaN included.
  __device__ __forceinline__ void apply(uint32_t kept, float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = kept >> e & 1u ? x[e] * scale : 0.0f;
  }
};

// What of a piece of 8 exists: its elements lo .. hi - 1.
struct Part {
  int lo, hi;
  // of n elements, the 8 from i on
  __device__ __forceinline__ Part(int64_t i, int64_t n)
      : lo(i < 0 ? (int)-i : 0), hi(n - i >= 8 ? 8 : n - i > 0 ? (int)(n - i) : 0) {}
  __device__ __forceinline__ Part() : lo(0), hi(0) {}
  __device__ __forceinline__ bool whole() const { return hi - lo == 8; }
  __device__ __forceinline__ bool any() const { return lo < hi; }
  __device__ __forceinline__ bool has(int k) const { return k >= lo && k < hi; }
};

// A sum of very many terms: what an addition rounds away goes in with the next one (compensated summation, Kahan 1965), or
// it would add up with their number where they have one sign: a plain chain of 2^14 equal terms is off by up to 1.7e-4.
// Sums that have overflowed stay infinite.
struct LongSum {
  float s = 0.0f, c = 0.0f;
  __device__ __forceinline__ void add(float v) {
    const float y = v + c, t = s + y, rest = y - (t - s);
    c = __builtin_isfinite(t) ? rest : 0.0f;
    s = t;
  }
  __device__ __forceinline__ float value() const { return s + c; }
};

// 8 elements as they lie in memory, from any element on.  Loads of several pieces are to be in flight together, so
// a piece begins as zeros, full() asks for all 8 where it may and does not wait, and part() reads what is left of one
// that goes over the end of its tensor, when all others have been asked for.
template <typename IO>
struct Piece {
  static constexpr int Q = (int)sizeof(IO) / 2;  // 16-byte words
  u32x4a w[Q];
  // again: it is to be read again (and is left to the caches)
  __device__ __forceinline__ void full(const IO* p, bool may, bool again = false) {
#pragma unroll
    for (int k = 0; k < Q; ++k) w[k] = u32x4a{0u, 0u, 0u, 0u};
    if (may) {
#pragma unroll
      for (int k = 0; k < Q; ++k) {
        const auto* a = reinterpret_cast<const typename Unaligned<IO>::type*>(p) + k;
        // (of two words of one line the first must not drop it)
        const auto q = Q == 1 && !again ? __builtin_nontemporal_load(a) : *a;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[k][i] = q[i];
      }
    }
  }
  // the elements lo .. hi - 1 (one at least) of the piece at p, in one go: the others repeat the nearest
  __device__ __forceinline__ void part(const IO* p, const Part& r) {
    IO v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = p[e < r.lo ? r.lo : e < r.hi ? e : r.hi - 1];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (Q == 1) w[0][e >> 1] = (e & 1 ? w[0][e >> 1] & 0xffffu : 0u) | (uint32_t)v[e] << (16 * (e & 1));
      else w[e >> 2][e & 3] = __float_as_uint(v[e]);
    }
  }
  // zeros for what does not exist
  __device__ __forceinline__ void cut(const Part& r) {
#pragma unroll
    for (int k = 0; k < 4 * Q; ++k) {
      if constexpr (Q == 1)
        w[0][k] &= (r.has(2 * k) ? 0xffffu : 0u) | (r.has(2 * k + 1) ? 0xffff0000u : 0u);
      else w[k >> 2][k & 3] = r.has(k) ? w[k >> 2][k & 3] : 0u;
    }
  }
  // zeros where the bit is not set
  __device__ __forceinline__ void keep(uint32_t kept) {
#pragma unroll
    for (int k = 0; k < 4 * Q; ++k) {
      if constexpr (Q == 1)
        w[0][k] &= (kept >> (2 * k) & 1u ? 0xffffu : 0u) | (kept >> (2 * k + 1) & 1u ? 0xffff0000u : 0u);
      else w[k >> 2][k & 3] = kept >> k & 1u ? w[k >> 2][k & 3] : 0u;
    }
  }
  // Keeps the compiler from holding what it has made of the piece (twice the registers) for a later pass.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int k = 0; k < Q; ++k) asm volatile("" : "+v"(w[k]));
  }
  __device__ __forceinline__ float at(int e) const {
    if constexpr (Q == 1) return __uint_as_float(e & 1 ? w[0][e >> 1] & 0xffff0000u : w[0][e >> 1] << 16);
    else return __uint_as_float(w[e >> 2][e & 3]);
  }
};

template <typename IO>
__device__ __forceinline__ void store_part(IO* p, const Part& r, const float (&x)[8]) {
  if (r.whole()) {
    store_n<IO, 8>(p, 8, x);
  } else if (r.any()) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (r.has(e)) store_io(p + e, x[e]);
  }
}

}  // namespace ssm
