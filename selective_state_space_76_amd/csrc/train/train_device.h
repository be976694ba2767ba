// train_device.h -- what the training operators' kernels share: pieces of rows at any alignment, and tokens.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../ssm_device.h"
#include "train_launch.h"

namespace ssm {

typedef uint32_t u32x4a __attribute__((ext_vector_type(4)));

// the workgroup's number in a grid_of() grid (a second row of which there is only behind a full one)
__device__ __forceinline__ uint32_t block_id() { return blockIdx.y * (uint32_t)kGridX + blockIdx.x; }

// 16 bytes that begin at any element
template <typename IO> struct Unaligned;
template <> struct Unaligned<float> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4))); };
template <> struct Unaligned<bf16_t> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2))); };

// the row that position t names, or V (no row) for a token outside the table
__device__ __forceinline__ int64_t token_at(const void* tokens, int i64, int64_t t, int64_t V) {
  const int64_t k = i64 ? static_cast<const int64_t*>(tokens)[t] : (int64_t)static_cast<const int32_t*>(tokens)[t];
  return k >= 0 && k < V ? k : V;
}

// N elements from p, of which the first n exist (the others are zero); NT: they are not needed again
template <typename IO, int N, bool NT = false>
__device__ __forceinline__ void load_n(const IO* p, int n, float (&x)[N]) {
  constexpr int V = 16 / (int)sizeof(IO);
  if (n == N && N % V == 0) {
#pragma unroll
    for (int k = 0; k < N / V; ++k) {
      const auto* a = reinterpret_cast<const typename Unaligned<IO>::type*>(p + k * V);
      // (of two pieces of one line the first must not drop it)
      const auto q = NT && N == V ? __builtin_nontemporal_load(a) : *a;
      if constexpr (V == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[k * V + 2 * i] = __uint_as_float(q[i] << 16);
          x[k * V + 2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[k * V + i] = __uint_as_float(q[i]);
      }
    }
  } else if (n == N && N == 4 && V == 8) {
    typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(2)));
    const auto* a = reinterpret_cast<const u32x2u*>(p);
    const auto q = NT ? __builtin_nontemporal_load(a) : *a;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[2 * i] = __uint_as_float(q[i] << 16);
      x[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = i < n ? to_f32(p[i]) : 0.0f;
  }
}

// The same, kept as they are in memory (half the registers of floats for bf16) until at().
template <typename IO, int N, bool NT = true>
struct Raw {
  static constexpr int W = N * (int)sizeof(IO) / 4, C = W < 4 ? W : 4;  // words, and of one piece
  uint32_t w[W];
  __device__ __forceinline__ void load(const IO* p, int n) {
    typedef uint32_t piece __attribute__((ext_vector_type(C), aligned(sizeof(IO))));
    if (n == N) {
#pragma unroll
      for (int k = 0; k < W / C; ++k) {
        const piece* a = reinterpret_cast<const piece*>(p + k * C * 4 / (int)sizeof(IO));
        // two pieces lie in one line: the first must not drop it
        const piece q = NT && W == C ? __builtin_nontemporal_load(a) : *a;
#pragma unroll
        for (int i = 0; i < C; ++i) w[k * C + i] = q[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if constexpr (sizeof(IO) == 4) w[i] = i < n ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
        else w[i] = (2 * i < n ? (uint32_t)p[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)p[2 * i + 1] << 16 : 0u);
      }
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(IO) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
};

template <typename IO, int N>
__device__ __forceinline__ void store_n(IO* p, int n, const float (&x)[N]) {
  constexpr int V = 16 / (int)sizeof(IO);
  if (n == N && N % V == 0) {
#pragma unroll
    for (int k = 0; k < N / V; ++k) {
      typename Unaligned<IO>::type q;
      if constexpr (V == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          q[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[k * V + 2 * i]) |
                 ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[k * V + 2 * i + 1]) << 16);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = __float_as_uint(x[k * V + i]);
      }
      auto* a = reinterpret_cast<typename Unaligned<IO>::type*>(p + k * V);
      if constexpr (N == V) __builtin_nontemporal_store(q, a);
      else *a = q;  // half a line at a time: put together by the cache
    }
  } else if (n == N && N == 4 && V == 8) {
    typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(2)));
    u32x2u q;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      q[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i]) |
             ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i + 1]) << 16);
    __builtin_nontemporal_store(q, reinterpret_cast<u32x2u*>(p));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) store_io(p + i, x[i]);
  }
}

}  // namespace ssm
