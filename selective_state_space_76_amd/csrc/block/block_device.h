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
#pragma unroll
      for (int k = 0; k < 6; ++k) v[k] = at & 4 ? v[k + 2] : v[k];  // (v[6] and v[7] are not looked at from here on)
#pragma unroll
      for (int k = 0; k < 5; ++k) v[k] = at & 2 ? v[k + 1] : v[k];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = at & 1 ? v[k] >> 16 | v[k + 1] << 16 : v[k];
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

}  // namespace ssm
