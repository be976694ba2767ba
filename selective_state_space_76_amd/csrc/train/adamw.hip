// adamw.hip -- one AdamW step over many tensors, the gradients' norm, and the 8-bit states.
//
//   g = clip * grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g g
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Layout: a launch covers up to kAdamTensors tensors whose addresses travel in the kernel arguments (no
// table in memory to fill, keep or wait for).  A workgroup owns one chunk of kAdamChunk elements of one
// tensor, found by bisection over the first workgroup of each tensor; a lane owns V consecutive elements
// (4 with fp32 states, 8 with 8-bit ones, so that every stream is read in 8- or 16-byte pieces).
// With fp32 states the step is bound by HBM: it touches every byte once, at 5.2 TB/s (a copy reaches 5.2, a plain
// sum 6.0): 127 M bf16 weights with masters 0.68 ms.  With 8-bit states the instructions (about 70 an
// element, three of them 32-bit integer products for the random numbers) take nearly as long as the 10 bytes:
// 311 M bf16 weights 0.60 ms, 5.2 TB/s (0.79 ms with 87 instructions).  Loading the next piece before
// the present one is worked on gained nothing with either.
// The gradients' norm comes first and reads them once more: 127 M in bf16 44 us, 5.8 TB/s.  Its last kernel also counts
// the step and writes what depends on the step's number (AdamProgress), so that neither is a matter of the host.
//
// 8-bit states.  A positive float's bit pattern is an increasing integer, and its top 12 bits a number
// of 4 significant bits.  A block of 128 elements (16 lanes of 8) keeps K, the largest element's top
// bits (rounded up) less the largest code, and an element the code c with (c + K) << 20 its bits; c = 0 is
// zero.  The scale of a code is thus its own exponent: 7 bits span 16 octaves (m, with a sign), 8 bits 32
// (v).  With b2 = 0.999 an average moves by a thousandth per step, a code by a sixteenth to an
// eighth, so rounding to nearest would never let it move; adding 16 random bits below the kept ones
// rounds up with the odds of the part cut off, which keeps the expected state exact.  A v > 0 is
// never rounded to zero: a zero under a nonzero m would divide by eps alone.  m below its smallest code
// becomes that code with the odds that keep its mean, else zero.
// A block in which a gradient, or a square of one, was not finite keeps the complement of K, a negative number: there
// the largest code stands for infinity, a NaN too, and the largest of the others has the code below.  So the neighbours
// of such an element go on as if it were not there, as they do with fp32 states.
#include <type_traits>

#include "../ssm_device.h"
#include "train_device.h"
#include "train_launch.h"

namespace ssm {

namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 32 bits mixed by xor-shifts and products with the fractions of sqrt(2) and sqrt(3)
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

template <int V>
__device__ __forceinline__ void store(float* p, int c, const float (&x)[V]) {
  if (c == V) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const f32x4 q = {x[i], x[i + 1], x[i + 2], x[i + 3]};
      if constexpr (V == 4) __builtin_nontemporal_store(q, reinterpret_cast<f32x4*>(p + i));
      else *reinterpret_cast<f32x4*>(p + i) = q;  // half a line at a time: put together by the cache
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < c) p[i] = x[i];
  }
}
// the upper halves of V words
template <int V>
__device__ __forceinline__ void store_high(bf16_t* p, int c, const uint32_t (&x)[V]) {
  if (c == V) {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = (x[2 * i] >> 16) | (x[2 * i + 1] & 0xffff0000u);
    if constexpr (V == 8)
      __builtin_nontemporal_store(u32x4{w[0], w[1], w[2], w[3]}, reinterpret_cast<u32x4*>(p));
    else
      __builtin_nontemporal_store(u32x2{w[0], w[1]}, reinterpret_cast<u32x2*>(p));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < c) p[i] = (bf16_t)(x[i] >> 16);
  }
}
// 8 codes, c of which are the tensor's (a block's room is there even where its tensor ends inside it)
__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int c) {
  u32x2 q = {0u, 0u};
  if (c > 0) q = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
  if (c < 8) {
    const uint64_t keep = (1ull << (8 * c)) - 1;
    q[0] &= (uint32_t)keep;
    q[1] &= (uint32_t)(keep >> 32);
  }
  return q;
}
__device__ __forceinline__ u32x2 pack_codes(const uint32_t (&x)[8]) {
  u32x2 q;
#pragma unroll
  for (int i = 0; i < 2; ++i) q[i] = x[4 * i] | x[4 * i + 1] << 8 | x[4 * i + 2] << 16 | x[4 * i + 3] << 24;
  return q;
}

// largest of a 16-lane row, in every lane of it
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  auto step = [&](auto ctrl) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, decltype(ctrl)::value, 0xf, 0xf, true);
    v = v > o ? v : o;
  };
  step(IC<0x128>{});  // row_ror:8
  step(IC<0x124>{});
  step(IC<0x122>{});
  step(IC<0x121>{});
  return v;
}

// the tensor that workgroup `block` works on
template <typename Table>
__device__ __forceinline__ int find(const Table& t, uint32_t block) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= block) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

constexpr uint32_t kInf = 0x7f800000u;
// what code c of a block with base K stands for; `top`: the largest code
__device__ __forceinline__ uint32_t code_bits(uint32_t c, uint32_t K, uint32_t top) {
  const bool odd = (int32_t)K < 0;
  return !c ? 0u : odd && c == top ? kInf : (c + (odd ? ~K : K)) << 20;
}
// bit 7 of each byte is clear where the byte's low 7 bits (8 bits) are zero
__device__ __forceinline__ uint32_t marks7(uint32_t w) { return (w | 0x80808080u) - 0x01010101u; }
__device__ __forceinline__ uint32_t marks8(uint32_t w) { return marks7(w & 0x7f7f7f7fu) | w; }
__device__ __forceinline__ int32_t clamp_code(int32_t q, int32_t lo, int32_t hi) {
  return q < lo ? lo : q > hi ? hi : q;
}

// base of a block from the bits of its largest magnitude: that element, rounded up, gets code `top`
__device__ __forceinline__ uint32_t block_base(uint32_t largest, uint32_t top) {
  const uint32_t q = (largest + 0xfffffu) >> 20;
  return q > top ? q - top : 0u;
}

}  // namespace

// What a lane reads for its V elements, as it lies in memory; c of them are there, the others are zero.
template <bool PB, bool GB, bool MW, bool S8>
struct AdamPieces {
  static constexpr int V = S8 ? 8 : 4;
  template <bool B> using IO = std::conditional_t<B, bf16_t, float>;
  Raw<IO<GB>, V> g;
  Raw<IO<PB && !MW>, V> p;  // the master weights where there are some
  Raw<float, V> m, v;       // fp32 states
  u32x2 mc, vc;             // 8-bit states: codes, and the block's bases
  uint32_t mk, vk;
  int c;
  __device__ __forceinline__ void load(const AdamTable& t, const AdamParams& a, int k, int64_t off, int64_t i,
                                       int64_t n) {
    const int64_t left = n - i;
    c = left >= V ? V : left > 0 ? (int)left : 0;
    g.load(static_cast<const IO<GB>*>(t.g[k]) + i, c);
    if constexpr (MW) p.load(a.master + off + i, c);
    else p.load(static_cast<const IO<PB>*>(t.p[k]) + i, c);
    if constexpr (S8) {
      mc = load_codes(static_cast<const uint8_t*>(a.m) + off + i, c);
      vc = load_codes(static_cast<const uint8_t*>(a.v) + off + i, c);
      mk = vk = 0;
      if (c > 0) {
        mk = (uint32_t)(int32_t)a.mb[(off + i) / kAdamBlock];
        vk = (uint32_t)(int32_t)a.vb[(off + i) / kAdamBlock];
      }
    } else {
      m.load(static_cast<const float*>(a.m) + off + i, c);
      v.load(static_cast<const float*>(a.v) + off + i, c);
    }
  }
};

template <bool PB, bool GB, bool MW, bool S8>
__global__ __launch_bounds__(256) void adamw_kernel(AdamTable t, AdamParams a) {
#pragma clang fp contract(off)  // every product and sum of the states rounds once: the codes depend on their bits
  constexpr int V = S8 ? 8 : 4;
  float clip = 1.0f, isb = a.isb, size = a.step;
  uint32_t now = 0;
  if (a.progress) {  // (under way while the tensor is looked for)
    clip = a.progress->factor;
    isb = a.progress->isb;
    size = a.progress->size;
    now = a.progress->key;
  } else if (a.clip) {
    clip = a.clip[1];
  }
  const int k = find(t, blockIdx.x);
  if (clip != clip) return;  // the gradients' norm is not finite: nothing changes
  const uint32_t key = a.progress ? mix32(now + t.key[k]) : t.key[k];
  const int64_t n = t.n[k], off = t.off[k];
  // the wave's first element
  const int64_t base = (int64_t)(blockIdx.x - t.first[k]) * kAdamChunk + (threadIdx.x & ~63) * V;
#pragma unroll 1
  for (int it = 0; it < kAdamChunk / (256 * V); ++it) {
    const int64_t w0 = base + it * (256 * V);
    if (w0 >= n) break;
    const int64_t i = w0 + (threadIdx.x & 63) * V;
    AdamPieces<PB, GB, MW, S8> x;
    x.load(t, a, k, off, i, n);
    const int c = x.c;
    const int64_t blk = (off + i) / kAdamBlock;
    float p[V], g[V], m[V], v[V];
    if constexpr (S8) {
      uint32_t mb[V], vb[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        mb[e] = (((x.mc[e >> 2] >> (8 * (e & 3))) & 127u) + x.mk) << 20;
        vb[e] = (((x.vc[e >> 2] >> (8 * (e & 3))) & 255u) + x.vk) << 20;
      }
      const uint32_t all = marks7(x.mc[0]) & marks7(x.mc[1]) & marks8(x.vc[0]) & marks8(x.vc[1]);
      if (~all & 0x80808080u) {  // codes of zero among them
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if (!((x.mc[e >> 2] >> (8 * (e & 3))) & 127u)) mb[e] = 0u;
          if (!((x.vc[e >> 2] >> (8 * (e & 3))) & 255u)) vb[e] = 0u;
        }
      }
      if (__builtin_expect((int32_t)(x.mk | x.vk) < 0, 0)) {  // blocks that hold infinities
#pragma unroll
        for (int e = 0; e < V; ++e) {
          mb[e] = code_bits((x.mc[e >> 2] >> (8 * (e & 3))) & 127u, x.mk, 127u);
          vb[e] = code_bits((x.vc[e >> 2] >> (8 * (e & 3))) & 255u, x.vk, 255u);
        }
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        m[e] = __uint_as_float(mb[e] | ((x.mc[e >> 2] << (24 - 8 * (e & 3))) & 0x80000000u));
        v[e] = __uint_as_float(vb[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      g[e] = x.g.at(e);
      p[e] = x.p.at(e);
      if constexpr (!S8) {
        m[e] = x.m.at(e);
        v[e] = x.v.at(e);
      }
    }
    uint32_t h[V];
    if constexpr (S8 || (PB && !MW)) {
#pragma unroll
      for (int e = 0; e < V; ++e) h[e] = mix32(((uint32_t)i + e) * 0x9E3779B9u + key);
    }
    uint32_t pb[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float ge = g[e] * clip;
      m[e] = m[e] * a.b1 + ge * a.c1;
      v[e] = v[e] * a.b2 + ge * a.c2 * ge;
      const float den = __builtin_fmaf(__builtin_amdgcn_sqrtf(v[e]), isb, a.eps);
      p[e] = __builtin_fmaf(-(m[e] * size), rcp_(den), p[e] * a.decay);
      if constexpr (PB) {
        if constexpr (MW) {
          pb[e] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)p[e]) << 16;
        } else {
          const uint32_t b = __float_as_uint(p[e]);
          // What is not finite stays so.  The lower half of an infinity is zero, and that of a NaN where every input
          // came in bf16 or codes; from fp32 gradients or states it may be all ones.
          const uint32_t r = (h[e] * 0x3C6EF373u) >> 16;
          pb[e] = b + ((GB && S8) || __builtin_isfinite(p[e]) ? r : 0u);
        }
      }
    }
    if constexpr (MW) store<V>(a.master + off + i, c, p);
    if constexpr (PB) store_high<V>(static_cast<bf16_t*>(t.p[k]) + i, c, pb);
    else store<V>(static_cast<float*>(t.p[k]) + i, c, p);
    if constexpr (S8) {
      // elements that are not there have been zero all along, and stay so
      uint32_t am = 0, av = 0;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const uint32_t x = __float_as_uint(m[e]) & 0x7fffffffu, y = __float_as_uint(v[e]);
        am = am > x ? am : x;
        av = av > y ? av : y;
      }
      am = row_max(am);
      av = row_max(av);
      uint32_t mc[8], vc[8], mk, vk;
      auto encode = [&](int32_t top_m, int32_t top_v) {
        mk = block_base(am, (uint32_t)top_m);
        vk = block_base(av, (uint32_t)top_v);
        const uint32_t least = (mk + 1) << 20, m0 = 8u - (mk << 20), v0 = 8u - (vk << 20);
        bool under = false;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const uint32_t x = __float_as_uint(m[e]) & 0x7fffffffu, y = __float_as_uint(v[e]);
          const uint32_t rm = (h[e] & 0xffffu) << 4, rv = (h[e] >> 16) << 4;
          mc[e] = (uint32_t)clamp_code((int32_t)(x + rm + m0) >> 20, 0, top_m);
          vc[e] = (uint32_t)clamp_code((int32_t)(y + rv + v0) >> 20, (int32_t)(y < 1u ? y : 1u), top_v);
          under |= x - 1u < least - 1u;  // 0 < x < least
        }
        if (under) {  // below the smallest code: that code or zero
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const uint32_t x = __float_as_uint(m[e]) & 0x7fffffffu;
            const bool up =
                __uint_as_float(x) > __uint_as_float(least) * ((float)(h[e] & 0xffffu) * 0x1p-16f + 0x1p-17f);
            if (x < least) mc[e] = up ? 1u : 0u;
          }
        }
      };
      if (__builtin_expect(am < kInf && av < kInf, 1)) {  // the same in all lanes of a block
        encode(127, 255);
      } else {  // what is not finite gets the largest code, and the base goes by the other elements
        const bool odd_m = am >= kInf, odd_v = av >= kInf;
        am = av = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const uint32_t x = __float_as_uint(m[e]) & 0x7fffffffu, y = __float_as_uint(v[e]) & 0x7fffffffu;
          if (x < kInf) am = am > x ? am : x;
          if (y < kInf) av = av > y ? av : y;
        }
        am = row_max(am);
        av = row_max(av);
        encode(odd_m ? 126 : 127, odd_v ? 254 : 255);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if ((__float_as_uint(m[e]) & 0x7fffffffu) >= kInf) mc[e] = 127u;
          if ((__float_as_uint(v[e]) & 0x7fffffffu) >= kInf) vc[e] = 255u;
        }
        if (odd_m) mk = ~mk;
        if (odd_v) vk = ~vk;
      }
      u32x2 mw = pack_codes(mc);
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // the signs: the upper bytes of 4 floats
        auto top = [&](int hi, int lo, uint32_t select) {
          return __builtin_amdgcn_perm(__float_as_uint(m[4 * e + hi]), __float_as_uint(m[4 * e + lo]), select);
        };
        const uint32_t s01 = top(1, 0, 0x0c0c0703u), s23 = top(3, 2, 0x07030c0cu);
        mw[e] |= (s01 | s23) & 0x80808080u;
      }
      if (c > 0) {
        __builtin_nontemporal_store(mw, reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.m) + off + i));
        __builtin_nontemporal_store(pack_codes(vc), reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.v) + off + i));
        if ((threadIdx.x & 15) == 0) {
          a.mb[blk] = (int16_t)mk;
          a.vb[blk] = (int16_t)vk;
        }
      }
    } else {
      store<V>(static_cast<float*>(a.m) + off + i, c, m);
      store<V>(static_cast<float*>(a.v) + off + i, c, v);
    }
  }
}

// Sum of the squares of one chunk, in fp64 (no overflow below fp32's largest squares, and no loss over
// many elements); the workgroup's 256 lanes are added in a fixed tree.
template <bool GB>
__global__ __launch_bounds__(256) void norm_part_kernel(NormTable t, double* part) {
  constexpr int V = GB ? 8 : 4;
  using IO = std::conditional_t<GB, bf16_t, float>;
  const int k = find(t, blockIdx.x);
  const int64_t n = t.n[k];
  const int64_t base = (int64_t)(blockIdx.x - t.first[k]) * kNormChunk + threadIdx.x * V;
  double s = 0.0;
#pragma unroll 1
  for (int it = 0; it < kNormChunk / (256 * V); it += 4) {
    if (base - threadIdx.x * V + it * (256 * V) >= n) break;
    Raw<IO, V> g[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t i = base + (it + q) * (256 * V), left = n - i;
      g[q].load(static_cast<const IO*>(t.g[k]) + i, left >= V ? V : left > 0 ? (int)left : 0);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < V; ++e) s = __builtin_fma((double)g[q].at(e), (double)g[q].at(e), s);
  }
  __shared__ double sm[256];
  sm[threadIdx.x] = s;
  __syncthreads();
#pragma unroll
  for (int h = 128; h > 0; h >>= 1) {
    if ((int)threadIdx.x < h) sm[threadIdx.x] += sm[threadIdx.x + h];
    __syncthreads();
  }
  if (threadIdx.x == 0) part[blockIdx.x] = sm[0];
}

// x^n by squaring: within n units of the last place of 1, which 1 - x^n is then right to
__device__ __forceinline__ double power(double x, int64_t n) {
  double r = 1.0;
  for (; n > 0; n >>= 1) {
    if (n & 1) r *= x;
    x *= x;
  }
  return r;
}

// What the next step takes, by the first wave while it waits for its gradients.
struct Next {
  AdamProgress p;
  __device__ __forceinline__ explicit Next(const AdamAdvance& a) {
    if (!a.progress || threadIdx.x >= 64) return;
    p.step = a.progress->step + 1;
    p.size = (float)(a.lr / (1.0 - power(a.b1, p.step)));
    p.isb = (float)(1.0 / sqrt(1.0 - power(a.b2, p.step)));
    p.key = mix32(a.seed + (uint32_t)p.step);
  }
};

// The sum of a workgroup's 1024 lanes in a fixed tree, and from it the result: result[0] the norm and result[1] the
// factor, or with progress the norm alone.
__device__ __forceinline__ void finish_norm(double s, double* sm, double max_norm, float* result, const AdamAdvance& adv,
                                            const Next& next) {
  sm[threadIdx.x] = s;
  __syncthreads();
  for (int h = 512; h > 0; h >>= 1) {
    if ((int)threadIdx.x < h) sm[threadIdx.x] += sm[threadIdx.x + h];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const double norm = sqrt(sm[0]);
    const float out = (float)norm;
    const bool finite = (__float_as_uint(out) & 0x7f800000u) != 0x7f800000u;
    const float factor = !finite ? __uint_as_float(0x7fc00000u) : norm > max_norm ? (float)(max_norm / norm) : 1.0f;
    result[0] = out;
    if (!adv.progress) {
      result[1] = factor;
    } else if (finite) {
      adv.progress->step = next.p.step;
      adv.progress->factor = factor;
      adv.progress->size = next.p.size;
      adv.progress->isb = next.p.isb;
      adv.progress->key = next.p.key;
    } else {
      adv.progress->factor = factor;  // and the step is not counted
    }
  }
}

__global__ __launch_bounds__(1024) void norm_join_kernel(const double* part, int64_t n, double max_norm, float* result,
                                                         AdamAdvance adv) {
  __shared__ double sm[1024];
  const Next next(adv);
  double s = 0.0;
  int64_t i = threadIdx.x;
  for (; i + 7 * 1024 < n; i += 8 * 1024) {
    double x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = part[i + e * 1024];
#pragma unroll
    for (int e = 0; e < 8; ++e) s += x[e];
  }
  for (; i < n; i += 1024) s += part[i];
  finish_norm(s, sm, max_norm, result, adv, next);
}

template <bool GB>
__device__ __forceinline__ double chunk_squares(const void* g, int64_t base, int64_t n) {
  constexpr int V = GB ? 8 : 4, N = (int)(kSmallChunk / (64 * V));
  using IO = std::conditional_t<GB, bf16_t, float>;
  Raw<IO, V> x[N];
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const int64_t i = base + (q * 64 + (threadIdx.x & 63)) * V, left = n - i;
    x[q].load(static_cast<const IO*>(g) + i, left >= V ? V : left > 0 ? (int)left : 0);
  }
  double s = 0.0;
#pragma unroll
  for (int q = 0; q < N; ++q)
#pragma unroll
    for (int e = 0; e < V; ++e) s = __builtin_fma((double)x[q].at(e), (double)x[q].at(e), s);
  return s;
}

// Few and small tensors: one workgroup, a wave per chunk, and no second launch.
__global__ __launch_bounds__(1024) void norm_small_kernel(SmallNormTable t, uint32_t chunks, double max_norm,
                                                          float* result, AdamAdvance adv) {
  __shared__ double sm[1024];
  const Next next(adv);
  double s = 0.0;
  for (uint32_t c = threadIdx.x >> 6; c < chunks; c += 16) {
    const int k = find(t, c);
    const int64_t base = (int64_t)(c - t.first[k]) * kSmallChunk;
    s += t.bf16[k] ? chunk_squares<true>(t.g[k], base, t.n[k]) : chunk_squares<false>(t.g[k], base, t.n[k]);
  }
  finish_norm(s, sm, max_norm, result, adv, next);
}

// (c + K) << 20 has its set bits in the upper half: the value in bf16 is (c + K) << 4, exactly
__global__ __launch_bounds__(256) void state_values_kernel(int64_t n, const uint8_t* m, const uint8_t* v,
                                                           const int16_t* mb, const int16_t* vb, bf16_t* mo,
                                                           bf16_t* vo) {
  const int64_t i = ((int64_t)block_id() * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  uint32_t x[8];
  if (mo) {
    const u32x2 w = load_codes(m + i, 8);
    const uint32_t K = (uint32_t)(int32_t)mb[i / kAdamBlock];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t c = w[e >> 2] >> (8 * (e & 3));
      x[e] = code_bits(c & 127u, K, 127u) | ((c << 24) & 0x80000000u);
    }
    store_high<8>(mo + i, 8, x);
  }
  if (vo) {
    const u32x2 w = load_codes(v + i, 8);
    const uint32_t K = (uint32_t)(int32_t)vb[i / kAdamBlock];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = code_bits((w[e >> 2] >> (8 * (e & 3))) & 255u, K, 255u);
    store_high<8>(vo + i, 8, x);
  }
}

uint32_t adam_seed(uint64_t seed) {
  const uint32_t x = mix32((uint32_t)seed);
  return seed >> 32 ? mix32(x + (uint32_t)(seed >> 32)) : x;
}

uint32_t adam_key(uint64_t seed, int64_t step, int64_t tensor) {
  return mix32(mix32(adam_seed(seed) + (uint32_t)step) + (uint32_t)tensor);
}

hipError_t launch_adamw(const AdamTable& t, const AdamParams& p, int kind, uint32_t blocks, hipStream_t s) {
  auto go = [&](auto fn) { hipLaunchKernelGGL(fn, dim3(blocks), dim3(256), 0, s, t, p); };
  switch (kind) {
    case 0: go(adamw_kernel<false, false, false, false>); break;
    case 1: go(adamw_kernel<true, false, false, false>); break;
    case 2: go(adamw_kernel<false, true, false, false>); break;
    case 3: go(adamw_kernel<true, true, false, false>); break;
    case 5: go(adamw_kernel<true, false, true, false>); break;
    case 7: go(adamw_kernel<true, true, true, false>); break;
    case 8: go(adamw_kernel<false, false, false, true>); break;
    case 9: go(adamw_kernel<true, false, false, true>); break;
    case 10: go(adamw_kernel<false, true, false, true>); break;
    case 11: go(adamw_kernel<true, true, false, true>); break;
    case 13: go(adamw_kernel<true, false, true, true>); break;
    case 15: go(adamw_kernel<true, true, true, true>); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_norm_part(const NormTable& t, double* part, bool bf16, uint32_t blocks, hipStream_t s) {
  if (bf16) hipLaunchKernelGGL(norm_part_kernel<true>, dim3(blocks), dim3(256), 0, s, t, part);
  else hipLaunchKernelGGL(norm_part_kernel<false>, dim3(blocks), dim3(256), 0, s, t, part);
  return hipGetLastError();
}

hipError_t launch_norm_small(const SmallNormTable& t, uint32_t chunks, double max_norm, float* result,
                             const AdamAdvance& adv, hipStream_t s) {
  hipLaunchKernelGGL(norm_small_kernel, dim3(1), dim3(1024), 0, s, t, chunks, max_norm, result, adv);
  return hipGetLastError();
}

hipError_t launch_norm_join(const double* part, int64_t n, double max_norm, float* result, const AdamAdvance& adv,
                            hipStream_t s) {
  hipLaunchKernelGGL(norm_join_kernel, dim3(1), dim3(1024), 0, s, part, n, max_norm, result, adv);
  return hipGetLastError();
}

hipError_t launch_state_values(int64_t n, const void* m, const void* v, const int16_t* mb, const int16_t* vb,
                               void* mo, void* vo, hipStream_t s) {
  hipLaunchKernelGGL(state_values_kernel, grid_of((n / 8 + 255) / 256), dim3(256), 0, s, n,
                     static_cast<const uint8_t*>(m), static_cast<const uint8_t*>(v), mb, vb,
                     static_cast<bf16_t*>(mo), static_cast<bf16_t*>(vo));
  return hipGetLastError();
}

}  // namespace ssm
