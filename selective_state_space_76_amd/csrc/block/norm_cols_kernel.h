// norm_cols_kernel.h -- the layer norm of norm_rows.hip over the channels of [B, E, L], the layout of the conv and the
// scan; compiled by norm_cols_{bf16,mixed,f32}.hip.
//
// A workgroup owns T = LP * 8 consecutive positions of one batch row and all of their channels: LP lanes hold a channel's
// positions, 8 each, and the NT / LP groups of lanes take the channels in turn, C of them at a time.  A position's sums go
// over the groups: within a wave by exchanges that leave each lane one position, over the waves through LDS.  KEEP: C
// channels a group are all there are, and stay in registers as they came from memory; otherwise they are read again
// for every pass.
//
// Bound by HBM: 2^17 positions x 1024 channels in bf16, RMS norm: 113-119 us by the box, 4.5-4.7 TB/s (a copy 104).  The
// gradients of 4 x 4096 x 2048 with a residual and the stream's own gradient: 63 us, and 5 for the join of the tiles'
// sums, 4.85 TB/s with what is read twice.
#pragma once
#include "block_device.h"

namespace ssm {

namespace {

// v[k] summed over all lanes of the workgroup that have the same positions; sm: (NT / 64 + 1) * LP * 8 floats
template <int NT, int LP>
__device__ __forceinline__ void sum_groups(float (&v)[8], float* sm) {
  constexpr int T = LP * 8, NW = NT / 64;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  // halves of the positions are exchanged with the lane 32, 16 and 8 away: its bits 5, 4 and 3 name what is left
  float* to = sm + w * T + (lane % LP) * 8 + (lane >> 5) * 4;
  float a[4], b[2], c;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float keep = lane & 32 ? v[k + 4] : v[k], send = lane & 32 ? v[k] : v[k + 4];
    a[k] = keep + __shfl_xor(send, 32);
  }
  if constexpr (LP == 32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) to[k] = a[k];
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float keep = lane & 16 ? a[k + 2] : a[k], send = lane & 16 ? a[k] : a[k + 2];
      b[k] = keep + __shfl_xor(send, 16);
    }
    to += (lane >> 4 & 1) * 2;
    if constexpr (LP == 16) {
      to[0] = b[0];
      to[1] = b[1];
    } else {
      const float keep = lane & 8 ? b[1] : b[0], send = lane & 8 ? b[0] : b[1];
      c = keep + __shfl_xor(send, 8);
#pragma unroll
      for (int m = 4; m >= LP; m /= 2) c += __shfl_xor(c, m);
      to[lane >> 3 & 1] = c;  // (lanes of the same position: the same sum)
    }
  }
  __syncthreads();
  if (threadIdx.x < T) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) s += sm[i * T + threadIdx.x];
    sm[NW * T + threadIdx.x] = s;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = sm[NW * T + (threadIdx.x % LP) * 8 + k];
}

// The workgroup's tile of `count`, or -1.  Where tiles share lines an XCD's tiles are neighbours, so that its L2 has a
// line once (4 x 2048 x 4095, gradients: 128 us in order, 88 so; 2^17 x 1024, which shares none: 119 and 132).
__device__ __forceinline__ int64_t tile_id(int64_t count, bool lines) {
  const uint32_t blk = block_id();
  return blk >= count ? -1 : lines ? (int64_t)blk : xcd_remap((int)blk, (int)count);
}

// sum over the LP lanes that hold a channel's positions
template <int LP> __device__ __forceinline__ float sum_positions(float v) {
  auto step = [&](auto ctrl) {
    v += __uint_as_float(
        (uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  step(IC<0xb1>{});                             // quad_perm [1,0,3,2]
  if constexpr (LP >= 4) step(IC<0x4e>{});      // quad_perm [2,3,0,1]
  if constexpr (LP >= 8) step(IC<0x141>{});     // row_half_mirror
  if constexpr (LP >= 16) step(IC<0x140>{});    // row_mirror
  if constexpr (LP >= 32) v += __shfl_xor(v, 16);
  return v;
}

// The sum is to be taken here: the compiler would put the additions off to where the sum is used, behind all channels, and
// keep all of their terms until then.
__device__ __forceinline__ void here(float& v) { asm volatile("" : "+v"(v)); }

// A channel's numbers join a lane's means and its squares about them; share: 1 / the channels so far.  RMS norm: the
// means are zero (by a mask: an infinite number times a share of zero would make the sum NaN, and it is infinite).
__device__ __forceinline__ void one_more(const float (&s)[8], float share, int rms, float (&mean)[8], float (&squares)[8]) {
  const uint32_t some = rms ? 0u : ~0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = s[i] - mean[i];
    mean[i] = __uint_as_float(__float_as_uint(__builtin_fmaf(d, share, mean[i])) & some);
    squares[i] = __builtin_fmaf(d, s[i] - mean[i], squares[i]);
  }
}

// Where rows do not begin with a line, neighbouring tiles write parts of one: put together by the cache.
template <typename IO>
__device__ __forceinline__ void store_cols(IO* p, int n, const float (&x)[8], bool lines) {
  if (lines || n < 8) return store_n<IO, 8>(p, n, x);
#pragma unroll
  for (int k = 0; k < (int)sizeof(IO) / 2; ++k) {
    typename Unaligned<IO>::type q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(IO) == 2)
        q[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i]) |
               (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i + 1]) << 16;
      else
        q[i] = __float_as_uint(x[k * 4 + i]);
    }
    *(reinterpret_cast<typename Unaligned<IO>::type*>(p) + k) = q;
  }
}

}  // namespace

// Of very many channels, the turns whose sums are taken by themselves and then compensated.
constexpr int kBlock = 64;

// On this architecture a wave that waits for a load waits for the stores that it issued before, too.  So nothing is
// loaded behind a store that it does not follow from: weights come with the pieces, and where pieces are read again, the
// next ones are asked for before the present ones are stored.

// C channels of a lane: NG apart, from channel e on
template <typename XT, typename HT, bool RES, int C>
struct Chunk {
  Piece<XT> x[C];  // zeros where dropped
  Piece<HT> q[RES ? C : 1];
  float w[C], c[C];
};

// RES: there is a residual.  DROP: there is dropout (not with KEEP: the masks of all channels at once would take more
// registers than there are).  ODD: L is no multiple of 8.  MANY: more than kManyChannels, not with KEEP.
template <typename XT, typename HT, bool RES, bool DROP, bool ODD, int NT, int LP, int C, bool KEEP, bool MANY>
__global__ __launch_bounds__(NT) void norm_cols_kernel(NormParams p) {
  constexpr int NG = NT / LP, T = LP * 8;
  constexpr bool SHARED = ODD || LP < 8;  // neighbouring tiles share lines
  __shared__ float sm[(NT / 64 + 1) * T];
  const int pl = threadIdx.x % LP, cg = threadIdx.x / LP, E = (int)p.E;
  const bool lines = !SHARED && p.L % 64 == 0;  // tiles are whole lines
  const int64_t tiles = (p.L + T - 1) / T, blk = tile_id(p.B * tiles, lines);
  if (blk < 0) return;
  const int64_t b = blk / tiles, t = blk % tiles * T + pl * 8, total = p.rows * p.E, step = NG * p.L;
  const int n = p.L - t >= 8 ? 8 : !ODD || p.L <= t ? 0 : (int)(p.L - t);
  const int64_t base = b * p.E * p.L + t;
  static_assert(!(DROP && KEEP), "");
  const Drop drop(p.drop);
  typedef Chunk<XT, HT, RES, C> Ch;
  // f(c, e, where it lies) for the lane's channels e from e0 on.  Where they lie is worked out again by every pass: kept
  // from one to the next it would take two registers a channel.
  auto channels = [&](int e0, auto f) {
    int e = e0 + cg;
    asm volatile("" : "+v"(e));
    int64_t at = base + e * p.L;
#pragma unroll
    for (int c = 0; c < C; ++c, e += NG, at += step) f(c, e, at);
  };
  auto fetch = [&](Ch& k, int e0, bool side) {  // (positions behind the last one: whatever is there)
    channels(e0, [&](int c, int e, int64_t at) {
      const bool may = e < E && n > 0 && (!ODD || at + 8 <= total);
      k.x[c].full(static_cast<const XT*>(p.x) + at, may, SHARED || (!KEEP && !side));
      if (RES) k.q[RES ? c : 0].full(static_cast<const HT*>(p.residual) + at, may, SHARED || (!KEEP && !side));
    });
    if (side) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int e = e0 + cg + c * NG, i = e < E ? e : 0;
        k.w[c] = p.weight ? p.weight[i] : 1.0f;
        k.c[c] = p.bias ? p.bias[i] : 0.0f;
      }
    }
    if (ODD)
      channels(e0, [&](int c, int e, int64_t at) {
        if (e < E && n > 0 && at + 8 > total) {  // the tensor's end
          Part r;
          r.hi = n;
          k.x[c].part(static_cast<const XT*>(p.x) + at, r);
          if (RES) k.q[RES ? c : 0].part(static_cast<const HT*>(p.residual) + at, r);
        }
      });
    if (DROP)
      channels(e0, [&](int c, int, int64_t at) {
        k.x[c].keep(drop.kept((uint64_t)at));
        __builtin_amdgcn_sched_barrier(0);
      });
  };
  auto sum = [&](const Ch& k, int c, float (&s)[8]) {  // what is normalised
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = DROP ? k.x[c].at(i) * drop.scale : k.x[c].at(i);
    if (RES) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += k.q[RES ? c : 0].at(i);
    }
  };
  // f(chunk, e0) for all channels
  Ch kept;
  if (KEEP) fetch(kept, 0, true);
  auto pass = [&](bool side, auto f) {
    if constexpr (KEEP) {
      f(kept, 0);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        kept.x[c].forget();
        if (RES) kept.q[RES ? c : 0].forget();
      }
    } else {
      Ch next;
      fetch(next, 0, side);
      for (int e0 = 0; e0 < E; e0 += C * NG) {
        const Ch now = next;
        if (e0 + C * NG < E) fetch(next, e0 + C * NG, side);
        f(now, e0);
      }
    }
  };
  auto keep = [&](const Ch& k, int e0) {
    channels(e0, [&](int c, int e, int64_t at) {
      float s[8];
      sum(k, c, s);
      if (e < E) store_cols(static_cast<HT*>(p.hidden) + at, n, s, lines);
    });
  };
  float m[8], r[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) m[k] = r[k] = 0.0f;
  if constexpr (KEEP) {
    if (p.hidden) pass(false, keep);
    if (!p.rms) {
      pass(false, [&](const Ch& k, int) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float s[8];
          sum(k, c, s);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            m[i] += s[i];  // (zero for a channel that is not there)
            here(m[i]);
          }
        }
      });
      sum_groups<NT, LP>(m, sm);
#pragma unroll
      for (int k = 0; k < 8; ++k) m[k] *= p.inv_e;
    }
    pass(false, [&](const Ch& k, int) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float s[8];
        sum(k, c, s);
        if (cg + c * NG < E) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float d = s[i] - m[i];
            r[i] = __builtin_fmaf(d, d, r[i]);
            here(r[i]);
          }
        }
      }
    });
  } else {
    // One pass: the lane's own mean and its squares about that, kept up to date channel by channel; the lanes' means
    // then differ from the whole mean by what is added to the squares.  MANY: kBlock turns at a time, each block's
    // numbers then put to those of the blocks before it.
    float mine[8], count = 0.0f, before = 0.0f;
    LongSum mean[MANY ? 8 : 1], squares[MANY ? 8 : 1];
    auto fold = [&] {
      before += count;
      const float share = count > 0.0f ? count / before : 0.0f;
#pragma unroll
      for (int i = 0; i < (MANY ? 8 : 0); ++i) {
        const float d = p.rms ? 0.0f : (mine[i] - mean[i].s) - mean[i].c;
        mean[i].add(d * share);
        squares[i].add(__builtin_fmaf(d * share * (before - count), d, r[i]));
        mine[i] = r[i] = 0.0f;
      }
      count = 0.0f;
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) mine[i] = 0.0f;
    pass(false, [&](const Ch& k, int e0) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (e0 + cg + c * NG < E) {
          float s[8];
          sum(k, c, s);
          count += 1.0f;
          one_more(s, rcp_(count), p.rms, mine, r);
        }
      }
      if (p.hidden) keep(k, e0);
      if (MANY && e0 / (C * NG) % kBlock == kBlock - 1) fold();
    });
    if constexpr (MANY) {
      fold();
      count = before;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        mine[i] = mean[i].value();
        r[i] = squares[i].value();
      }
    }
    if (!p.rms) {
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = mine[i] * count;
      sum_groups<NT, LP>(m, sm);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m[i] *= p.inv_e;
        const float d = mine[i] - m[i];
        r[i] = __builtin_fmaf(d * count, d, r[i]);
      }
    }
  }
  sum_groups<NT, LP>(r, sm);
#pragma unroll
  for (int k = 0; k < 8; ++k) r[k] = 1.0f / sqrtf(r[k] * p.inv_e + p.eps);
  pass(true, [&](const Ch& k, int e0) {
    channels(e0, [&](int c, int e, int64_t at) {
      if (e >= E) return;
      float s[8];
      sum(k, c, s);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = __builtin_fmaf((s[i] - m[i]) * r[i], k.w[c], k.c[c]);
      store_cols(static_cast<XT*>(p.out) + at, n, s, lines);
      __builtin_amdgcn_sched_barrier(0);  // a channel at a time: all together would take several times the registers
    });
  });
  if (p.stats && cg == 0) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) {
        p.stats[b * p.L + t + k] = m[k];
        p.stats[p.rows + b * p.L + t + k] = r[k];
      }
  }
}

// The same with a residual for tiles of 64 positions by 1024 lanes that keep what they can of C channels each, all there
// are: x in registers (what is dropped is zero there), the residual of the first HL in LDS (up to 128 KB; each lane
// its own pieces), the others' is read again.
template <typename XT, typename HT, int C>
__global__ __launch_bounds__(1024) void norm_cols_keep_kernel(NormParams p) {
  constexpr int NT = 1024, LP = 8, NG = NT / LP, T = LP * 8, QH = (int)sizeof(HT) / 2;
  constexpr int HL = C < 16 / (int)sizeof(HT) ? C : 16 / (int)sizeof(HT);
  __shared__ float sm[(NT / 64 + 1) * T];
  __shared__ u32x4a own[HL * QH][NT];
  const int pl = threadIdx.x % LP, cg = threadIdx.x / LP, E = (int)p.E;
  const bool lines = p.L % 64 == 0;
  const int64_t tiles = (p.L + T - 1) / T, step = NG * p.L, tile = tile_id(p.B * tiles, lines);
  if (tile < 0) return;
  const Drop drop(p.drop);
  const float scale = drop.any() ? drop.scale : 1.0f;
  const int64_t b = tile / tiles, t = tile % tiles * T + pl * 8;
  const bool in = t < p.L;
  const int64_t base = b * p.E * p.L + t;
  Piece<XT> x[C];
  Piece<HT> q[2];
  int e0 = cg;
  asm volatile("" : "+v"(e0));
  int64_t at0 = base + e0 * p.L;
  auto other = [&](int c, bool again) {
    q[c & 1].full(static_cast<const HT*>(p.residual) + at0 + c * step, in && e0 + c * NG < E, again);
  };
  auto sum = [&](int c, const Piece<HT>& o, float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = __builtin_fmaf(x[c].at(i), scale, o.at(i));
  };
#pragma unroll
  for (int c = 0; c < C; ++c) x[c].full(static_cast<const XT*>(p.x) + at0 + c * step, in && e0 + c * NG < E);
  other(0, 0 >= HL);
  float m[8], r[8], count = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) m[k] = r[k] = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (c + 1 < C) other(c + 1, c + 1 >= HL);
    const Piece<HT>& now = q[c & 1];
    const int64_t at = at0 + c * step;
    if (drop.any()) x[c].keep(drop.kept((uint64_t)at));
    float s[8];
    sum(c, now, s);
    if (e0 + c * NG < E) {
      count += 1.0f;
      one_more(s, rcp_(count), p.rms, m, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        here(m[i]);
        here(r[i]);
      }
      if (in && p.hidden) store_cols(static_cast<HT*>(p.hidden) + at, 8, s, lines);
    }
    if (c < HL) {
#pragma unroll
      for (int k = 0; k < QH; ++k) own[(c < HL ? c : 0) * QH + k][threadIdx.x] = now.w[k];
    }
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) x[c].forget();
  e0 = cg;
  asm volatile("" : "+v"(e0));
  at0 = base + e0 * p.L;
  float w[2], o[2];
  auto second = [&](int c) {
    if (c >= HL) other(c, false);
    const int e = e0 + c * NG < E ? e0 + c * NG : 0;
    w[c & 1] = p.weight ? p.weight[e] : 1.0f;
    o[c & 1] = p.bias ? p.bias[e] : 0.0f;
  };
  second(0);
  if (!p.rms) {
    float mine[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mine[i] = m[i];
      m[i] *= count;
    }
    sum_groups<NT, LP>(m, sm);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] *= p.inv_e;
      const float d = mine[i] - m[i];
      r[i] = __builtin_fmaf(d * count, d, r[i]);
    }
  }
  sum_groups<NT, LP>(r, sm);
#pragma unroll
  for (int k = 0; k < 8; ++k) r[k] = 1.0f / sqrtf(r[k] * p.inv_e + p.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (c + 1 < C) second(c + 1);
    Piece<HT> now = q[c & 1];
    if (c < HL) {
#pragma unroll
      for (int k = 0; k < QH; ++k) now.w[k] = own[(c < HL ? c : 0) * QH + k][threadIdx.x];
    }
    float s[8];
    sum(c, now, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = __builtin_fmaf((s[i] - m[i]) * r[i], w[c & 1], o[c & 1]);
    if (in && e0 + c * NG < E) store_cols(static_cast<XT*>(p.out) + at0 + c * step, 8, s, lines);
    __builtin_amdgcn_sched_barrier(0);
  }
  if (p.stats && cg == 0 && in) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      p.stats[b * p.L + t + k] = m[k];
      p.stats[p.rows + b * p.L + t + k] = r[k];
    }
  }
}

// A tile each, everything read twice.  The tile's dw and db are a partial sum of its own.
template <typename XT, typename HT, bool ODD, int NT, int LP, int C, bool MANY>
__global__ __launch_bounds__(NT) void norm_cols_bwd_kernel(NormParams p) {
  constexpr int NG = NT / LP, T = LP * 8;
  constexpr bool SHARED = ODD || LP < 8;  // neighbouring tiles share lines
  __shared__ float sm[(NT / 64 + 1) * T];
  const int pl = threadIdx.x % LP, cg = threadIdx.x / LP, E = (int)p.E;
  const bool lines = !SHARED && p.L % 64 == 0;
  const int64_t tiles = (p.L + T - 1) / T, total = p.rows * p.E, step = NG * p.L, tile = tile_id(p.blocks, lines);
  if (tile < 0) return;
  const Drop drop(p.drop);
  float* part = p.part ? p.part + tile * 2 * p.E : nullptr;
  struct Ch {
    Piece<XT> d[C];
    Piece<HT> h[C], q[C];
    float w[C];
  };
  const int64_t b = tile / tiles, t = tile % tiles * T + pl * 8;
  const int n = p.L - t >= 8 ? 8 : !ODD || p.L <= t ? 0 : (int)(p.L - t);
  const int64_t base = b * p.E * p.L + t;
  Part real;
  real.hi = n;
  auto channels = [&](int e0, auto f) {
    int e = e0 + cg;
    asm volatile("" : "+v"(e));
    int64_t at = base + e * p.L;
#pragma unroll
    for (int c = 0; c < C; ++c, e += NG, at += step) f(c, e, at);
  };
  auto fetch = [&](Ch& k, int e0, bool third) {
    channels(e0, [&](int c, int e, int64_t at) {
      const bool may = e < E && n > 0 && (!ODD || at + 8 <= total), again = SHARED || (LP < 32 && !third);
      k.d[c].full(static_cast<const XT*>(p.x) + at, may, again);
      k.h[c].full(static_cast<const HT*>(p.residual) + at, may, again);
      if (third && p.dhidden) k.q[c].full(static_cast<const HT*>(p.dhidden) + at, may, SHARED);
      k.w[c] = p.weight ? p.weight[e < E ? e : 0] : 1.0f;
    });
    if (ODD)
      channels(e0, [&](int c, int e, int64_t at) {
        if (e < E && n > 0 && at + 8 > total) {
          k.d[c].part(static_cast<const XT*>(p.x) + at, real);
          k.h[c].part(static_cast<const HT*>(p.residual) + at, real);
          if (third && p.dhidden) k.q[c].part(static_cast<const HT*>(p.dhidden) + at, real);
        }
        k.d[c].cut(real);  // (what lies behind the last position takes no part in dw and db)
        k.h[c].cut(real);
      });
  };
  // f(channels, e0) for all channels
  auto pass = [&](bool third, auto f) {
    Ch next;
    fetch(next, 0, third);
    for (int e0 = 0; e0 < E; e0 += C * NG) {
      const Ch now = next;
      if (e0 + C * NG < E) fetch(next, e0 + C * NG, third);
      f(now, e0);
    }
  };
  float m[8], r[8], c1[8], c2[8];
  load_n<float, 8>(p.stats + b * p.L + t, n, m);
  load_n<float, 8>(p.stats + p.rows + b * p.L + t, n, r);
#pragma unroll
  for (int k = 0; k < 8; ++k) c1[k] = c2[k] = 0.0f;
  LongSum s1[MANY ? 8 : 1], s2[MANY ? 8 : 1];
  pass(false, [&](const Ch& k, int e0) {
    if (MANY && e0 / (C * NG) % kBlock == 0) {  // the sums of the block of channels before
#pragma unroll
      for (int i = 0; i < (MANY ? 8 : 0); ++i) {
        s1[i].add(c1[i]);
        s2[i].add(c2[i]);
        c1[i] = c2[i] = 0.0f;
      }
    }
    channels(e0, [&](int c, int e, int64_t) {
      float dw = 0.0f, db = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // (d is 0 for a channel that is not there, r behind the last position)
        const float g = k.d[c].at(i), x = (k.h[c].at(i) - m[i]) * r[i];
        dw = __builtin_fmaf(g, x, dw);
        db += g;
        c1[i] = __builtin_fmaf(g, k.w[c], c1[i]);
        c2[i] = __builtin_fmaf(g * k.w[c], x, c2[i]);
      }
      if (part) {
        dw = sum_positions<LP>(dw);
        db = sum_positions<LP>(db);
        if (pl == 0 && e < E) {
          part[e] = dw;
          part[E + e] = db;
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  });
  if constexpr (MANY) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c1[i] += s1[i].value();
      c2[i] += s2[i].value();
    }
  }
  if (!p.rms) sum_groups<NT, LP>(c1, sm);
  sum_groups<NT, LP>(c2, sm);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    c1[k] = p.rms ? 0.0f : c1[k] * p.inv_e;
    c2[k] *= p.inv_e;
  }
  pass(true, [&](const Ch& k, int e0) {
    channels(e0, [&](int c, int e, int64_t at) {
      if (e >= E) return;
      float g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = (k.h[c].at(i) - m[i]) * r[i];
        g[i] = r[i] * (k.d[c].at(i) * k.w[c] - c1[i] - x * c2[i]);
      }
      if (p.dhidden) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] += k.q[c].at(i);
      }
      if (p.hidden) store_cols(static_cast<HT*>(p.hidden) + at, n, g, lines);
      if (p.out) {
        if (drop.any()) drop.apply(drop.kept((uint64_t)at), g);
        store_cols(static_cast<XT*>(p.out) + at, n, g, lines);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  });
}

// The same for tiles of 64 positions by 1024 lanes that keep what they can of C channels each, all there are: dout in
// registers, hidden of the first HL in LDS (up to 128 KB; each lane its own pieces), the others' is read again (2^17
// positions x 1024 channels, RMS norm in bf16: 262 us, with all of hidden read again 279; 16384 x 2048: 66.5 and 70).
// RMS is the template's for its registers: C = 16 fits them, and not with m and c1 beside them.
template <typename XT, typename HT, bool RMS, int C>
__global__ __launch_bounds__(1024) void norm_cols_bwd_keep_kernel(NormParams p) {
  constexpr int NT = 1024, LP = 8, NG = NT / LP, T = LP * 8, QH = (int)sizeof(HT) / 2;
  constexpr int HL = C < 16 / (int)sizeof(HT) ? C : 16 / (int)sizeof(HT);
  __shared__ float sm[(NT / 64 + 1) * T];
  __shared__ u32x4a own[HL * QH][NT];
  const int pl = threadIdx.x % LP, cg = threadIdx.x / LP, E = (int)p.E;
  const bool lines = p.L % 64 == 0;
  const int64_t tiles = (p.L + T - 1) / T, step = NG * p.L, tile = tile_id(p.blocks, lines);
  if (tile < 0) return;
  const Drop drop(p.drop);
  float* part = p.part ? p.part + tile * 2 * p.E : nullptr;
  const int64_t b = tile / tiles, t = tile % tiles * T + pl * 8;
  const bool in = t < p.L;
  const int64_t base = b * p.E * p.L + t;
  Piece<XT> d[C];
  Piece<HT> h[2];
  float w[2];
  int e0 = cg;
  asm volatile("" : "+v"(e0));
  int64_t at0 = base + e0 * p.L;
  auto side = [&](int e) { return p.weight ? p.weight[e < E ? e : 0] : 1.0f; };
  auto hidden = [&](int c, bool again) {
    h[c & 1].full(static_cast<const HT*>(p.residual) + at0 + c * step, in && e0 + c * NG < E, again);
  };
#pragma unroll
  for (int c = 0; c < C; ++c) d[c].full(static_cast<const XT*>(p.x) + at0 + c * step, in && e0 + c * NG < E);
  hidden(0, 0 >= HL);
  w[0] = side(e0);
  float m[8], r[8], c1[8], c2[8];
  if (!RMS) load_n<float, 8>(p.stats + b * p.L + t, in ? 8 : 0, m);
  load_n<float, 8>(p.stats + p.rows + b * p.L + t, in ? 8 : 0, r);
#pragma unroll
  for (int k = 0; k < 8; ++k) c1[k] = c2[k] = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (c + 1 < C) {
      hidden(c + 1, c + 1 >= HL);
      w[(c + 1) & 1] = side(e0 + (c + 1) * NG);
    }
    const Piece<HT>& now = h[c & 1];
    float dw = 0.0f, db = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float g = d[c].at(i), x = (RMS ? now.at(i) : now.at(i) - m[i]) * r[i], gw = g * w[c & 1];
      dw = __builtin_fmaf(g, x, dw);
      db += g;
      if (!RMS) c1[i] += gw;
      c2[i] = __builtin_fmaf(gw, x, c2[i]);
      if (!RMS) here(c1[i]);
      here(c2[i]);
    }
    if (c < HL) {
#pragma unroll
      for (int q = 0; q < QH; ++q) own[(c < HL ? c : 0) * QH + q][threadIdx.x] = now.w[q];
    }
    if (part) {
      dw = sum_positions<LP>(dw);
      db = sum_positions<LP>(db);
      const int e = e0 + c * NG;
      if (pl == 0 && e < E) {
        part[e] = dw;
        part[E + e] = db;
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) d[c].forget();
  // the second pass asks for its first pieces before the sums
  Piece<HT> q[2];
  e0 = cg;
  asm volatile("" : "+v"(e0));
  at0 = base + e0 * p.L;
  auto second = [&](int c) {
    const bool may = in && e0 + c * NG < E;
    if (p.dhidden) q[c & 1].full(static_cast<const HT*>(p.dhidden) + at0 + c * step, may);
    if (c >= HL) hidden(c, false);
    w[c & 1] = side(e0 + c * NG);
  };
  second(0);
  if (!RMS) sum_groups<NT, LP>(c1, sm);
  sum_groups<NT, LP>(c2, sm);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    c1[k] *= p.inv_e;
    c2[k] *= p.inv_e * r[k];
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (c + 1 < C) second(c + 1);
    const int e = e0 + c * NG;
    Piece<HT> now = h[c & 1];
    if (c < HL) {
#pragma unroll
      for (int k = 0; k < QH; ++k) now.w[k] = own[(c < HL ? c : 0) * QH + k][threadIdx.x];
    }
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g[i] = d[c].at(i) * w[c & 1] - (RMS ? now.at(i) : now.at(i) - m[i]) * c2[i];
      g[i] = r[i] * (RMS ? g[i] : g[i] - c1[i]);
      if (p.dhidden) g[i] += q[c & 1].at(i);
    }
    const int64_t at = at0 + c * step;
    if (in && e < E) {
      if (p.hidden) store_cols(static_cast<HT*>(p.hidden) + at, 8, g, lines);
      if (p.out) {
        if (drop.any()) drop.apply(drop.kept((uint64_t)at), g);
        store_cols(static_cast<XT*>(p.out) + at, 8, g, lines);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

namespace {

// Channels that a lane keeps: of 512 lanes they fill 128 registers each.
template <typename XT, typename HT, bool RES> constexpr int kept_channels() {
  constexpr int regs = 2 * (int)sizeof(XT) + (RES ? 2 * (int)sizeof(HT) : 0);  // of one
  return regs <= 4 ? 32 : regs <= 8 ? 16 : 8;
}

template <typename XT, typename HT, bool RES, bool DROP, bool ODD, int NT, int LP, int C, bool KEEP, bool MANY = false>
void go(const NormParams& p, hipStream_t s) {
  hipLaunchKernelGGL((norm_cols_kernel<XT, HT, RES, DROP, ODD, NT, LP, C, KEEP, MANY>),
                     grid_of(p.B * ((p.L + LP * 8 - 1) / (LP * 8))), dim3(NT), 0, s, p);
}

// Everything read again for each pass, in tiles of T = 16, 64 or 256 positions (of very many channels, 16 or 64).
template <typename XT, typename HT, bool RES, bool DROP, bool ODD>
void again(const NormParams& p, int T, hipStream_t s) {
  if (p.E > kManyChannels)
    T == 16 ? go<XT, HT, RES, DROP, ODD, 512, 2, 2, false, true>(p, s)
            : go<XT, HT, RES, DROP, ODD, 512, 8, 2, false, true>(p, s);
  else if (T == 16) go<XT, HT, RES, DROP, ODD, 512, 2, 2, false>(p, s);
  else if (T == 64) go<XT, HT, RES, DROP, ODD, 512, 8, 2, false>(p, s);
  else go<XT, HT, RES, DROP, ODD, 512, 32, 2, false>(p, s);
}

// With a residual, channels that do not fit the registers: x alone does (4 x 4096 positions x 2048 channels in bf16: 75
// us, everything read again 81; 2^17 x 2048: 521 and 625; 2^18 x 512 with dropout: 281 and 308; 8 x 2048 x 768 with
// dropout into fp32: 40 and 45).
template <typename XT> constexpr int keep_most() { return sizeof(XT) == 2 ? 16 : 8; }

template <typename XT, typename HT>
void keep_fwd(const NormParams& p, hipStream_t s) {
  auto go = [&](auto c) {
    hipLaunchKernelGGL((norm_cols_keep_kernel<XT, HT, decltype(c)::value>), grid_of(p.B * ((p.L + 63) / 64)), dim3(1024),
                       0, s, p);
  };
  const int64_t c = (p.E + 127) / 128;
  c <= 2 ? go(IC<2>()) : c <= 4 ? go(IC<4>()) : c <= 8 ? go(IC<8>()) : go(IC<keep_most<XT>()>());
}

// Wide tiles read and write longer pieces of the rows, which lie far apart (2^17 positions x 1024 channels in bf16: 125
// us with 64 positions, 114 with 128; 2^18 x 512: 122, 112, and 105 with 256), but hold fewer channels and leave compute
// units idle where there are few of them.  With few tiles of 64 positions they are cut to 16, and what is kept gains
// nothing then (8 x 512 positions x 768 channels with a residual: 9.8 us, kept 9.8, 64 positions and kept 14.6).
template <typename XT, typename HT, bool RES, bool ODD>
void fwd_of(const NormParams& p, hipStream_t s) {
  constexpr int C = kept_channels<XT, HT, RES>();
  const bool wide = p.L >= 128 && p.B * ((p.L + 127) / 128) >= 512;
  const int T = norm_cols_narrow(p.B, p.E, p.L) ? 16 : wide && p.L >= 256 ? 256 : 64;  // of what is read again
  if (T == 16) {
    if (p.drop.below) return again<XT, HT, RES, true, ODD>(p, T, s);
    return again<XT, HT, RES, false, ODD>(p, T, s);
  }
  if constexpr (RES && !ODD) {
    if (p.E >= 128 && p.E <= 128 * keep_most<XT>() && (p.drop.below || p.E > 64 * C)) return keep_fwd<XT, HT>(p, s);
  }
  if (p.drop.below) return again<XT, HT, RES, true, ODD>(p, T, s);
  if (p.E <= 16 * (C / 4)) return go<XT, HT, RES, false, ODD, 256, 16, C / 4, true>(p, s);
  if (wide && p.E <= 32 * (C / 4)) return go<XT, HT, RES, false, ODD, 512, 16, C / 4, true>(p, s);
  if (p.E <= 64 * (C / 4)) return go<XT, HT, RES, false, ODD, 512, 8, C / 4, true>(p, s);
  if (wide && p.E <= 32 * C) return go<XT, HT, RES, false, ODD, 512, 16, C, true>(p, s);
  if (p.E <= 64 * C) return go<XT, HT, RES, false, ODD, 512, 8, C, true>(p, s);
  again<XT, HT, RES, false, ODD>(p, T, s);
}

template <typename XT, typename HT, bool RES>
void fwd(const NormParams& p, hipStream_t s) {
  p.L % 8 ? fwd_of<XT, HT, RES, true>(p, s) : fwd_of<XT, HT, RES, false>(p, s);
}

template <typename XT, typename HT, bool ODD, int NT, int LP, int C, bool MANY = false>
void go_bwd(const NormParams& p, hipStream_t s) {
  hipLaunchKernelGGL((norm_cols_bwd_kernel<XT, HT, ODD, NT, LP, C, MANY>), grid_of(p.blocks), dim3(NT), 0, s, p);
}

template <typename XT, typename HT, bool RMS>
void keep_bwd(const NormParams& p, hipStream_t s) {
  constexpr int most = norm_cols_bwd_kept(sizeof(XT) == 2, sizeof(HT) == 2, RMS) / 128;
  auto go = [&](auto c) {
    if constexpr (decltype(c)::value <= most)
      hipLaunchKernelGGL((norm_cols_bwd_keep_kernel<XT, HT, RMS, decltype(c)::value>), grid_of(p.blocks), dim3(1024), 0,
                         s, p);
  };
  const int64_t c = (p.E + 127) / 128;
  c <= 2 ? go(IC<2>()) : c <= 4 ? go(IC<4>()) : c <= 8 && c <= most ? go(IC<(most < 8 ? most : 8)>()) : go(IC<most>());
}

template <typename XT, typename HT>
void bwd(const NormParams& p, hipStream_t s) {
  const int kind = (sizeof(XT) == 2 ? 1 : 0) + (sizeof(HT) == 2 ? 2 : 0);
  const NormTile tile = norm_cols_bwd_tile(p.B, p.E, p.L, kind, p.rms);
  if (tile.keep) return p.rms ? keep_bwd<XT, HT, true>(p, s) : keep_bwd<XT, HT, false>(p, s);
  if (p.E > kManyChannels) {
    if (tile.T == 16)
      return p.L % 8 ? go_bwd<XT, HT, true, 512, 2, 2, true>(p, s) : go_bwd<XT, HT, false, 512, 2, 2, true>(p, s);
    return p.L % 8 ? go_bwd<XT, HT, true, 512, 8, 2, true>(p, s) : go_bwd<XT, HT, false, 512, 8, 2, true>(p, s);
  }
  if (p.L % 8) {
    if (tile.T == 16) return go_bwd<XT, HT, true, 512, 2, 2>(p, s);
    return tile.T > 64 ? go_bwd<XT, HT, true, 512, 16, 2>(p, s) : go_bwd<XT, HT, true, 512, 8, 2>(p, s);
  }
  if (tile.T == 256) return go_bwd<XT, HT, false, 512, 32, 2>(p, s);
  if (tile.T == 128) return go_bwd<XT, HT, false, 512, 16, 2>(p, s);
  if (tile.T == 16) return go_bwd<XT, HT, false, 512, 2, 2>(p, s);
  go_bwd<XT, HT, false, 512, 8, 2>(p, s);
}

}  // namespace

}  // namespace ssm
