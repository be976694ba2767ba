// block_launch.h -- internal interface between the residual block's C entry points (block_abi.cpp) and their
// gfx950 kernels: layer norm, dropout, the gated linear recurrence.  Not installed; not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../train/train_launch.h"

namespace ssm {

// ---- dropout (block_device.h, dropout.hip): what a kernel needs to know of a mask
struct DropParams {
  const int64_t* device_seed;  // the seed on the device, or null: then `seed`
  uint64_t seed, call;
  uint32_t below;              // elements whose 16 bits are below this are dropped; 0: no dropout
  float scale;                 // of the others
};

struct DropoutParams {
  const void* x;
  const void* residual;  // or null
  void* out;
  int64_t n;
  DropParams drop;
};
hipError_t launch_dropout(const DropoutParams& p, bool x_bf16, bool out_bf16, hipStream_t s);

// ---- layer norm (norm_rows.hip: [rows, E]; norm_cols_kernel.h: [B, E, L])
struct NormParams {
  const void* x;         // forward; backward: dout
  const void* residual;  // forward, or null; backward: hidden
  const float* weight;   // or null (ones)
  const float* bias;     // forward, or null
  void* out;             // forward; backward: dx, or null
  void* hidden;          // forward, or null; backward: dresidual, or null
  const void* dhidden;   // backward, or null
  float* stats;          // [2][rows]: means and factors; forward: or null
  float* part;           // backward: [blocks][2][E] partial sums of dweight and dbias, or null
  float* dweight;        // backward, or null
  float* dbias;
  int64_t rows, E, B, L;
  int64_t blocks;        // backward: workgroups, each with its partial sums
  int64_t from, to;      // backward, rows of a launch
  float eps, inv_e;
  int rms;
  DropParams drop;
};
// kind: bit 0 bf16 x, bit 1 bf16 hidden
hipError_t launch_norm_rows(const NormParams& p, int kind, hipStream_t s);
hipError_t launch_norm_cols_bf16(const NormParams& p, hipStream_t s);  // x and hidden
hipError_t launch_norm_cols_mixed(const NormParams& p, hipStream_t s);  // x in bf16, hidden in fp32
hipError_t launch_norm_cols_f32(const NormParams& p, hipStream_t s);
hipError_t launch_norm_cols_bwd_bf16(const NormParams& p, hipStream_t s);
hipError_t launch_norm_cols_bwd_mixed(const NormParams& p, hipStream_t s);
hipError_t launch_norm_cols_bwd_f32(const NormParams& p, hipStream_t s);
inline hipError_t launch_norm_cols(const NormParams& p, int kind, hipStream_t s) {
  return kind == 3 ? launch_norm_cols_bf16(p, s) : kind == 1 ? launch_norm_cols_mixed(p, s) : launch_norm_cols_f32(p, s);
}
inline hipError_t launch_norm_cols_bwd(const NormParams& p, int kind, hipStream_t s) {
  return kind == 3 ? launch_norm_cols_bwd_bf16(p, s) : kind == 1 ? launch_norm_cols_bwd_mixed(p, s)
                                                                 : launch_norm_cols_bwd_f32(p, s);
}
int64_t norm_rows_bwd_blocks(int64_t rows, int64_t E);
// Over [B, E, L]: tiles of 16 positions, lines shared through the caches, where there are few of 64, or where rows are so
// short that most lanes of those would have none (4096 x 768 x 8 in bf16 with a residual: 71 us, 187 in tiles of 64; but
// few channels leave more lanes without any: 65536 x 16 x 8: 355 and 186).
inline bool norm_cols_narrow(int64_t B, int64_t E, int64_t L) {
  return B * ((L + 63) / 64) < 128 || (L <= 32 && E >= 256);
}
// With more channels than these, tiles of 16 or 64 positions whose lanes add up blocks of 128 channels (a lane has up to
// 2^24 of them); with as many, a lane's share is 1024 at the most.
constexpr int64_t kManyChannels = 16384;
// The backward pass there: a workgroup and a partial sum of dw and db for each tile.
// Channels up to which a tile of 64 positions keeps dout between its two passes, as far as 128 registers go.
constexpr int norm_cols_bwd_kept(bool x16, bool h16, bool rms) {
  return 128 * (!x16 ? (rms ? 8 : 6) : !h16 ? 8 : rms ? 16 : 12);
}
struct NormTile {
  int T;      // positions
  bool keep;  // dout is kept
};
// Kept dout spares a reading, but takes 128 channels to fill its lanes (RMS norm in bf16 with the stream's own gradient;
// 2^17 positions x 1024 channels: 263 us, read twice 312 in tiles of 64 positions, 323 in tiles of 256; 2^17 x 2048:
// 562, 712 and 643; 16384 x 2048: 67 and 78; 2^19 x 128: 114, 145 and 129; 2^20 x 64: 173, 220 and 138).  Read twice, wide
// tiles are better where there are enough of them (2^15 x 4096: 317 us with 128 positions, 375 with 64, 404 with 256).
inline NormTile norm_cols_bwd_tile(int64_t B, int64_t E, int64_t L, int kind, bool rms) {
  auto tiles = [&](int64_t T) { return B * ((L + T - 1) / T); };
  if (norm_cols_narrow(B, E, L)) return {16, false};
  if (E > kManyChannels) return {64, false};
  if (L % 8) return {L >= 128 && tiles(128) >= 256 ? 128 : 64, false};
  if (E >= 128 && E <= norm_cols_bwd_kept(kind & 1, kind & 2, rms)) return {64, true};
  return {L >= 256 && tiles(256) >= 512 ? 256 : L >= 128 && tiles(128) >= 256 ? 128 : 64, false};
}
inline int64_t norm_cols_bwd_blocks(int64_t B, int64_t E, int64_t L, int kind, bool rms) {
  const int T = norm_cols_bwd_tile(B, E, L, kind, rms).T;
  return B * ((L + T - 1) / T);
}
hipError_t launch_norm_rows_bwd(const NormParams& p, int kind, hipStream_t s);

// ---- the sums of partial sums (join.hip); part is overwritten where there are more than 4096
struct JoinParams {
  float* part;      // [count][kinds][E]
  int64_t count, E;
  int kinds;        // 2 or 3
  float* out[3];    // [E] each, or null
};
hipError_t launch_join(const JoinParams& p, hipStream_t s);

// ---- gated linear recurrence (recur_fwd.hip, recur_bwd.hip)
struct RecurPlan {
  int lanes = 64;       // lanes per row: 1, 4, 16, 32 or 64
  int waves = 1;        // waves that share a row: 1, 4 or 8
  int64_t S = 1;        // segments of a row
  int64_t blocks = 0;   // blocks of 64 pieces in a row, each with a checkpoint
  int64_t tiles = 0;    // turns of a row's team
  int64_t per = 0;      // tiles in a segment
  int chain = 0;        // backward: turns that a lane adds up before they become a partial sum
  int parts = 1;        // such sums of a segment
};
RecurPlan recur_plan(int64_t B, int64_t D, int64_t L, bool bf16);

struct RecurParams {
  const void* x;      // [B,D,L]
  const void* r;
  const void* i;
  const void* z;      // or null
  const float* decay; // [D]
  const float* rb;    // [D] or null (zeros)
  const float* ib;
  const float* init;  // [B,D] or null (zeros)
  void* out;          // forward; null: checkpoints only
  float* last;        // [B,D] or null
  float* ckpt;        // [B,D,blocks]: written by the forward pass (or null), read by the backward
  float* seg;         // [S][B*D][2]: what a segment makes of the state that enters it, S > 1
  // backward
  const void* dout;
  const float* dlast; // [B,D] or null (zeros)
  void* dx;
  void* dr;
  void* di;
  void* dz;           // with z
  float* dinit;       // [B,D] or null
  float* part;        // [B*S*waves*parts][3][D]
  float* ddecay;      // [D]
  float* drb;         // or null
  float* dib;
  int64_t B, D, L;
  bool whole;         // backward: a team has all of a channel and joins its sums itself
  RecurPlan plan;
};
hipError_t launch_recur_fwd(const RecurParams& p, bool bf16, bool reverse, hipStream_t s);
hipError_t launch_recur_bwd(const RecurParams& p, bool bf16, bool reverse, hipStream_t s);

struct RecurStepParams {
  float* state;       // [B,D]
  const void* x;      // [B,D]
  const void* r;
  const void* i;
  const void* z;      // or null
  const float* decay;
  const float* rb;
  const float* ib;
  void* out;
  int64_t n, D;
};
hipError_t launch_recur_step(const RecurStepParams& p, bool bf16, hipStream_t s);

}  // namespace ssm
