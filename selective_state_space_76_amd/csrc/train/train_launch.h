// train_launch.h -- internal interface between the training operators' C entry points
// (train_abi.cpp) and their gfx950 kernels.  Not installed; not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm {

// A launch takes fewer than 2^32 threads in x; workgroups (of up to 1024) beyond kGridX go on in y.  A kernel knows its workgroup by
// block_id() (train_device.h); the last row of y may hold some past the last one.
constexpr int64_t kGridX = int64_t(1) << 21;
inline dim3 grid_of(int64_t blocks) {
  const int64_t x = blocks < kGridX ? blocks : kGridX;
  return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}

// ---- gradients of conv1d + SiLU (conv_bwd.hip)
struct ConvBwdParams {
  const void* x;        // [B,D,L]
  const float* w;       // [D,K]
  const float* bias;    // [D] or null
  const void* init;     // [B,D,K-1] or null (zeros)
  const void* dout;     // [B,D,L]
  const void* dfinal;   // [B,D,K-1] or null (zeros)
  void* dx;             // [B,D,L]
  void* dinit;          // [B,D,K-1] or null
  float* dw;            // [D,K]
  float* db;            // [D] or null
  float* part;          // [B*S][D][K+1]: dweight and dbias summed over one segment of one row
  int64_t Bsz, Dm, L;
  int64_t S;            // segments per row
  uint32_t units;       // segments of all rows, below 2^31
  int K;
  int lanes;            // lanes per row segment, 16 or 64
};
int64_t conv_bwd_segments(int64_t L, bool bf16, int* lanes);
hipError_t launch_conv_bwd(const ConvBwdParams& p, bool bf16, hipStream_t s);

// ---- AdamW (adamw.hip)
constexpr int kAdamBlock = 128;
constexpr int kAdamTensors = 80;  // tensors per launch: their table travels in the kernel arguments (3.3 KB)
constexpr int64_t kAdamChunk = 8192;  // elements per workgroup
constexpr int kNormTensors = 192;  // as many with less to say of each
constexpr int64_t kNormChunk = 16384;

struct AdamTable {
  void* p[kAdamTensors];
  const void* g[kAdamTensors];
  int64_t n[kAdamTensors];
  int64_t off[kAdamTensors];
  uint32_t first[kAdamTensors];  // workgroup that a tensor begins with
  uint32_t key[kAdamTensors];    // of its random numbers
  int count;
};

struct NormTable {
  const void* g[kNormTensors];
  int64_t n[kNormTensors];
  uint32_t first[kNormTensors];
  int count;
};

constexpr int kSmallTensors = 64, kSmallChunks = 64;  // what one workgroup sums up by itself
constexpr int64_t kSmallChunk = 2048;
struct SmallNormTable {
  const void* g[kSmallTensors];
  int64_t n[kSmallTensors];
  uint32_t first[kSmallTensors];
  uint8_t bf16[kSmallTensors];
  int count;
};

// A clipped step's numbers, on the device: the last kernel of the norm counts the step and writes them, where the norm
// is finite; the step's own kernels read them.  (struct ssm_adamw_progress.)
struct AdamProgress {
  int64_t step;             // steps made
  float factor;             // of the gradients; NaN: nothing changes
  float size, isb;          // lr / (1 - b1^step), 1 / sqrt(1 - b2^step)
  uint32_t key;             // hash of seed and step
  uint32_t unused[2];
};
struct AdamAdvance {
  AdamProgress* progress;   // null: the norm alone
  double lr, b1, b2;
  uint32_t seed;            // hashed
};

struct AdamParams {
  void* m;
  void* v;
  int16_t* mb;
  int16_t* vb;
  float* master;
  const float* clip;   // {norm, factor} or null
  const AdamProgress* progress;  // or null: then clip and what follows; with it a table's keys are the tensors' numbers
  float b1, c1, b2, c2, eps, isb, step, decay;
};

// of a tensor: a hash of the seed, the step and its place in the list
uint32_t adam_key(uint64_t seed, int64_t step, int64_t tensor);
uint32_t adam_seed(uint64_t seed);  // its part that is of the seed
// kind: bit 0 bf16 params, bit 1 bf16 gradients, bit 2 master weights, bit 3 8-bit states
hipError_t launch_adamw(const AdamTable& t, const AdamParams& p, int kind, uint32_t blocks, hipStream_t s);
hipError_t launch_norm_part(const NormTable& t, double* part, bool bf16, uint32_t blocks, hipStream_t s);
hipError_t launch_norm_small(const SmallNormTable& t, uint32_t chunks, double max_norm, float* result,
                             const AdamAdvance& adv, hipStream_t s);
hipError_t launch_norm_join(const double* part, int64_t n, double max_norm, float* result, const AdamAdvance& adv,
                            hipStream_t s);
hipError_t launch_state_values(int64_t n, const void* m, const void* v, const int16_t* mb, const int16_t* vb,
                               void* mo, void* vo, hipStream_t s);

// ---- embedding (embed_fwd.hip, embed_bwd.hip)
struct EmbedParams {
  const void* tokens;
  const void* table;   // weight (forward)
  void* out;           // out (forward), dweight (backward)
  const void* dout;
  int64_t Bsz, L, V, E, T;
  float scale;
  int i64;             // tokens are int64
  int cf;              // [B,E,L]
  int add;
  int64_t tiles;       // [B,E,L] forward: tiles along a row
};
hipError_t launch_embed_fwd(const EmbedParams& p, bool table_bf16, bool io_bf16, hipStream_t s);

struct EmbedBwdPlan {
  bool few = false;               // [B,E,L], few rows, not too short: products (embed_bwd_few.hip); run: positions per segment
  bool transpose = false;         // [B,E,L]: dout is brought to [B,L,E] first
  bool once = false;              // short lists: all steps in one launch, no workspace but the turned dout
  int bits = 0, passes = 0, digit_bits = 0;
  int64_t tile = 0, tiles = 0;    // of the sort; one tile: one launch
  int64_t run = 0, chunks = 0;    // sorted rows per chunk of the sums
  size_t rows = 0, key[2] = {0, 0}, pos[2] = {0, 0}, hist = 0, part = 0, total = 0;  // offsets, bytes
};
void plan_embed_bwd(int64_t Bsz, int64_t L, int64_t V, int64_t E, int64_t table_size, bool io_bf16, bool cf, bool add,
                    EmbedBwdPlan* pl);
hipError_t launch_embed_bwd(const EmbedParams& p, const EmbedBwdPlan& pl, bool table_bf16, bool io_bf16, void* ws,
                            hipStream_t s);
bool embed_few_pays(int64_t Bsz, int64_t L, int64_t V, int64_t E, bool io_bf16);
void plan_embed_few(int64_t Bsz, int64_t L, int64_t V, int64_t E, EmbedBwdPlan* pl);
hipError_t launch_embed_few(const EmbedParams& p, const EmbedBwdPlan& pl, bool table_bf16, bool io_bf16, void* ws,
                            hipStream_t s);

}  // namespace ssm
