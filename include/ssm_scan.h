/*
 * ssm_scan.h -- C ABI of libssmscan.so, the MI355X (gfx950) selective state-space scan.
 *
 * The operation (per batch b, channel d, state n, step t) is the selective SSM
 * recurrence that the pages describe:
 *   dt      = softplus(delta[b,d,t] + delta_bias[d])   -- step size from the input,
 *             bias inside the softplus ("Mamba: 基于选择状态空间的线性时间序列模型",
 *             freeguideonline.com, section 4.2 step 2; fsdata.site
 *             "mamba-state-space-model" article, section 3.2)
 *   A_bar   = exp(dt * A[d,n])                          -- fsdata.site article, section 3.2
 *   B_bar   = dt * B[b,n,t]                             -- same section (default)
 *           = (exp(dt*A) - 1) / A * B[b,n,t]            -- exact zero-order hold, with
 *             SSM_FLAG_ZOH (freeguideonline tutorial, section 2.2)
 *   h[n]    = A_bar * h[n] + B_bar * u[b,d,t]
 *   y       = sum_n C[b,n,t] * h[n] + D[d] * u[b,d,t]   -- output read from the updated
 *             state plus the skip term ("Mamba: Linear-Time Sequence Modeling with
 *             Selective State Spaces", ai.xwebgame.com, section on what an SSM is)
 *   out     = y * silu(z[b,d,t])                        -- gate by the second branch
 *             (same page, the PyTorch block's gating step)
 * Each channel d is an independent SSM with its own diagonal A[d,:]
 * (freeguideonline tutorial, section 4.3); B and C are shared by all channels of
 * a batch row.  The scan computes the sequential recurrence exactly up to
 * floating-point rounding order (freeguideonline tutorial, section 5.1).  The
 * state is fp32; streams are fp32 or bf16 (rounded to nearest even on output).
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller (the library
 *     allocates nothing and keeps no pointer after returning).  Tensors are
 *     dense, row-major, with the layouts given below, and every base pointer
 *     must be 16-byte aligned.
 *   - Work is enqueued asynchronously on `stream` (a hipStream_t; NULL is the
 *     null stream).  Outputs are valid once the stream has been synchronised.
 *   - Every argument is checked on the host before anything is enqueued; on any
 *     error nothing is launched and no output is touched.  The return code is
 *     the only error channel.
 *   - `out` and `final_state` must not overlap any input (checked: SSM_ERR_OVERLAP).
 *   - Calls are reentrant; concurrent calls on different streams are safe when
 *     their output buffers are distinct.
 *   - Indexing is 64-bit: a tensor may hold more than 2^31 elements.
 *   - Arithmetic is fp32: a result whose exact magnitude is below about 1e-36
 *     (near or under fp32's smallest normal number) may come back as 0.
 */
#ifndef SSM_SCAN_H
#define SSM_SCAN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct ihipStream_t; /* hipStream_t is `struct ihipStream_t*` */

typedef enum ssm_status {
  SSM_OK = 0,
  SSM_ERR_NULL = 1,        /* a required pointer is NULL */
  SSM_ERR_SHAPE = 2,       /* a size is out of range (batch/dim/seqlen < 1, dstate not in [1,64],
                              conv width not in [1,4]) */
  SSM_ERR_DTYPE = 3,       /* io_dtype is not SSM_F32 or SSM_BF16 */
  SSM_ERR_ALIGN = 4,       /* a base pointer is not 16-byte aligned */
  SSM_ERR_UNSUPPORTED = 5, /* unknown flag bits */
  SSM_ERR_WORKSPACE = 6,   /* workspace non-NULL but smaller than ssm_scan_workspace_size() */
  SSM_ERR_LAUNCH = 7,      /* the HIP runtime rejected a launch (hipGetLastError) */
  SSM_ERR_OVERLAP = 8,     /* an output buffer overlaps an input buffer */
  SSM_ERR_TOO_LARGE = 9    /* ssm_scan_fwd_noalloc: the shape needs more than its 34 MiB of scratch */
} ssm_status;

typedef enum ssm_dtype { SSM_F32 = 0, SSM_BF16 = 1 } ssm_dtype;

/* flag bits for ssm_shape.flags / ssm_state_update(flags) */
#define SSM_FLAG_ZOH 1u     /* exact zero-order-hold B_bar instead of dt*B */
#define SSM_FLAG_REVERSE 2u /* scan from t = L-1 down to 0 (a backward-in-time SSM;
                               fsdata.site article, section 7 pitfalls table) */

typedef struct ssm_shape {
  int64_t batch;   /* B >= 1 */
  int64_t dim;     /* D (d_inner) >= 1 */
  int64_t dstate;  /* N in [1, 64] */
  int64_t seqlen;  /* L >= 1 */
  int32_t io_dtype;/* ssm_dtype of u, delta, B, C, z and out */
  uint32_t flags;  /* SSM_FLAG_* bits */
} ssm_shape;

/* Version of this header's ABI (bumped on any incompatible change). */
#define SSM_ABI_VERSION 2
int ssm_abi_version(void);

/* Static string for a status code (never NULL). */
const char* ssm_status_str(int status);

/* Bytes of device workspace that ssm_scan_fwd may use for this shape to split
 * long sequences across workgroups (0 when no split is used).  Depends on the
 * shape only.  Returns 0 for an invalid shape. */
size_t ssm_scan_workspace_size(const ssm_shape* shape);

/* Selective scan over a whole sequence (prefill / training forward).
 *   u, delta, z, out : [B, D, L]  io_dtype
 *   A                : [D, N]     fp32 (the pages use negative reals)
 *   B, C             : [B, N, L]  io_dtype, shared by all D channels of a batch row
 *   D, delta_bias    : [D]        fp32, NULL means zero
 *   z                : NULL means no gate (out = y)
 *   initial_state    : [B, D, N]  fp32 state before the first processed step,
 *                      NULL means zero (lets a long sequence be scanned in
 *                      several calls; mlqm.cn article, section 6.2)
 *   final_state      : [B, D, N]  fp32 state after the last processed step,
 *                      NULL means not written
 *   workspace        : device scratch of workspace_bytes; NULL with 0 bytes runs
 *                      without splitting the sequence (always correct, slower when
 *                      batch*dim is small).  Non-NULL but smaller than
 *                      ssm_scan_workspace_size() is SSM_ERR_WORKSPACE.  The
 *                      library does not keep it; its contents are not preserved.
 * With SSM_FLAG_REVERSE the steps run from L-1 to 0; final_state is then the
 * state after step 0. */
ssm_status ssm_scan_fwd(const ssm_shape* shape,
                        const void* u, const void* delta, const float* A,
                        const void* B, const void* C, const float* D,
                        const void* z, const float* delta_bias,
                        const float* initial_state,
                        void* out, float* final_state,
                        void* workspace, size_t workspace_bytes,
                        struct ihipStream_t* stream);

/* ssm_scan_fwd that also saves what ssm_scan_bwd_saved needs, so a training step does
 * not recompute it:
 *   checkpoints      : [B, ceil(L/64), D, N] fp32, written: the state entering every
 *                      64-step block (block k starts at step 64 k in scan order).
 *                      Required; must not overlap any other argument.
 * Every other argument, the outputs and the errors are those of ssm_scan_fwd. */
ssm_status ssm_scan_fwd_save(const ssm_shape* shape,
                             const void* u, const void* delta, const float* A,
                             const void* B, const void* C, const float* D,
                             const void* z, const float* delta_bias,
                             const float* initial_state,
                             void* out, float* final_state, float* checkpoints,
                             void* workspace, size_t workspace_bytes,
                             struct ihipStream_t* stream);

/* ssm_scan_fwd for callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): it takes no workspace
 * and allocates nothing.  A sequence split uses a scratch array of 34 MiB that the
 * library holds in static device memory, one copy per GPU, kept until the process
 * ends (it holds the split of 1 x 1024 x 16 x 2^20, bf16, which needs 33.996 MiB);
 * its address is looked up once per device, on the first call there.
 *   - Arguments, outputs and errors are those of ssm_scan_fwd, with the split always
 *     enabled; a shape whose split needs more than 34 MiB (ssm_scan_workspace_size()
 *     > 34 MiB) is refused with SSM_ERR_TOO_LARGE before anything is enqueued.
 *   - `stream` must belong to the device whose scratch is used (its own device).
 *   - Every call on one GPU shares that GPU's scratch, which keeps the last call's
 *     contents: calls that overlap in time on one GPU (on different streams, or
 *     from different host threads without ordering) race on it and give undefined
 *     results.  Serialise them, e.g. on one stream.
 * Results are bitwise those of ssm_scan_fwd with a workspace. */
ssm_status ssm_scan_fwd_noalloc(const ssm_shape* shape,
                                const void* u, const void* delta, const float* A,
                                const void* B, const void* C, const float* D,
                                const void* z, const float* delta_bias,
                                const float* initial_state,
                                void* out, float* final_state,
                                struct ihipStream_t* stream);

/* One recurrent generation step (the scan body with L = 1), state updated in place:
 * the fixed-size state replaces a growing cache (fsdata.site article, section 3.2
 * and the comparison table in section 5).
 *   state            : [B, D, N]  fp32, read and written
 *   u, delta, z, out : [B, D]     io_dtype
 *   A                : [D, N]     fp32
 *   B, C             : [B, N]     io_dtype
 *   D, delta_bias    : [D]        fp32, NULL means zero; z NULL means no gate
 * flags: SSM_FLAG_ZOH only. */
ssm_status ssm_state_update(int64_t batch, int64_t dim, int64_t dstate, int32_t io_dtype,
                            uint32_t flags, float* state,
                            const void* u, const void* delta, const float* A,
                            const void* B, const void* C, const float* D,
                            const void* z, const float* delta_bias,
                            void* out, struct ihipStream_t* stream);

/* Bytes of device workspace ssm_scan_bwd needs for this shape (0 for an invalid
 * shape): block checkpoints of the state, B*D*ceil(L/64)*N fp32; per-workgroup
 * partial sums of dB and dC, 2*ceil(D/16)*B*N*L fp32; and the per-(segment,
 * batch row) partial sums of dA, dD and ddelta_bias.  When the shape has few
 * channels and a long sequence (fewer than 384 blocks of 16 channels over the batch
 * and L >= 2048) the sequence is split into S segments, as in the forward: then
 * also the carried states of the checkpoints and, per segment, the summary and the
 * carried value of the adjoint (O(S*B*D*N) fp32).  The choice depends on the shape
 * only. */
size_t ssm_scan_bwd_workspace_size(const ssm_shape* shape);

/* Gradients of ssm_scan_fwd (training backward pass).  The pages describe only the
 * forward recurrence; these are its exact derivatives by the chain rule (the
 * reverse-time adjoint recurrence), computed from the forward inputs alone: the
 * forward states are recomputed from checkpoints, nothing from the forward call
 * is needed.
 *   Inputs: the forward's inputs (same layouts, same NULL rules) plus
 *   dout             : [B, D, L] io_dtype, gradient of out
 *   dfinal_state     : [B, D, N] fp32 gradient of final_state, NULL means zero
 *   Outputs (all fully written):
 *   du, ddelta       : [B, D, L] io_dtype
 *   dA               : [D, N]    fp32, summed over batch rows and steps
 *   dB, dC           : [B, N, L] fp32, summed over channels
 *   dD, ddelta_bias  : [D]       fp32, NULL means not computed (written even when
 *                      D / delta_bias is NULL: the gradient at zero)
 *   dz               : [B, D, L] io_dtype, required when z is given, else ignored
 *   dinitial_state   : [B, D, N] fp32 gradient of initial_state, NULL means not written
 *   workspace        : required, at least ssm_scan_bwd_workspace_size() bytes
 * shape->flags may hold SSM_FLAG_REVERSE and SSM_FLAG_ZOH, as in the forward call
 * (under ZOH the derivatives of B_bar = (exp(dt A) - 1) / A * B with respect to dt, A,
 * B and u are taken, with the A -> 0 limit where A is zero).  No output may overlap an
 * input, another output or the workspace.  Every sum is taken in a fixed order, so
 * results are bitwise reproducible. */
ssm_status ssm_scan_bwd(const ssm_shape* shape,
                        const void* u, const void* delta, const float* A,
                        const void* B, const void* C, const float* D,
                        const void* z, const float* delta_bias,
                        const float* initial_state,
                        const void* dout, const float* dfinal_state,
                        void* du, void* ddelta, float* dA, float* dB, float* dC,
                        float* dD, void* dz, float* ddelta_bias, float* dinitial_state,
                        void* workspace, size_t workspace_bytes,
                        struct ihipStream_t* stream);

/* Bytes of device workspace ssm_scan_bwd_saved needs for this shape (0 for an invalid
 * shape): that of ssm_scan_bwd without the checkpoints and their split. */
size_t ssm_scan_bwd_saved_workspace_size(const ssm_shape* shape);

/* ssm_scan_bwd from the checkpoints that ssm_scan_fwd_save wrote for the same inputs
 * (same shape, flags, initial_state, A, B, delta, delta_bias and u), instead of a
 * checkpoint pass of its own:
 *   checkpoints      : [B, ceil(L/64), D, N] fp32, read only.  Required; must not
 *                      overlap an output or the workspace.
 *   workspace        : required, at least ssm_scan_bwd_saved_workspace_size() bytes
 * Every other argument, the outputs and the errors are those of ssm_scan_bwd. */
ssm_status ssm_scan_bwd_saved(const ssm_shape* shape,
                              const void* u, const void* delta, const float* A,
                              const void* B, const void* C, const float* D,
                              const void* z, const float* delta_bias,
                              const float* initial_state,
                              const void* dout, const float* dfinal_state,
                              const float* checkpoints,
                              void* du, void* ddelta, float* dA, float* dB, float* dC,
                              float* dD, void* dz, float* ddelta_bias, float* dinitial_state,
                              void* workspace, size_t workspace_bytes,
                              struct ihipStream_t* stream);

/* The step that produces u: causal depthwise conv1d over time, plus a bias, then
 * SiLU (ai.xwebgame.com Mamba page, the PyTorch block's step 2: a Conv1d with one
 * group per channel and width-1 padding whose output is cut to the sequence
 * length, followed by SiLU):
 *   u[b,d,t] = silu(bias[d] + sum_{k<width} weight[d,k] * x[b,d,t-(width-1)+k])
 * Inputs before step 0 are taken from initial_conv_state, else zero.
 *   x, u               : [B, D, L]        io_dtype
 *   weight             : [D, width]       fp32 (the page's Conv1d weight [D,1,width])
 *   bias               : [D]              fp32, NULL means zero
 *   initial_conv_state : [B, D, width-1]  io_dtype, the width-1 inputs before x,
 *                        oldest first; NULL means zeros
 *   final_conv_state   : [B, D, width-1]  io_dtype, the last width-1 inputs of the
 *                        sequence initial_conv_state followed by x (what the next
 *                        call or ssm_conv1d_update continues from); NULL means not
 *                        written.  Must not overlap any input (use two buffers when
 *                        processing a sequence in pieces).
 * width must be in [1, 4] (the pages use 4); with width 1 the state pointers are
 * ignored.  Other conventions as above (device pointers, 16-byte aligned bases,
 * host-side checks, asynchronous on `stream`, u must not overlap any input). */
ssm_status ssm_conv1d_fwd(int64_t batch, int64_t dim, int64_t seqlen, int64_t width,
                          int32_t io_dtype, const void* x, const float* weight,
                          const float* bias, const void* initial_conv_state, void* u,
                          void* final_conv_state, struct ihipStream_t* stream);

/* One generation step of the same convolution: u = silu(bias + weight . (state, x)),
 * then the state drops its oldest input and appends x (updated in place).
 *   conv_state : [B, D, width-1] io_dtype, read and written (NULL allowed if width == 1)
 *   x, u       : [B, D]          io_dtype
 *   weight     : [D, width] fp32; bias : [D] fp32 or NULL */
ssm_status ssm_conv1d_update(int64_t batch, int64_t dim, int64_t width, int32_t io_dtype,
                             void* conv_state, const void* x, const float* weight,
                             const float* bias, void* u, struct ihipStream_t* stream);

/* ------------------------------------------------------------------ training operators
 *
 * What a training step needs next to the scan and its gradients: the gradients of the conv,
 * the embedding of the tokens with its gradient, and the optimizer.  Conventions as above:
 * device pointers, 16-byte aligned bases, host-side checks before any launch, asynchronous on
 * `stream`, no allocation, fixed-order sums (bitwise reproducible).  A number that is out of its
 * stated range (a scale that is not finite, a beta of 1) is SSM_ERR_UNSUPPORTED. */

/* Bytes of device workspace ssm_conv1d_bwd needs (0 for invalid sizes): one partial sum of
 * dweight and dbias per row and segment of the sequence. */
size_t ssm_conv1d_bwd_workspace_size(int64_t batch, int64_t dim, int64_t seqlen, int64_t width,
                                     int32_t io_dtype);

/* Gradients of ssm_conv1d_fwd, from its inputs alone.  With a the pre-activation,
 * g = dout * silu'(a), H = width - 1 and x extended to the left by the initial state:
 *   dx[b,d,t]    = sum_k weight[d,k] * g[b,d,t+H-k]   (g is zero past the last step)
 *   dweight[d,k] = sum_{b,t} g[b,d,t] * x[b,d,t-H+k];   dbias[d] = sum_{b,t} g[b,d,t]
 * and the gradient of the initial state is dx's formula at the steps before 0.
 *   x, dout, dx               : [B, D, L] io_dtype
 *   weight, dweight           : [D, width] fp32;  bias (NULL means zero), dbias : [D] fp32
 *   initial_conv_state        : [B, D, H] io_dtype, NULL means zeros
 *   dfinal_conv_state         : [B, D, H] io_dtype gradient of final_conv_state, NULL means zero
 *   dinitial_conv_state       : [B, D, H] io_dtype, NULL means not written
 *   dbias                     : NULL means not computed (written even when bias is NULL)
 *   workspace                 : required, at least ssm_conv1d_bwd_workspace_size() bytes
 * width in [1, 4]; with width 1 the state pointers are ignored.  No output may overlap an
 * input, another output or the workspace. */
ssm_status ssm_conv1d_bwd(int64_t batch, int64_t dim, int64_t seqlen, int64_t width, int32_t io_dtype,
                          const void* x, const float* weight, const float* bias,
                          const void* initial_conv_state, const void* dout,
                          const void* dfinal_conv_state, void* dx, float* dweight, float* dbias,
                          void* dinitial_conv_state, void* workspace, size_t workspace_bytes,
                          struct ihipStream_t* stream);

typedef enum ssm_index_dtype { SSM_I32 = 0, SSM_I64 = 1 } ssm_index_dtype;

/* flag bits for ssm_embed_shape.flags */
#define SSM_FLAG_CHANNELS_FIRST 1u /* out and dout are [B, E, L], the layout of the conv and the scan */
#define SSM_FLAG_ACCUMULATE 2u     /* the gradient is added to dweight, whose other rows stay untouched */

typedef struct ssm_embed_shape {
  int64_t batch;        /* B >= 1 */
  int64_t seqlen;       /* L >= 1; B * L below 2^31 */
  int64_t rows;         /* V >= 1, below 2^31 - 1: rows of the table */
  int64_t dim;          /* E >= 1 */
  int32_t index_dtype;  /* ssm_index_dtype of tokens */
  int32_t table_dtype;  /* ssm_dtype of weight (forward) or dweight (backward) */
  int32_t io_dtype;     /* ssm_dtype of out or dout */
  uint32_t flags;       /* SSM_FLAG_CHANNELS_FIRST; backward: SSM_FLAG_ACCUMULATE */
} ssm_embed_shape;

/* Embedding: out[b,t,:] = scale * weight[tokens[b,t],:], rounded once to io_dtype.
 *   tokens : [B, L], aligned to their own size;  weight : [V, E];
 *   out    : [B, L, E], or [B, E, L] with SSM_FLAG_CHANNELS_FIRST
 * A token outside [0, V) (a padding mark such as -1) gives zeros. */
ssm_status ssm_embedding_fwd(const ssm_embed_shape* shape, const void* tokens, const void* weight,
                             float scale, void* out, struct ihipStream_t* stream);

/* Bytes of device workspace ssm_embedding_bwd needs for this shape (0 for an invalid one). */
size_t ssm_embedding_bwd_workspace_size(const ssm_embed_shape* shape);

/* Gradient of ssm_embedding_fwd: dweight[v,:] = scale * sum of dout over the positions whose
 * token is v.  The positions are sorted by token (equal tokens in order of position) and each
 * token's rows are summed in fp32 in a fixed order.  Tokens outside [0, V) take no part.
 *   dout    : [B, L, E] or [B, E, L], io_dtype
 *   dweight : [V, E] table_dtype, fully written (zeros for tokens that do not occur), or with
 *             SSM_FLAG_ACCUMULATE added to: then only the rows of tokens that occur are touched
 *   workspace : required, at least ssm_embedding_bwd_workspace_size() bytes */
ssm_status ssm_embedding_bwd(const ssm_embed_shape* shape, const void* tokens, const void* dout,
                             float scale, void* dweight, void* workspace, size_t workspace_bytes,
                             struct ihipStream_t* stream);

/* One parameter tensor of an optimizer step (dense, any shape).  The params, gradients and state
 * buffers of a step must not overlap (checked; gradients may overlap one another). */
typedef struct ssm_adamw_tensor {
  void* param;          /* read and written */
  const void* grad;
  int64_t numel;        /* >= 1 */
  int64_t offset;       /* where its states begin in the state buffers, in elements: a multiple of
                           SSM_ADAMW_BLOCK; they take numel rounded up to whole blocks, and the
                           next tensor's begin behind them */
  int32_t param_dtype;  /* ssm_dtype */
  int32_t grad_dtype;   /* ssm_dtype */
} ssm_adamw_tensor;

#define SSM_ADAMW_BLOCK 128 /* elements that share a base of the 8-bit states */

typedef struct ssm_adamw_config {
  double lr, beta1, beta2, eps, weight_decay; /* finite; betas in [0, 1); eps in [1e-30, 1e30] */
  int64_t step;        /* number of this step, from 1 */
  uint64_t seed;       /* of the stochastic rounding */
  int32_t state_bits;  /* 32: fp32 states; 8: one byte per element and one base per block */
  uint32_t flags;      /* 0 */
} ssm_adamw_config;

/* Norm of all gradients together and the factor that clips it to max_norm:
 *   result[0] = sqrt(sum of squares) (summed in fp64, in a fixed order; fp32)
 *   result[1] = max_norm / norm where norm > max_norm, else 1; NaN where the norm is not finite
 * tensors is a host array of `count` descriptors (only grad, numel and grad_dtype are read); it is
 * not needed after the call returns.  result: 2 floats on the device.  workspace: required, at
 * least ssm_grad_norm_workspace_size() bytes. */
size_t ssm_grad_norm_workspace_size(const ssm_adamw_tensor* tensors, int64_t count);
ssm_status ssm_grad_norm(const ssm_adamw_tensor* tensors, int64_t count, double max_norm, float* result,
                         void* workspace, size_t workspace_bytes, struct ihipStream_t* stream);

/* One AdamW step over all tensors (decoupled weight decay, bias-corrected moments):
 *   g = clip * grad;  m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g g
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^step) * m / (sqrt(v / (1 - beta2^step)) + eps)
 * in fp32.  tensors: a host array, not needed after the call returns; params must not overlap one
 * another, the gradients or the states.
 *   exp_avg, exp_avg_sq : m and v of all tensors, tensor k's at its offset: fp32 (state_bits 32) or
 *       codes of one byte (state_bits 8).  8-bit: with the bits of a positive fp32 number read as an
 *       integer, an element of code c >= 1 in a block of base K stands for the number whose bits are
 *       (c + K) << 20 (a sign bit, 8 exponent bits and 3 mantissa bits); code 0 stands for zero.  m has a
 *       sign in bit 7 and c in bits 0-6, v has c in 8 bits.  A block's base puts its largest
 *       element at the largest code, the others are rounded stochastically, and a v that is not zero
 *       is not rounded to zero.  In a block with elements that are not finite the base is stored as its
 *       complement (-1 - K): there the largest code stands for infinity (a NaN is held as one: its param
 *       is a NaN already) and the block's largest finite element is put at the code below it.
 *   exp_avg_base, exp_avg_sq_base : the blocks' K, int16, element offset / 128 onwards; 8-bit only
 *   master : fp32 weights of all bf16 tensors at their offsets (the step works on these and writes
 *       their rounded values to param), or NULL: then a bf16 param is itself rounded stochastically.
 *       Not used for fp32 tensors.
 *   clip : result of ssm_grad_norm on the device, or NULL for no clipping.  Where result[1] is
 *       NaN the step changes nothing.
 * The random numbers are a hash of (seed, step, index of the tensor, index of the element). */
ssm_status ssm_adamw_step(const ssm_adamw_config* config, const ssm_adamw_tensor* tensors, int64_t count,
                          void* exp_avg, void* exp_avg_sq, int16_t* exp_avg_base, int16_t* exp_avg_sq_base,
                          float* master, const float* clip, struct ihipStream_t* stream);

/* What a clipped step counts and keeps on the device, 32 bytes: only `step` is the caller's to set (the
 * steps already made, 0 for a new optimizer), and to read after the stream's work is done. */
typedef struct ssm_adamw_progress {
  int64_t step;
  uint32_t internal[6];
} ssm_adamw_progress;

/* ssm_grad_norm and ssm_adamw_step in one call, with the number of the step on the device: a step whose
 * norm is not finite changes nothing and is not counted, and the call may be captured in a graph, each
 * replay of which is the next step (with the settings and addresses of the capture).
 *   config   : its `step` is not used
 *   progress : on the device, 16-byte aligned; read and written
 *   norm     : one float on the device, the norm before clipping
 *   workspace: required, at least ssm_grad_norm_workspace_size() bytes
 * Everything else as in the two calls; all checks come before the first launch. */
ssm_status ssm_adamw_clipped_step(const ssm_adamw_config* config, const ssm_adamw_tensor* tensors, int64_t count,
                                  double max_norm, void* exp_avg, void* exp_avg_sq, int16_t* exp_avg_base,
                                  int16_t* exp_avg_sq_base, float* master, ssm_adamw_progress* progress, float* norm,
                                  void* workspace, size_t workspace_bytes, struct ihipStream_t* stream);

/* The values that 8-bit states stand for, exactly, in bf16: `numel` codes (a multiple of
 * SSM_ADAMW_BLOCK), numel / 128 bases each.  m_values and v_values : [numel] bf16; NULL means not wanted. */
ssm_status ssm_adamw_state_values(int64_t numel, const void* exp_avg, const void* exp_avg_sq,
                                  const int16_t* exp_avg_base, const int16_t* exp_avg_sq_base,
                                  void* m_values, void* v_values, struct ihipStream_t* stream);

#ifdef __cplusplus
}
#endif
#endif /* SSM_SCAN_H */
