// block_abi.cpp -- the C entry points of the residual block's operators declared in include/ssm_scan.h: layer norm,
// dropout, the gated linear recurrence, and their gradients.  Every argument is validated on the host before
// anything is enqueued, and nothing is allocated or kept.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../../include/ssm_scan.h"
#include "../train/abi_checks.h"
#include "block_launch.h"

using namespace ssm::abi;

namespace {

template <size_t N> bool any_misaligned(const void* const (&ptrs)[N]) {
  for (const void* q : ptrs)
    if (misaligned(q)) return true;
  return false;
}

// NULL: no dropout
ssm_status drop_params(const ssm_dropout* d, ssm::DropParams* p) {
  memset(p, 0, sizeof(*p));
  if (!d) return SSM_OK;
  if (!(d->p >= 0 && d->p <= 1)) return SSM_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(d->device_seed) & 7u) return SSM_ERR_ALIGN;
  p->below = (uint32_t)rint(d->p * 65536);
  p->scale = p->below < 65536 ? 65536.0f / (float)(65536 - p->below) : 0.0f;
  p->device_seed = d->device_seed;
  p->seed = d->seed;
  p->call = d->call;
  return SSM_OK;
}

Range seed_span(const ssm_dropout* d) { return span(d ? d->device_seed : nullptr, 8); }

struct NormSizes {
  int64_t rows, n, xs, hs;
  int kind;
};

ssm_status norm_check(const ssm_norm_shape* s, NormSizes* z, ssm::NormParams* p) {
  if (!s) return SSM_ERR_NULL;
  if (!dtype_ok(s->x_dtype) || !dtype_ok(s->hidden_dtype)) return SSM_ERR_DTYPE;
  if (s->x_dtype == SSM_F32 && s->hidden_dtype == SSM_BF16) return SSM_ERR_DTYPE;
  if (s->flags & ~(SSM_FLAG_CHANNELS_FIRST | SSM_FLAG_RMS)) return SSM_ERR_UNSUPPORTED;
  if (s->batch < 1 || s->seqlen < 1 || s->dim < 1 || s->dim > (int64_t(1) << 30)) return SSM_ERR_SHAPE;
  int64_t bytes;
  if (!mul_ok(s->batch, s->seqlen, &z->rows) || z->rows > kMaxGrid) return SSM_ERR_SHAPE;
  if (!mul_ok(z->rows, s->dim, &z->n) || !mul_ok(z->n, 4, &bytes)) return SSM_ERR_SHAPE;
  z->xs = dtype_size(s->x_dtype);
  z->hs = dtype_size(s->hidden_dtype);
  z->kind = (s->x_dtype == SSM_BF16 ? 1 : 0) + (s->hidden_dtype == SSM_BF16 ? 2 : 0);
  memset(p, 0, sizeof(*p));
  p->rows = z->rows; p->E = s->dim; p->B = s->batch; p->L = s->seqlen;
  p->inv_e = (float)(1.0 / (double)s->dim);
  p->rms = (s->flags & SSM_FLAG_RMS) ? 1 : 0;
  return SSM_OK;
}

// one step: the layouts agree
bool norm_cols(const ssm_norm_shape* s) { return (s->flags & SSM_FLAG_CHANNELS_FIRST) && s->seqlen > 1; }

int64_t norm_bwd_blocks(const ssm_norm_shape* s, const NormSizes& z) {
  return norm_cols(s) ? ssm::norm_cols_bwd_blocks(s->batch, s->dim, s->seqlen, z.kind, s->flags & SSM_FLAG_RMS)
                      : ssm::norm_rows_bwd_blocks(z.rows, s->dim);
}

}  // namespace

extern "C" {

ssm_status ssm_layer_norm_fwd(const ssm_norm_shape* shape, const void* x, const float* weight, const float* bias,
                              const void* residual, double eps, const ssm_dropout* drop, void* out, void* hidden,
                              float* stats, struct ihipStream_t* stream) {
  NormSizes z;
  ssm::NormParams p;
  ssm_status rc = norm_check(shape, &z, &p);
  if (rc != SSM_OK) return rc;
  if (!x || !out) return SSM_ERR_NULL;
  if (!(eps >= 0) || !isfinite(eps)) return SSM_ERR_UNSUPPORTED;
  rc = drop_params(drop, &p.drop);
  if (rc != SSM_OK) return rc;
  const void* const ptrs[] = {x, weight, bias, residual, out, hidden};
  if (any_misaligned(ptrs) || (reinterpret_cast<uintptr_t>(stats) & 3u)) return SSM_ERR_ALIGN;
  const int64_t side = shape->dim * 4;
  const Range ins[] = {span(x, z.n * z.xs), span(weight, side), span(bias, side), span(residual, z.n * z.hs),
                       seed_span(drop)};
  const Range outs[] = {span(out, z.n * z.xs), span(hidden, z.n * z.hs), span(stats, z.rows * 8)};
  if (any_overlap(outs, 3, ins, 5)) return SSM_ERR_OVERLAP;
  p.x = x; p.weight = weight; p.bias = bias; p.residual = residual; p.out = out; p.hidden = hidden; p.stats = stats;
  p.eps = (float)eps;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  return launch_status(norm_cols(shape) ? ssm::launch_norm_cols(p, z.kind, st) : ssm::launch_norm_rows(p, z.kind, st));
}

size_t ssm_layer_norm_bwd_workspace_size(const ssm_norm_shape* shape) {
  NormSizes z;
  ssm::NormParams p;
  if (norm_check(shape, &z, &p) != SSM_OK) return 0;
  return (size_t)norm_bwd_blocks(shape, z) * 2 * (size_t)shape->dim * 4;
}

ssm_status ssm_layer_norm_bwd(const ssm_norm_shape* shape, const void* dout, const void* hidden, const float* weight,
                              const float* stats, const void* dhidden, const ssm_dropout* drop, void* dx, void* dresidual,
                              float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                              struct ihipStream_t* stream) {
  NormSizes z;
  ssm::NormParams p;
  ssm_status rc = norm_check(shape, &z, &p);
  if (rc != SSM_OK) return rc;
  if (!dout || !hidden || !stats || (!dx && !dresidual)) return SSM_ERR_NULL;
  const bool sums = dweight || dbias;
  if (sums && !workspace) return SSM_ERR_NULL;
  rc = drop_params(drop, &p.drop);
  if (rc != SSM_OK) return rc;
  const void* const ptrs[] = {dout, hidden, weight, dhidden, dx, dresidual, dweight, dbias, workspace};
  if (any_misaligned(ptrs) || (reinterpret_cast<uintptr_t>(stats) & 3u)) return SSM_ERR_ALIGN;
  const int64_t need = norm_bwd_blocks(shape, z) * 2 * shape->dim * 4, side = shape->dim * 4;
  if (sums && workspace_bytes < (size_t)need) return SSM_ERR_WORKSPACE;
  const Range ins[] = {span(dout, z.n * z.xs),    span(hidden, z.n * z.hs),  span(weight, side),
                       span(stats, z.rows * 8),   span(dhidden, z.n * z.hs), seed_span(drop)};
  const Range outs[] = {span(dx, z.n * z.xs), span(dresidual, z.n * z.hs), span(dweight, side), span(dbias, side),
                        span(sums ? workspace : nullptr, need)};
  if (any_overlap(outs, 5, ins, 6)) return SSM_ERR_OVERLAP;
  p.x = dout; p.residual = hidden; p.weight = weight; p.stats = const_cast<float*>(stats); p.dhidden = dhidden;
  p.out = dx; p.hidden = dresidual; p.dweight = dweight; p.dbias = dbias;
  p.part = sums ? static_cast<float*>(workspace) : nullptr;
  p.blocks = norm_bwd_blocks(shape, z);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  rc = launch_status(norm_cols(shape) ? ssm::launch_norm_cols_bwd(p, z.kind, st) : ssm::launch_norm_rows_bwd(p, z.kind, st));
  if (rc != SSM_OK || !sums) return rc;
  return launch_status(ssm::launch_join({p.part, p.blocks, p.E, 2, {dweight, dbias, nullptr}}, st));
}

ssm_status ssm_dropout_fwd(int64_t numel, int32_t x_dtype, int32_t out_dtype, const void* x, const void* residual,
                           const ssm_dropout* drop, void* out, struct ihipStream_t* stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(out_dtype)) return SSM_ERR_DTYPE;
  if (numel < 1 || numel > (int64_t(1) << 42)) return SSM_ERR_SHAPE;
  if (!x || !drop || !out) return SSM_ERR_NULL;
  ssm::DropoutParams p;
  memset(&p, 0, sizeof(p));
  const ssm_status rc = drop_params(drop, &p.drop);
  if (rc != SSM_OK) return rc;
  const void* const ptrs[] = {x, residual, out};
  if (any_misaligned(ptrs)) return SSM_ERR_ALIGN;
  const int64_t os = dtype_size(out_dtype);
  const Range ins[] = {span(x, numel * dtype_size(x_dtype)), span(residual, numel * os), seed_span(drop)};
  const Range outs[] = {span(out, numel * os)};
  if (any_overlap(outs, 1, ins, 3)) return SSM_ERR_OVERLAP;
  p.x = x; p.residual = residual; p.out = out; p.n = numel;
  return launch_status(ssm::launch_dropout(p, x_dtype == SSM_BF16, out_dtype == SSM_BF16,
                                           reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

struct RecurSizes {
  int64_t bd, n;      // elements of [B, D], of [B, D, L]
  int64_t es;
  bool bf16, rev;
  ssm::RecurPlan plan;
  int64_t ckpt, seg, part;  // bytes
};

ssm_status recur_check(const ssm_recurrence_shape* s, RecurSizes* z) {
  if (!s) return SSM_ERR_NULL;
  if (!dtype_ok(s->io_dtype)) return SSM_ERR_DTYPE;
  if (s->flags & ~SSM_FLAG_REVERSE) return SSM_ERR_UNSUPPORTED;
  if (s->batch < 1 || s->dim < 1 || s->seqlen < 1 || s->seqlen > kMaxSize) return SSM_ERR_SHAPE;
  int64_t bytes;
  if (!mul_ok(s->batch, s->dim, &z->bd) || z->bd > kMaxGrid) return SSM_ERR_SHAPE;
  if (!mul_ok(z->bd, s->seqlen, &z->n) || !mul_ok(z->n, 4, &bytes)) return SSM_ERR_SHAPE;
  z->es = dtype_size(s->io_dtype);
  z->bf16 = s->io_dtype == SSM_BF16;
  z->rev = (s->flags & SSM_FLAG_REVERSE) != 0;
  z->plan = ssm::recur_plan(s->batch, s->dim, s->seqlen, z->bf16);
  z->ckpt = z->bd * z->plan.blocks * 4;
  z->seg = z->plan.S > 1 ? z->bd * z->plan.S * 8 : 0;
  z->part = z->bd * z->plan.S * z->plan.waves * z->plan.parts * 12;
  return SSM_OK;
}

int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

ssm::RecurParams recur_params(const ssm_recurrence_shape* s, const RecurSizes& z, const void* x, const void* r,
                              const void* i, const float* decay, const float* r_bias, const float* i_bias, const void* gate,
                              const float* init) {
  ssm::RecurParams p;
  memset(static_cast<void*>(&p), 0, sizeof(p));
  p.x = x; p.r = r; p.i = i; p.z = gate; p.decay = decay; p.rb = r_bias; p.ib = i_bias; p.init = init;
  p.B = s->batch; p.D = s->dim; p.L = s->seqlen; p.plan = z.plan;
  return p;
}

int64_t recur_bwd_bytes(const RecurSizes& z, bool saved) {
  return round16(z.seg) + round16(z.part) + (saved ? 0 : round16(z.ckpt));
}

}  // namespace

extern "C" {

int64_t ssm_recurrence_checkpoints(const ssm_recurrence_shape* shape) {
  RecurSizes z;
  return recur_check(shape, &z) == SSM_OK ? z.plan.blocks : 0;
}

size_t ssm_recurrence_workspace_size(const ssm_recurrence_shape* shape) {
  RecurSizes z;
  return recur_check(shape, &z) == SSM_OK ? (size_t)z.seg : 0;
}

ssm_status ssm_recurrence_fwd(const ssm_recurrence_shape* shape, const void* x, const void* r, const void* i,
                              const float* decay, const float* r_bias, const float* i_bias, const void* z,
                              const float* initial_state, void* out, float* final_state, float* checkpoints,
                              void* workspace, size_t workspace_bytes, struct ihipStream_t* stream) {
  RecurSizes k;
  const ssm_status rc = recur_check(shape, &k);
  if (rc != SSM_OK) return rc;
  if (!x || !r || !i || !decay || !out || (k.seg && !workspace)) return SSM_ERR_NULL;
  const void* const ptrs[] = {x, r, i, decay, r_bias, i_bias, z, initial_state, out, final_state, checkpoints, workspace};
  if (any_misaligned(ptrs)) return SSM_ERR_ALIGN;
  if (workspace_bytes < (size_t)k.seg) return SSM_ERR_WORKSPACE;
  const int64_t n = k.n * k.es, side = shape->dim * 4;
  const Range ins[] = {span(x, n),         span(r, n),         span(i, n), span(decay, side), span(r_bias, side),
                       span(i_bias, side), span(z, n),         span(initial_state, k.bd * 4)};
  const Range outs[] = {span(out, n), span(final_state, k.bd * 4), span(checkpoints, k.ckpt), span(workspace, k.seg)};
  if (any_overlap(outs, 4, ins, 8)) return SSM_ERR_OVERLAP;
  ssm::RecurParams p = recur_params(shape, k, x, r, i, decay, r_bias, i_bias, z, initial_state);
  p.out = out; p.last = final_state; p.ckpt = checkpoints; p.seg = static_cast<float*>(workspace);
  return launch_status(ssm::launch_recur_fwd(p, k.bf16, k.rev, reinterpret_cast<hipStream_t>(stream)));
}

size_t ssm_recurrence_bwd_workspace_size(const ssm_recurrence_shape* shape, int32_t saved) {
  RecurSizes k;
  return recur_check(shape, &k) == SSM_OK ? (size_t)recur_bwd_bytes(k, saved != 0) : 0;
}

ssm_status ssm_recurrence_bwd(const ssm_recurrence_shape* shape, const void* x, const void* r, const void* i,
                              const float* decay, const float* r_bias, const float* i_bias, const void* z,
                              const float* initial_state, const void* dout, const float* dfinal_state,
                              const float* checkpoints, void* dx, void* dr, void* di, void* dz, float* ddecay,
                              float* dr_bias, float* di_bias, float* dinitial_state, void* workspace,
                              size_t workspace_bytes, struct ihipStream_t* stream) {
  RecurSizes k;
  const ssm_status rc = recur_check(shape, &k);
  if (rc != SSM_OK) return rc;
  if (!x || !r || !i || !decay || !dout || !dx || !dr || !di || !ddecay || !workspace || (z && !dz)) return SSM_ERR_NULL;
  if (!z) dz = nullptr;
  const void* const ptrs[] = {x, r, i, decay, r_bias, i_bias, z, initial_state, dout, dfinal_state, checkpoints,
                              dx, dr, di, dz, ddecay, dr_bias, di_bias, dinitial_state, workspace};
  if (any_misaligned(ptrs)) return SSM_ERR_ALIGN;
  const int64_t need = recur_bwd_bytes(k, checkpoints != nullptr);
  if (workspace_bytes < (size_t)need) return SSM_ERR_WORKSPACE;
  const int64_t n = k.n * k.es, side = shape->dim * 4;
  const Range ins[] = {span(x, n),         span(r, n),    span(i, n),
                       span(decay, side),  span(r_bias, side), span(i_bias, side),
                       span(z, n),         span(initial_state, k.bd * 4), span(dout, n),
                       span(dfinal_state, k.bd * 4), span(checkpoints, k.ckpt)};
  const Range outs[] = {span(dx, n), span(dr, n), span(di, n), span(dz, n), span(ddecay, side), span(dr_bias, side),
                        span(di_bias, side), span(dinitial_state, k.bd * 4), span(workspace, need)};
  if (any_overlap(outs, 9, ins, 11)) return SSM_ERR_OVERLAP;
  ssm::RecurParams p = recur_params(shape, k, x, r, i, decay, r_bias, i_bias, z, initial_state);
  char* ws = static_cast<char*>(workspace);
  p.seg = reinterpret_cast<float*>(ws);
  p.part = reinterpret_cast<float*>(ws + round16(k.seg));
  p.ckpt = const_cast<float*>(checkpoints);
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (!checkpoints) {  // the forward pass for the checkpoints alone
    p.ckpt = reinterpret_cast<float*>(ws + round16(k.seg) + round16(k.part));
    const ssm_status rf = launch_status(ssm::launch_recur_fwd(p, k.bf16, k.rev, st));
    if (rf != SSM_OK) return rf;
  }
  p.dout = dout; p.dlast = dfinal_state; p.dx = dx; p.dr = dr; p.di = di; p.dz = dz; p.dinit = dinitial_state;
  p.ddecay = ddecay; p.drb = dr_bias; p.dib = di_bias;
  return launch_status(ssm::launch_recur_bwd(p, k.bf16, k.rev, st));
}

ssm_status ssm_recurrence_update(int64_t batch, int64_t dim, int32_t io_dtype, float* state, const void* x, const void* r,
                                 const void* i, const float* decay, const float* r_bias, const float* i_bias,
                                 const void* z, void* out, struct ihipStream_t* stream) {
  if (!dtype_ok(io_dtype)) return SSM_ERR_DTYPE;
  int64_t bd;
  if (batch < 1 || dim < 1 || !mul_ok(batch, dim, &bd) || bd > (int64_t(1) << 40)) return SSM_ERR_SHAPE;
  if (!state || !x || !r || !i || !decay || !out) return SSM_ERR_NULL;
  const void* const ptrs[] = {state, x, r, i, decay, r_bias, i_bias, z, out};
  if (any_misaligned(ptrs)) return SSM_ERR_ALIGN;
  const int64_t n = bd * dtype_size(io_dtype), side = dim * 4;
  const Range ins[] = {span(x, n), span(r, n), span(i, n), span(decay, side), span(r_bias, side), span(i_bias, side),
                       span(z, n)};
  const Range outs[] = {span(state, bd * 4), span(out, n)};
  if (any_overlap(outs, 2, ins, 7)) return SSM_ERR_OVERLAP;
  ssm::RecurStepParams p;
  p.state = state; p.x = x; p.r = r; p.i = i; p.z = z; p.decay = decay; p.rb = r_bias; p.ib = i_bias; p.out = out;
  p.n = bd; p.D = dim;
  return launch_status(ssm::launch_recur_step(p, io_dtype == SSM_BF16, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
