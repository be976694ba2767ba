// train_abi.cpp -- the C entry points of the training operators declared in include/ssm_scan.h: the
// conv's gradients, the embedding and its gradient, AdamW.  As in ssm_abi.cpp every argument is
// validated on the host before anything is enqueued, and nothing is allocated or kept.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "../../../include/ssm_scan.h"
#include "abi_checks.h"
#include "train_launch.h"

using namespace ssm::abi;

namespace {

struct ConvPlan {
  int64_t bd, bdl, S;
  int lanes;
  size_t bytes;
};

bool conv_plan(int64_t batch, int64_t dim, int64_t seqlen, int64_t width, int32_t io, ConvPlan* pl) {
  if (batch < 1 || dim < 1 || seqlen < 1 || width < 1 || width > 4) return false;
  if (batch > kMaxSize || dim > kMaxSize || seqlen > kMaxSize) return false;
  if (!mul_ok(batch, dim, &pl->bd) || !mul_ok(pl->bd, seqlen, &pl->bdl)) return false;
  pl->S = ssm::conv_bwd_segments(seqlen, io == SSM_BF16, &pl->lanes);
  int64_t units, elems;
  if (!mul_ok(pl->bd, pl->S, &units) || !mul_ok(units, 4 * (width + 1), &elems)) return false;
  if (units > kMaxGrid || dim > kMaxGrid) return false;
  pl->bytes = static_cast<size_t>(units) * (width + 1) * 4;
  return true;
}

}  // namespace

extern "C" {

size_t ssm_conv1d_bwd_workspace_size(int64_t batch, int64_t dim, int64_t seqlen, int64_t width, int32_t io_dtype) {
  ConvPlan pl;
  if (!dtype_ok(io_dtype) || !conv_plan(batch, dim, seqlen, width, io_dtype, &pl)) return 0;
  return pl.bytes;
}

ssm_status ssm_conv1d_bwd(int64_t batch, int64_t dim, int64_t seqlen, int64_t width, int32_t io_dtype,
                          const void* x, const float* weight, const float* bias, const void* initial_conv_state,
                          const void* dout, const void* dfinal_conv_state, void* dx, float* dweight, float* dbias,
                          void* dinitial_conv_state, void* workspace, size_t workspace_bytes,
                          struct ihipStream_t* stream) {
  if (!dtype_ok(io_dtype)) return SSM_ERR_DTYPE;
  ConvPlan pl;
  if (!conv_plan(batch, dim, seqlen, width, io_dtype, &pl)) return SSM_ERR_SHAPE;
  if (!x || !weight || !dout || !dx || !dweight || !workspace) return SSM_ERR_NULL;
  const int64_t H = width - 1, es = dtype_size(io_dtype);
  const void* init = H > 0 ? initial_conv_state : nullptr;
  const void* dfinal = H > 0 ? dfinal_conv_state : nullptr;
  void* dinit = H > 0 ? dinitial_conv_state : nullptr;
  const void* ptrs[] = {x, weight, bias, init, dout, dfinal, dx, dweight, dbias, dinit, workspace};
  for (const void* q : ptrs)
    if (misaligned(q)) return SSM_ERR_ALIGN;
  if (workspace_bytes < pl.bytes) return SSM_ERR_WORKSPACE;
  const Range ins[] = {span(x, pl.bdl * es),       span(weight, dim * width * 4), span(bias, dim * 4),
                       span(init, pl.bd * H * es), span(dout, pl.bdl * es),       span(dfinal, pl.bd * H * es)};
  const Range outs[] = {span(dx, pl.bdl * es), span(dweight, dim * width * 4), span(dbias, dim * 4),
                        span(dinit, pl.bd * H * es), span(workspace, (int64_t)pl.bytes)};
  if (any_overlap(outs, 5, ins, 6)) return SSM_ERR_OVERLAP;

  ssm::ConvBwdParams p;
  memset(&p, 0, sizeof(p));
  p.x = x; p.w = weight; p.bias = bias; p.init = init; p.dout = dout; p.dfinal = dfinal;
  p.dx = dx; p.dinit = dinit; p.dw = dweight; p.db = dbias; p.part = static_cast<float*>(workspace);
  p.Bsz = batch; p.Dm = dim; p.L = seqlen; p.K = (int)width;
  p.S = pl.S; p.units = (uint32_t)(pl.bd * pl.S); p.lanes = pl.lanes;
  return launch_status(ssm::launch_conv_bwd(p, io_dtype == SSM_BF16, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

ssm_status embed_check(const ssm_embed_shape* s, uint32_t flags, ssm::EmbedParams* p) {
  if (!s) return SSM_ERR_NULL;
  if (!dtype_ok(s->table_dtype) || !dtype_ok(s->io_dtype)) return SSM_ERR_DTYPE;
  if (s->index_dtype != SSM_I32 && s->index_dtype != SSM_I64) return SSM_ERR_DTYPE;
  if (s->flags & ~flags) return SSM_ERR_UNSUPPORTED;
  if (s->batch < 1 || s->seqlen < 1 || s->rows < 1 || s->dim < 1) return SSM_ERR_SHAPE;
  int64_t n, te, ve;
  if (!mul_ok(s->batch, s->seqlen, &n) || n > kMaxGrid) return SSM_ERR_SHAPE;
  if (s->rows >= kMaxGrid || s->dim > kMaxSize) return SSM_ERR_SHAPE;
  if (!mul_ok(n, s->dim, &te) || !mul_ok(s->rows, s->dim, &ve)) return SSM_ERR_SHAPE;
  if (ve > (int64_t(1) << 42)) return SSM_ERR_SHAPE;  // more than any memory holds
  // every kernel's grid: at most one workgroup per position and 64 columns, or per 256 pieces of 16 bytes
  int64_t blocks;
  if (!mul_ok(n, (s->dim + 63) / 64, &blocks) || blocks > kMaxGrid) return SSM_ERR_SHAPE;
  memset(p, 0, sizeof(*p));
  p->Bsz = s->batch; p->L = s->seqlen; p->V = s->rows; p->E = s->dim; p->T = n;
  p->i64 = s->index_dtype == SSM_I64;
  p->cf = (s->flags & SSM_FLAG_CHANNELS_FIRST) && s->seqlen > 1 ? 1 : 0;  // one step: the layouts agree
  p->add = (s->flags & SSM_FLAG_ACCUMULATE) ? 1 : 0;
  return SSM_OK;
}

// tokens are read one at a time: a row of a batch of odd length will do
bool tokens_misaligned(const ssm::EmbedParams& p, const void* tokens) {
  return (reinterpret_cast<uintptr_t>(tokens) & (p.i64 ? 7u : 3u)) != 0;
}

}  // namespace

extern "C" {

ssm_status ssm_embedding_fwd(const ssm_embed_shape* shape, const void* tokens, const void* weight, float scale,
                             void* out, struct ihipStream_t* stream) {
  ssm::EmbedParams p;
  const ssm_status rc = embed_check(shape, SSM_FLAG_CHANNELS_FIRST, &p);
  if (rc != SSM_OK) return rc;
  if (!tokens || !weight || !out) return SSM_ERR_NULL;
  if (!isfinite(scale)) return SSM_ERR_UNSUPPORTED;
  if (tokens_misaligned(p, tokens) || misaligned(weight) || misaligned(out)) return SSM_ERR_ALIGN;
  const Range ins[] = {span(tokens, p.T * (p.i64 ? 8 : 4)),
                       span(weight, p.V * p.E * dtype_size(shape->table_dtype))};
  const Range outs[] = {span(out, p.T * p.E * dtype_size(shape->io_dtype))};
  if (any_overlap(outs, 1, ins, 2)) return SSM_ERR_OVERLAP;
  p.tokens = tokens; p.table = weight; p.out = out; p.scale = scale;
  return launch_status(ssm::launch_embed_fwd(p, shape->table_dtype == SSM_BF16, shape->io_dtype == SSM_BF16,
                                             reinterpret_cast<hipStream_t>(stream)));
}

size_t ssm_embedding_bwd_workspace_size(const ssm_embed_shape* shape) {
  ssm::EmbedParams p;
  if (embed_check(shape, SSM_FLAG_CHANNELS_FIRST | SSM_FLAG_ACCUMULATE, &p) != SSM_OK) return 0;
  ssm::EmbedBwdPlan pl;
  ssm::plan_embed_bwd(p.Bsz, p.L, p.V, p.E, dtype_size(shape->table_dtype), shape->io_dtype == SSM_BF16, p.cf, p.add,
                      &pl);
  return pl.total;
}

ssm_status ssm_embedding_bwd(const ssm_embed_shape* shape, const void* tokens, const void* dout, float scale,
                             void* dweight, void* workspace, size_t workspace_bytes, struct ihipStream_t* stream) {
  ssm::EmbedParams p;
  const ssm_status rc = embed_check(shape, SSM_FLAG_CHANNELS_FIRST | SSM_FLAG_ACCUMULATE, &p);
  if (rc != SSM_OK) return rc;
  if (!tokens || !dout || !dweight || !workspace) return SSM_ERR_NULL;
  if (!isfinite(scale)) return SSM_ERR_UNSUPPORTED;
  if (tokens_misaligned(p, tokens) || misaligned(dout) || misaligned(dweight) || misaligned(workspace)) return SSM_ERR_ALIGN;
  ssm::EmbedBwdPlan pl;
  ssm::plan_embed_bwd(p.Bsz, p.L, p.V, p.E, dtype_size(shape->table_dtype), shape->io_dtype == SSM_BF16, p.cf, p.add,
                      &pl);
  if (workspace_bytes < pl.total) return SSM_ERR_WORKSPACE;
  const Range ins[] = {span(tokens, p.T * (p.i64 ? 8 : 4)), span(dout, p.T * p.E * dtype_size(shape->io_dtype))};
  const Range outs[] = {span(dweight, p.V * p.E * dtype_size(shape->table_dtype)),
                        span(workspace, (int64_t)pl.total)};
  if (any_overlap(outs, 2, ins, 2)) return SSM_ERR_OVERLAP;
  p.tokens = tokens; p.dout = dout; p.out = dweight; p.scale = scale;
  return launch_status(ssm::launch_embed_bwd(p, pl, shape->table_dtype == SSM_BF16, shape->io_dtype == SSM_BF16,
                                             workspace, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

bool finite_in(double x, double lo, double hi) { return isfinite(x) && x >= lo && x <= hi; }

int64_t chunks_of(int64_t n, int64_t chunk) { return (n + chunk - 1) / chunk; }

// what both calls ask of the descriptors; *elems: where the last tensor's states end
ssm_status check_tensors(const ssm_adamw_tensor* t, int64_t count, bool grads_only, int64_t* elems) {
  if (!t) return SSM_ERR_NULL;
  if (count < 1 || count > (int64_t(1) << 31)) return SSM_ERR_SHAPE;
  int64_t end = 0;
  for (int64_t k = 0; k < count; ++k) {
    if (!t[k].grad || (!grads_only && !t[k].param)) return SSM_ERR_NULL;
    if (t[k].numel < 1 || t[k].numel > kMaxSize) return SSM_ERR_SHAPE;
    if (!dtype_ok(t[k].grad_dtype) || (!grads_only && !dtype_ok(t[k].param_dtype))) return SSM_ERR_DTYPE;
    if (misaligned(t[k].grad) || (!grads_only && misaligned(t[k].param))) return SSM_ERR_ALIGN;
    if (grads_only) continue;
    if (t[k].offset < end || t[k].offset % SSM_ADAMW_BLOCK || t[k].offset > (int64_t(1) << 58)) return SSM_ERR_SHAPE;
    end = t[k].offset + chunks_of(t[k].numel, SSM_ADAMW_BLOCK) * SSM_ADAMW_BLOCK;
  }
  *elems = end;
  return SSM_OK;
}

// Whether a tensor's param lies over a gradient, its own or another's, or over another param.  The params are sorted
// a block at a time on the stack, and all other ranges are looked up among them.
bool params_clash(const ssm_adamw_tensor* t, int64_t count) {
  constexpr int64_t kBlock = 2048;
  Range r[kBlock];
  auto param = [&](int64_t k) { return span(t[k].param, t[k].numel * dtype_size(t[k].param_dtype)); };
  for (int64_t b = 0; b < count; b += kBlock) {
    const int64_t n = count - b < kBlock ? count - b : kBlock;
    for (int64_t i = 0; i < n; ++i) r[i] = param(b + i);
    auto before = [](const Range& x, const Range& y) { return x.lo < y.lo; };
    if (!std::is_sorted(r, r + n, before)) std::sort(r, r + n, before);
    for (int64_t i = 1; i < n; ++i)
      if (overlaps(r[i - 1], r[i])) return true;
    auto hit = [&](Range q) {
      if (q.hi <= r[0].lo || q.lo >= r[n - 1].hi) return false;
      // the first that ends behind q's beginning: the only one before those behind q
      const Range* f = std::partition_point(r, r + n, [&](const Range& x) { return x.hi <= q.lo; });
      return f < r + n && overlaps(*f, q);
    };
    for (int64_t k = 0; k < count; ++k) {
      if (hit(span(t[k].grad, t[k].numel * dtype_size(t[k].grad_dtype)))) return true;
      if (k >= b + n && hit(param(k))) return true;
    }
  }
  return false;
}

// Calls go(table, workgroups) for the tensors that `take` accepts, as many at a time as a table holds and a
// launch's workgroups allow, `chunk` elements per workgroup; put(table, slot, place in the list) enters one.
template <typename Table, int kRoom, typename Take, typename Put, typename Go>
hipError_t in_tables(const ssm_adamw_tensor* t, int64_t count, int64_t chunk, Take take, Put put, Go go) {
  Table tab;
  tab.count = 0;
  int64_t blocks = 0;
  for (int64_t k = 0; k <= count; ++k) {
    const bool here = k < count && take(t[k]);
    const int64_t more = here ? chunks_of(t[k].numel, chunk) : 0;
    if (tab.count && (k == count || (here && (tab.count == kRoom || blocks + more > kMaxBlocks)))) {
      const hipError_t e = go(tab, (uint32_t)blocks);
      if (e != hipSuccess) return e;
      tab.count = 0;
      blocks = 0;
    }
    if (!here) continue;
    tab.g[tab.count] = t[k].grad;
    tab.n[tab.count] = t[k].numel;
    tab.first[tab.count] = (uint32_t)blocks;
    put(tab, tab.count, k);
    ++tab.count;
    blocks += more;
  }
  return hipSuccess;
}

// (after check_tensors) what the norm's calls ask for; the result takes `result_bytes`
ssm_status check_norm(const ssm_adamw_tensor* tensors, int64_t count, double max_norm, float* result,
                      int64_t result_bytes, void* workspace, size_t workspace_bytes) {
  if (!result || !workspace) return SSM_ERR_NULL;
  if (!(max_norm > 0)) return SSM_ERR_UNSUPPORTED;
  if (misaligned(workspace) || (reinterpret_cast<uintptr_t>(result) & 3u)) return SSM_ERR_ALIGN;
  const size_t need = ssm_grad_norm_workspace_size(tensors, count);
  if (workspace_bytes < need) return SSM_ERR_WORKSPACE;
  const Range outs[] = {span(result, result_bytes), span(workspace, (int64_t)need)};
  if (overlaps(outs[0], outs[1])) return SSM_ERR_OVERLAP;
  for (int64_t k = 0; k < count; ++k) {
    const Range g = span(tensors[k].grad, tensors[k].numel * dtype_size(tensors[k].grad_dtype));
    if (overlaps(outs[0], g) || overlaps(outs[1], g)) return SSM_ERR_OVERLAP;
  }
  return SSM_OK;
}

ssm_status launch_norm(const ssm_adamw_tensor* tensors, int64_t count, double max_norm, float* result, void* workspace,
                       const ssm::AdamAdvance& adv, hipStream_t st) {
  int64_t chunks = 0;
  for (int64_t k = 0; k < count && chunks <= ssm::kSmallChunks; ++k)
    chunks += chunks_of(tensors[k].numel, ssm::kSmallChunk);
  if (count <= ssm::kSmallTensors && chunks <= ssm::kSmallChunks) {
    ssm::SmallNormTable t;
    uint32_t first = 0;
    for (int k = 0; k < (int)count; ++k) {
      t.g[k] = tensors[k].grad;
      t.n[k] = tensors[k].numel;
      t.first[k] = first;
      t.bf16[k] = tensors[k].grad_dtype == SSM_BF16;
      first += (uint32_t)chunks_of(tensors[k].numel, ssm::kSmallChunk);
    }
    t.count = (int)count;
    return launch_status(ssm::launch_norm_small(t, first, max_norm, result, adv, st));
  }
  double* part = static_cast<double*>(workspace);
  int64_t done = 0;
  for (int b = 0; b < 2; ++b) {
    const hipError_t e = in_tables<ssm::NormTable, ssm::kNormTensors>(
        tensors, count, ssm::kNormChunk,
        [&](const ssm_adamw_tensor& t) { return (t.grad_dtype == SSM_BF16) == (b == 1); },
        [](ssm::NormTable&, int, int64_t) {},
        [&](const ssm::NormTable& tab, uint32_t blocks) {
          const hipError_t r = ssm::launch_norm_part(tab, part + done, b == 1, blocks, st);
          done += blocks;
          return r;
        });
    if (e != hipSuccess) return SSM_ERR_LAUNCH;
  }
  return launch_status(ssm::launch_norm_join(part, done, max_norm, result, adv, st));
}

// what both step calls ask for, but for the step's number; `given`: what the step reads besides, `given_bytes` of it.
// *a gets the buffers and the settings.
ssm_status check_step(const ssm_adamw_config* c, const ssm_adamw_tensor* tensors, int64_t count, void* exp_avg,
                      void* exp_avg_sq, int16_t* exp_avg_base, int16_t* exp_avg_sq_base, float* master,
                      const void* given, int64_t given_bytes, ssm::AdamParams* a) {
  if (c->flags || (c->state_bits != 32 && c->state_bits != 8)) return SSM_ERR_UNSUPPORTED;
  if (!isfinite(c->lr) || !isfinite(c->weight_decay) || !finite_in(c->beta1, 0, 1) || !finite_in(c->beta2, 0, 1) ||
      c->beta1 == 1 || c->beta2 == 1 || !finite_in(c->eps, 1e-30, 1e30))
    return SSM_ERR_UNSUPPORTED;
  int64_t elems;
  const ssm_status rc = check_tensors(tensors, count, false, &elems);
  if (rc != SSM_OK) return rc;
  const bool s8 = c->state_bits == 8;
  if (!exp_avg || !exp_avg_sq || (s8 && (!exp_avg_base || !exp_avg_sq_base))) return SSM_ERR_NULL;
  if (!s8) exp_avg_base = exp_avg_sq_base = nullptr;
  const void* ptrs[] = {exp_avg, exp_avg_sq, exp_avg_base, exp_avg_sq_base, master};
  for (const void* q : ptrs)
    if (misaligned(q)) return SSM_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(given) & 3u) return SSM_ERR_ALIGN;
  const int64_t nb = elems / SSM_ADAMW_BLOCK;
  const Range outs[] = {span(exp_avg, elems * (s8 ? 1 : 4)), span(exp_avg_sq, elems * (s8 ? 1 : 4)),
                        span(exp_avg_base, nb * 2), span(exp_avg_sq_base, nb * 2), span(master, elems * 4)};
  const Range ins[] = {span(given, given_bytes)};
  if (any_overlap(outs, 5, ins, 1)) return SSM_ERR_OVERLAP;
  for (int64_t k = 0; k < count; ++k) {
    const Range p = span(tensors[k].param, tensors[k].numel * dtype_size(tensors[k].param_dtype));
    const Range g = span(tensors[k].grad, tensors[k].numel * dtype_size(tensors[k].grad_dtype));
    if (overlaps(p, ins[0])) return SSM_ERR_OVERLAP;
    for (const Range& o : outs)
      if (overlaps(o, p) || overlaps(o, g)) return SSM_ERR_OVERLAP;
  }
  if (params_clash(tensors, count)) return SSM_ERR_OVERLAP;

  memset(a, 0, sizeof(*a));
  a->m = exp_avg; a->v = exp_avg_sq; a->mb = exp_avg_base; a->vb = exp_avg_sq_base; a->master = master;
  a->b1 = (float)c->beta1; a->c1 = (float)(1 - c->beta1);
  a->b2 = (float)c->beta2; a->c2 = (float)(1 - c->beta2);
  a->eps = (float)c->eps;
  a->decay = (float)(1 - c->lr * c->weight_decay);
  return SSM_OK;
}

ssm_status launch_step(const ssm_adamw_config* c, const ssm_adamw_tensor* tensors, int64_t count,
                       const ssm::AdamParams& a, hipStream_t st) {
  for (int kind = 0; kind < 8; ++kind) {  // bit 0 bf16 params, bit 1 bf16 gradients, bit 2 masters
    const hipError_t e = in_tables<ssm::AdamTable, ssm::kAdamTensors>(
        tensors, count, ssm::kAdamChunk,
        [&](const ssm_adamw_tensor& t) {
          const bool pb = t.param_dtype == SSM_BF16;
          return kind == (pb ? 1 : 0) + (t.grad_dtype == SSM_BF16 ? 2 : 0) + (pb && a.master ? 4 : 0);
        },
        [&](ssm::AdamTable& tab, int i, int64_t k) {
          tab.p[i] = tensors[k].param;
          tab.off[i] = tensors[k].offset;
          tab.key[i] = a.progress ? (uint32_t)k : ssm::adam_key(c->seed, c->step, k);
        },
        [&](const ssm::AdamTable& tab, uint32_t blocks) {
          return ssm::launch_adamw(tab, a, kind + (c->state_bits == 8 ? 8 : 0), blocks, st);
        });
    if (e != hipSuccess) return SSM_ERR_LAUNCH;
  }
  return SSM_OK;
}

}  // namespace

extern "C" {

size_t ssm_grad_norm_workspace_size(const ssm_adamw_tensor* tensors, int64_t count) {
  if (!tensors || count < 1) return 0;
  int64_t n = 0;
  for (int64_t k = 0; k < count; ++k) {
    if (tensors[k].numel < 1 || tensors[k].numel > kMaxSize) return 0;
    n += chunks_of(tensors[k].numel, ssm::kNormChunk);
  }
  return (size_t)n * sizeof(double);
}

ssm_status ssm_grad_norm(const ssm_adamw_tensor* tensors, int64_t count, double max_norm, float* result,
                         void* workspace, size_t workspace_bytes, struct ihipStream_t* stream) {
  int64_t elems;
  const ssm_status rc = check_tensors(tensors, count, true, &elems);
  if (rc != SSM_OK) return rc;
  const ssm_status rn = check_norm(tensors, count, max_norm, result, 8, workspace, workspace_bytes);
  if (rn != SSM_OK) return rn;
  return launch_norm(tensors, count, max_norm, result, workspace, ssm::AdamAdvance{},
                     reinterpret_cast<hipStream_t>(stream));
}

ssm_status ssm_adamw_step(const ssm_adamw_config* c, const ssm_adamw_tensor* tensors, int64_t count, void* exp_avg,
                          void* exp_avg_sq, int16_t* exp_avg_base, int16_t* exp_avg_sq_base, float* master,
                          const float* clip, struct ihipStream_t* stream) {
  if (!c) return SSM_ERR_NULL;
  if (c->step < 1) return SSM_ERR_UNSUPPORTED;
  ssm::AdamParams a;
  const ssm_status rc = check_step(c, tensors, count, exp_avg, exp_avg_sq, exp_avg_base, exp_avg_sq_base, master, clip,
                                   8, &a);
  if (rc != SSM_OK) return rc;
  a.clip = clip;
  a.isb = (float)(1 / sqrt(1 - pow(c->beta2, (double)c->step)));
  a.step = (float)(c->lr / (1 - pow(c->beta1, (double)c->step)));
  return launch_step(c, tensors, count, a, reinterpret_cast<hipStream_t>(stream));
}

ssm_status ssm_adamw_clipped_step(const ssm_adamw_config* c, const ssm_adamw_tensor* tensors, int64_t count,
                                  double max_norm, void* exp_avg, void* exp_avg_sq, int16_t* exp_avg_base,
                                  int16_t* exp_avg_sq_base, float* master, ssm_adamw_progress* progress, float* norm,
                                  void* workspace, size_t workspace_bytes, struct ihipStream_t* stream) {
  static_assert(sizeof(ssm::AdamProgress) == sizeof(ssm_adamw_progress), "one struct in two places");
  if (!c || !progress) return SSM_ERR_NULL;
  ssm::AdamParams a;
  ssm_status rc = check_step(c, tensors, count, exp_avg, exp_avg_sq, exp_avg_base, exp_avg_sq_base, master, progress,
                             (int64_t)sizeof(*progress), &a);
  if (rc != SSM_OK) return rc;
  rc = check_norm(tensors, count, max_norm, norm, 4, workspace, workspace_bytes);
  if (rc != SSM_OK) return rc;
  if (misaligned(progress)) return SSM_ERR_ALIGN;
  const int64_t bytes = (int64_t)ssm_grad_norm_workspace_size(tensors, count);
  const Range own[] = {span(norm, 4), span(workspace, bytes), span(progress, (int64_t)sizeof(*progress))};
  if (any_overlap(own, 3, nullptr, 0)) return SSM_ERR_OVERLAP;
  const int64_t elems = tensors[count - 1].offset + chunks_of(tensors[count - 1].numel, SSM_ADAMW_BLOCK) * SSM_ADAMW_BLOCK;
  const int64_t es = c->state_bits == 8 ? 1 : 4, nb = elems / SSM_ADAMW_BLOCK * 2;
  const Range states[] = {span(a.m, elems * es), span(a.v, elems * es), span(a.mb, nb), span(a.vb, nb),
                          span(a.master, elems * 4)};
  for (int i = 0; i < 2; ++i) {
    for (const Range& q : states)
      if (overlaps(own[i], q)) return SSM_ERR_OVERLAP;
    for (int64_t k = 0; k < count; ++k)
      if (overlaps(own[i], span(tensors[k].param, tensors[k].numel * dtype_size(tensors[k].param_dtype))))
        return SSM_ERR_OVERLAP;
  }
  for (int64_t k = 0; k < count; ++k)
    if (overlaps(own[2], span(tensors[k].grad, tensors[k].numel * dtype_size(tensors[k].grad_dtype))))
      return SSM_ERR_OVERLAP;

  a.progress = reinterpret_cast<ssm::AdamProgress*>(progress);
  const ssm::AdamAdvance adv{reinterpret_cast<ssm::AdamProgress*>(progress), c->lr, c->beta1, c->beta2,
                             ssm::adam_seed(c->seed)};
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  rc = launch_norm(tensors, count, max_norm, norm, workspace, adv, st);
  return rc != SSM_OK ? rc : launch_step(c, tensors, count, a, st);
}

ssm_status ssm_adamw_state_values(int64_t numel, const void* exp_avg, const void* exp_avg_sq,
                                  const int16_t* exp_avg_base, const int16_t* exp_avg_sq_base, void* m_values,
                                  void* v_values, struct ihipStream_t* stream) {
  if (numel < 1 || numel > kMaxSize || numel % SSM_ADAMW_BLOCK) return SSM_ERR_SHAPE;
  if (!m_values && !v_values) return SSM_ERR_NULL;
  if (m_values && (!exp_avg || !exp_avg_base)) return SSM_ERR_NULL;
  if (v_values && (!exp_avg_sq || !exp_avg_sq_base)) return SSM_ERR_NULL;
  const void* ptrs[] = {exp_avg, exp_avg_sq, exp_avg_base, exp_avg_sq_base, m_values, v_values};
  for (const void* q : ptrs)
    if (misaligned(q)) return SSM_ERR_ALIGN;
  const int64_t nb = numel / SSM_ADAMW_BLOCK;
  const Range ins[] = {span(exp_avg, numel), span(exp_avg_sq, numel), span(exp_avg_base, nb * 2),
                       span(exp_avg_sq_base, nb * 2)};
  const Range outs[] = {span(m_values, numel * 2), span(v_values, numel * 2)};
  if (any_overlap(outs, 2, ins, 4)) return SSM_ERR_OVERLAP;
  return launch_status(ssm::launch_state_values(numel, exp_avg, exp_avg_sq, exp_avg_base, exp_avg_sq_base, m_values,
                                                v_values, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
