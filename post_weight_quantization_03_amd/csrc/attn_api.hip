// C ABI of the attention operators: argument checks on the host and the launch of
// each entry point.  Every declaration is documented in include/gptq_attn.h.
#include <math.h>

#include "attn.h"

namespace {

using namespace gptq;

constexpr int64_t MAX_DIM = (int64_t)1 << 30;
constexpr int64_t MAX_WORK = INT32_MAX;             // lanes of the norm and rotation, counted in 32 bits
constexpr int64_t MAX_GRID = ((int64_t)1 << 24) - 1;  // workgroups of 256 threads: fewer than 2^32 threads a launch

bool dtype_ok(gptq_dtype dt) { return dt == GPTQ_BF16 || dt == GPTQ_F32; }
int64_t elem_size(gptq_dtype dt) { return dt == GPTQ_BF16 ? 2 : 4; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool stride_ok(int64_t s) { return s > -((int64_t)1 << 40) && s < ((int64_t)1 << 40); }

// Whether 16-byte vectors reach every element run of 8: pointer, token and head strides.
bool vec_ok(const void* p, int64_t st, int64_t sh, gptq_dtype dt) {
  const int64_t per = 16 / elem_size(dt);
  return aligned(p, 16) && st % per == 0 && sh % per == 0;
}

int rope_check(const gptq_rope* r, int32_t dim) {
  if (r->rot < 0 || r->rot > dim || !(r->interleaved == 0 || r->interleaved == 1)) return GPTQ_EINVAL;
  if (!(r->eps >= 0.0f) || !(r->eps < INFINITY) || r->max_pos < 0) return GPTQ_EINVAL;
  if (r->rot % 16 != 0) return GPTQ_EUNSUPPORTED;
  if (r->rot > 0 && (!r->cos || !r->sin)) return GPTQ_EINVAL;
  if (r->rot > 0 && (!aligned(r->cos, 16) || !aligned(r->sin, 16))) return GPTQ_EINVAL;
  return GPTQ_OK;
}

int cache_check(const gptq_kv_cache* c) {
  if (!c || c->pages < 0 || c->pages > MAX_DIM || c->kv_heads < 1 || c->kv_heads > 65536) return GPTQ_EINVAL;
  if (c->block <= 0 || c->dim <= 0) return GPTQ_EINVAL;
  if (!kv_block_ok(c->block) || !kv_dim_ok(c->dim)) return GPTQ_EUNSUPPORTED;
  return GPTQ_OK;
}
int cache_pointers(const gptq_kv_cache* c) {
  if (c->pages < 1 || !c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return GPTQ_EINVAL;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 4) || !aligned(c->v_scales, 4))
    return GPTQ_EINVAL;
  return GPTQ_OK;
}

int batch_check(const gptq_kv_batch* b, const gptq_kv_cache* c) {
  if (!b || b->batch < 0 || b->batch > MAX_DIM || b->total < 0 || b->total > MAX_DIM || b->max_new < 0 ||
      b->max_new > MAX_DIM || b->max_kv < 0 || b->max_kv > MAX_DIM)
    return GPTQ_EINVAL;
  if (b->table_stride < (b->max_kv + c->block - 1) / c->block || !stride_ok(b->table_stride)) return GPTQ_EINVAL;
  return GPTQ_OK;
}
bool batch_empty(const gptq_kv_batch* b) { return b->batch == 0 || b->total == 0 || b->max_new == 0; }
bool batch_pointers(const gptq_kv_batch* b) {
  return b->q_start && b->kv_len && (b->block_table || b->max_kv == 0) && aligned(b->q_start, 4) &&
         aligned(b->kv_len, 4) && aligned(b->block_table, 4);
}

// The heads of one side in a norm-and-rotation call, forward (y) or backward (dy, dx).
// Without tokens no element is pointed at.
int side_check(const gptq_heads* s, gptq_dtype dt, bool any, HeadSide* out, bool* vec) {
  *out = HeadSide{};
  if (!s || s->heads == 0) return GPTQ_OK;
  if (s->heads < 0 || s->heads > 65536 || (any && (!s->x || !s->y))) return GPTQ_EINVAL;
  if (!stride_ok(s->x_token) || !stride_ok(s->x_head) || !stride_ok(s->y_token) || !stride_ok(s->y_head))
    return GPTQ_EINVAL;
  const uintptr_t a = (uintptr_t)elem_size(dt);
  if (!aligned(s->x, a) || !aligned(s->y, a) || !aligned(s->weight, a)) return GPTQ_EINVAL;
  if (any && s->x == s->y && (s->x_token != s->y_token || s->x_head != s->y_head)) return GPTQ_EINVAL;
  *vec = *vec && vec_ok(s->x, s->x_token, s->x_head, dt) && vec_ok(s->y, s->y_token, s->y_head, dt) &&
         aligned(s->weight, 16);
  out->x = s->x, out->x_token = s->x_token, out->x_head = s->x_head;
  out->y = s->y, out->y_token = s->y_token, out->y_head = s->y_head;
  out->weight = s->weight, out->heads = s->heads;
  return GPTQ_OK;
}
int side_check(const gptq_heads_grad* s, gptq_dtype dt, bool any, HeadSide* out, bool* vec) {
  *out = HeadSide{};
  if (!s) return GPTQ_OK;
  if (s->heads == 0) {
    out->weight = s->weight;  // its gradient is written: 0
    return aligned(s->dweight, 4) ? GPTQ_OK : GPTQ_EINVAL;
  }
  if (s->heads < 0 || s->heads > 65536 || (any && (!s->dy || !s->dx || (s->weight && !s->x)))) return GPTQ_EINVAL;
  if (!stride_ok(s->dy_token) || !stride_ok(s->dy_head) || !stride_ok(s->dx_token) || !stride_ok(s->dx_head) ||
      (s->weight && (!stride_ok(s->x_token) || !stride_ok(s->x_head))))
    return GPTQ_EINVAL;
  const uintptr_t a = (uintptr_t)elem_size(dt);
  if (!aligned(s->dy, a) || !aligned(s->dx, a) || !aligned(s->weight, a) || (s->weight && !aligned(s->x, a)) ||
      !aligned(s->dweight, 4))
    return GPTQ_EINVAL;
  if (any && s->dy == s->dx && (s->dy_token != s->dx_token || s->dy_head != s->dx_head)) return GPTQ_EINVAL;
  if (any && s->weight && s->x == s->dx) return GPTQ_EINVAL;
  *vec = *vec && vec_ok(s->dy, s->dy_token, s->dy_head, dt) && vec_ok(s->dx, s->dx_token, s->dx_head, dt) &&
         aligned(s->weight, 16) && (!s->weight || vec_ok(s->x, s->x_token, s->x_head, dt));
  out->dy = s->dy, out->dy_token = s->dy_token, out->dy_head = s->dy_head;
  out->y = s->dx, out->y_token = s->dx_token, out->y_head = s->dx_head;
  out->x = s->x, out->x_token = s->x_token, out->x_head = s->x_head;
  out->weight = s->weight, out->heads = s->heads;
  return GPTQ_OK;
}

template <typename Heads>
int norm_rope_args(const Heads* q, const Heads* k, gptq_dtype dt, int64_t tokens, int32_t dim,
                   const int32_t* positions, const gptq_rope* rope, int32_t* d_status, NormRope* a) {
  if (!dtype_ok(dt) || tokens < 0 || tokens > MAX_DIM || dim <= 0 || !rope) return GPTQ_EINVAL;
  if (dim % 16 != 0 || dim > 512) return GPTQ_EUNSUPPORTED;
  int st = rope_check(rope, dim);
  if (st != GPTQ_OK) return st;
  *a = NormRope{};
  bool vec = true;
  if ((st = side_check(q, dt, tokens > 0, &a->q, &vec)) != GPTQ_OK) return st;
  if ((st = side_check(k, dt, tokens > 0, &a->k, &vec)) != GPTQ_OK) return st;
  // a position out of range is replaced by 0, so there has to be a row 0 of cos and sin
  if (tokens > 0 && a->q.heads + a->k.heads > 0 && rope->rot > 0 &&
      (!positions || !aligned(positions, 4) || rope->max_pos < 1))
    return GPTQ_EINVAL;
  if (!aligned(d_status, 4)) return GPTQ_EINVAL;
  // an item (token and heads) and a thread of it are counted in 32 bits
  if (tokens * ((int64_t)a->q.heads + a->k.heads) > MAX_WORK / head_lanes(dim)) return GPTQ_EUNSUPPORTED;
  a->bf16 = dt == GPTQ_BF16;
  a->vec = vec;
  a->tokens = tokens;
  a->dim = dim;
  a->positions = positions;
  a->rope = *rope;
  a->d_status = d_status;
  return GPTQ_OK;
}

}  // namespace

extern "C" {

int gptq_qk_norm_rope(const gptq_heads* q, const gptq_heads* k, gptq_dtype dtype, int64_t tokens, int32_t dim,
                      const int32_t* positions, const gptq_rope* rope, int32_t* d_status, gptq_stream_t stream) {
  NormRope a;
  const int st = norm_rope_args(q, k, dtype, tokens, dim, positions, rope, d_status, &a);
  if (st != GPTQ_OK) return st;
  if (tokens == 0 || a.q.heads + a.k.heads == 0) return GPTQ_OK;
  return qk_norm_rope(a, (hipStream_t)stream) == hipSuccess ? GPTQ_OK : GPTQ_EHIP;
}

size_t gptq_qk_norm_rope_backward_workspace_bytes(int64_t tokens, int32_t dim, int32_t q_heads, int32_t k_heads) {
  if (tokens <= 0 || tokens > MAX_DIM || dim <= 0 || dim % 16 != 0 || dim > 512 || q_heads < 0 || k_heads < 0 ||
      q_heads > 65536 || k_heads > 65536)
    return 0;
  return (size_t)(norm_rope_partials(tokens, dim, q_heads) + norm_rope_partials(tokens, dim, k_heads)) * dim *
         sizeof(float);
}

int gptq_qk_norm_rope_backward(const gptq_heads_grad* q, const gptq_heads_grad* k, gptq_dtype dtype, int64_t tokens,
                               int32_t dim, const int32_t* positions, const gptq_rope* rope, void* workspace,
                               size_t workspace_bytes, int32_t* d_status, gptq_stream_t stream) {
  NormRope a;
  const int st = norm_rope_args(q, k, dtype, tokens, dim, positions, rope, d_status, &a);
  if (st != GPTQ_OK) return st;
  float* dqw = a.q.weight ? q->dweight : nullptr;
  float* dkw = a.k.weight ? k->dweight : nullptr;
  if ((tokens == 0 || a.q.heads + a.k.heads == 0) && !dqw && !dkw) return GPTQ_OK;
  if ((a.q.weight && a.q.heads) || (a.k.weight && a.k.heads)) {
    const size_t need = gptq_qk_norm_rope_backward_workspace_bytes(tokens, dim, a.q.heads, a.k.heads);
    if (workspace_bytes < need || (need > 0 && !workspace)) return GPTQ_EWORKSPACE;
    if (!aligned(workspace, 4)) return GPTQ_EINVAL;
  }
  return qk_norm_rope_backward(a, dqw, dkw, static_cast<float*>(workspace), (hipStream_t)stream) == hipSuccess
             ? GPTQ_OK
             : GPTQ_EHIP;
}

int gptq_kv_append(const gptq_kv_cache* cache, const gptq_kv_batch* batch, const void* k, int64_t k_token,
                   int64_t k_head, const void* v, int64_t v_token, int64_t v_head, gptq_dtype dtype,
                   const void* k_weight, const gptq_rope* rope, int32_t* d_status, gptq_stream_t stream) {
  int st = cache_check(cache);
  if (st != GPTQ_OK) return st;
  if ((st = batch_check(batch, cache)) != GPTQ_OK) return st;
  if (!dtype_ok(dtype) || !stride_ok(k_token) || !stride_ok(k_head) || !stride_ok(v_token) || !stride_ok(v_head) ||
      !aligned(d_status, 4))
    return GPTQ_EINVAL;
  if (rope && (st = rope_check(rope, cache->dim)) != GPTQ_OK) return st;
  if (k_weight && !rope) return GPTQ_EINVAL;  // the norm's eps is in gptq_rope
  if (batch_empty(batch)) return GPTQ_OK;
  if ((st = cache_pointers(cache)) != GPTQ_OK) return st;
  const uintptr_t e = (uintptr_t)elem_size(dtype);
  if (!batch_pointers(batch) || !k || !v || !aligned(k, e) || !aligned(v, e) || !aligned(k_weight, e))
    return GPTQ_EINVAL;
  const int64_t nblk = (batch->max_new + cache->block - 2) / cache->block + 1;
  if (batch->batch * nblk > MAX_GRID / (2 * (int64_t)cache->kv_heads)) return GPTQ_EUNSUPPORTED;
  KvAppend a{};
  a.cache = *cache;
  a.batch = *batch;
  a.k = k, a.k_token = k_token, a.k_head = k_head;
  a.v = v, a.v_token = v_token, a.v_head = v_head;
  a.bf16 = dtype == GPTQ_BF16;
  a.vec = vec_ok(k, k_token, k_head, dtype) && vec_ok(v, v_token, v_head, dtype) && aligned(k_weight, 16);
  a.k_weight = k_weight;
  if (rope) a.rope = *rope;
  a.d_status = d_status;
  return kv_append(a, (hipStream_t)stream) == hipSuccess ? GPTQ_OK : GPTQ_EHIP;
}

int gptq_kv_read(const gptq_kv_cache* cache, const gptq_kv_batch* batch, void* k, int64_t k_token, int64_t k_head,
                 void* v, int64_t v_token, int64_t v_head, gptq_dtype dtype, int32_t* d_status,
                 gptq_stream_t stream) {
  int st = cache_check(cache);
  if (st != GPTQ_OK) return st;
  if ((st = batch_check(batch, cache)) != GPTQ_OK) return st;
  if (!dtype_ok(dtype) || !stride_ok(k_token) || !stride_ok(k_head) || !stride_ok(v_token) || !stride_ok(v_head) ||
      !aligned(d_status, 4))
    return GPTQ_EINVAL;
  if (batch_empty(batch) || (!k && !v)) return GPTQ_OK;
  if ((st = cache_pointers(cache)) != GPTQ_OK) return st;
  const uintptr_t e = (uintptr_t)elem_size(dtype);
  if (!batch_pointers(batch) || !aligned(k, e) || !aligned(v, e)) return GPTQ_EINVAL;
  const int64_t ntile = (batch->max_new + 78) / 64;
  if (batch->batch * ntile > MAX_GRID / (2 * (int64_t)cache->kv_heads)) return GPTQ_EUNSUPPORTED;
  KvRead a{};
  a.cache = *cache;
  a.batch = *batch;
  a.k = k, a.k_token = k_token, a.k_head = k_head;
  a.v = v, a.v_token = v_token, a.v_head = v_head;
  a.bf16 = dtype == GPTQ_BF16;
  a.vec = (!k || vec_ok(k, k_token, k_head, dtype)) && (!v || vec_ok(v, v_token, v_head, dtype));
  a.d_status = d_status;
  return kv_read(a, (hipStream_t)stream) == hipSuccess ? GPTQ_OK : GPTQ_EHIP;
}

static int attention_check(const gptq_kv_cache* cache, const gptq_kv_batch* batch, gptq_dtype dtype,
                           const gptq_attention* a) {
  int st = cache_check(cache);
  if (st != GPTQ_OK) return st;
  if ((st = batch_check(batch, cache)) != GPTQ_OK) return st;
  if (!a || !dtype_ok(dtype) || a->q_heads < 1 || a->q_heads > 65536 || a->q_heads % cache->kv_heads != 0 ||
      !(fabsf(a->sm_scale) < INFINITY) || !(a->causal == 0 || a->causal == 1) || a->window < 0)
    return GPTQ_EINVAL;
  return GPTQ_OK;
}

// A window that no sequence outgrows is no window (places are below max_kv); what is left of it stays below
// 2^30, so sums with it fit.
static gptq_attention limited(const gptq_attention* a, const gptq_kv_batch* batch) {
  gptq_attention r = *a;
  if (r.window >= batch->max_kv) r.window = 0;
  return r;
}

static int mask_check(const gptq_kv_batch* batch, const gptq_attention* a, const gptq_kv_mask* m) {
  if (!m || m->sinks < 0) return GPTQ_EINVAL;
  if (m->tree && (!a->causal || m->tree_stride < (batch->max_new + 63) / 64 || !stride_ok(m->tree_stride)))
    return GPTQ_EINVAL;
  return GPTQ_OK;
}

// First tokens that count: none without a window, and no more than a sequence has.
static int64_t counted_sinks(const gptq_attention& seen, const gptq_kv_batch* batch, const gptq_kv_mask* m) {
  if (!m || seen.window == 0) return 0;
  return m->sinks < batch->max_kv ? m->sinks : batch->max_kv;
}

static size_t workspace_of(const gptq_kv_cache* cache, const gptq_kv_batch* batch, gptq_dtype dtype,
                           const gptq_attention* a, const gptq_kv_mask* mask) {
  if (batch_empty(batch)) return 0;
  const gptq_attention seen = limited(a, batch);
  return kv_attention_workspace(*cache, *batch, dtype == GPTQ_BF16, seen, counted_sinks(seen, batch, mask));
}

size_t gptq_kv_attention_workspace_bytes(const gptq_kv_cache* cache, const gptq_kv_batch* batch, gptq_dtype dtype,
                                         const gptq_attention* a) {
  if (attention_check(cache, batch, dtype, a) != GPTQ_OK) return 0;
  return workspace_of(cache, batch, dtype, a, nullptr);
}

size_t gptq_kv_masked_attention_workspace_bytes(const gptq_kv_cache* cache, const gptq_kv_batch* batch,
                                                gptq_dtype dtype, const gptq_attention* a, const gptq_kv_mask* mask) {
  if (attention_check(cache, batch, dtype, a) != GPTQ_OK || mask_check(batch, a, mask) != GPTQ_OK) return 0;
  return workspace_of(cache, batch, dtype, a, mask);
}

// The call behind both entry points; mask NULL: none.
static int attend(const gptq_kv_cache* cache, const gptq_kv_batch* batch, const gptq_attention* att,
                  const gptq_kv_mask* mask, const void* q, int64_t q_token, int64_t q_head, void* out,
                  int64_t out_token, int64_t out_head, float* lse, gptq_dtype dtype, void* workspace,
                  size_t workspace_bytes, int32_t* d_status, gptq_stream_t stream) {
  int st;
  if (!stride_ok(q_token) || !stride_ok(q_head) || !stride_ok(out_token) || !stride_ok(out_head) ||
      !aligned(d_status, 4))
    return GPTQ_EINVAL;
  if (batch_empty(batch)) return GPTQ_OK;
  const uintptr_t e = (uintptr_t)elem_size(dtype);
  if (!q || !out || q == out || !aligned(q, e) || !aligned(out, e) || !aligned(lse, 4) || !batch_pointers(batch))
    return GPTQ_EINVAL;
  // with no token in any sequence no page exists to be pointed at
  if (batch->max_kv > 0 && (st = cache_pointers(cache)) != GPTQ_OK) return st;
  const gptq_attention seen = limited(att, batch);
  const int64_t sinks = counted_sinks(seen, batch, mask);
  const bool tree = mask && mask->tree;
  if (tree && (!aligned(mask->tree, 8) || (seen.window > 0 && (!mask->positions || !aligned(mask->positions, 4)))))
    return GPTQ_EINVAL;
  if (!kv_attention_fits(*cache, *batch, dtype == GPTQ_BF16, seen, sinks)) return GPTQ_EUNSUPPORTED;
  const size_t need = kv_attention_workspace(*cache, *batch, dtype == GPTQ_BF16, seen, sinks);
  if (workspace_bytes < need || (need > 0 && !workspace)) return GPTQ_EWORKSPACE;
  if (need > 0 && !aligned(workspace, 16)) return GPTQ_EINVAL;
  KvAttention a{};
  a.cache = *cache;
  a.batch = *batch;
  a.a = seen;
  a.q = q, a.q_token = q_token, a.q_head = q_head;
  a.out = out, a.out_token = out_token, a.out_head = out_head;
  a.lse = lse;
  a.bf16 = dtype == GPTQ_BF16;
  a.vec = vec_ok(q, q_token, q_head, dtype) && vec_ok(out, out_token, out_head, dtype);
  a.workspace = workspace;
  a.d_status = d_status;
  // a window without first tokens too: the plain kernels look up the blocks of a whole tile at its edge
  a.masked = tree || (mask && seen.window > 0);
  if (a.masked) a.mask = *mask;
  a.mask.sinks = sinks;
  return kv_attention(a, (hipStream_t)stream) == hipSuccess ? GPTQ_OK : GPTQ_EHIP;
}

int gptq_kv_attention(const gptq_kv_cache* cache, const gptq_kv_batch* batch, const gptq_attention* att, const void* q,
                      int64_t q_token, int64_t q_head, void* out, int64_t out_token, int64_t out_head, float* lse,
                      gptq_dtype dtype, void* workspace, size_t workspace_bytes, int32_t* d_status,
                      gptq_stream_t stream) {
  const int st = attention_check(cache, batch, dtype, att);
  if (st != GPTQ_OK) return st;
  return attend(cache, batch, att, nullptr, q, q_token, q_head, out, out_token, out_head, lse, dtype, workspace,
                workspace_bytes, d_status, stream);
}

int gptq_kv_masked_attention(const gptq_kv_cache* cache, const gptq_kv_batch* batch, const gptq_attention* att,
                             const gptq_kv_mask* mask, const void* q, int64_t q_token, int64_t q_head, void* out,
                             int64_t out_token, int64_t out_head, float* lse, gptq_dtype dtype, void* workspace,
                             size_t workspace_bytes, int32_t* d_status, gptq_stream_t stream) {
  int st = attention_check(cache, batch, dtype, att);
  if (st != GPTQ_OK || (st = mask_check(batch, att, mask)) != GPTQ_OK) return st;
  return attend(cache, batch, att, mask, q, q_token, q_head, out, out_token, out_head, lse, dtype, workspace,
                workspace_bytes, d_status, stream);
}

int gptq_kv_tree(const gptq_kv_batch* batch, const int32_t* parents, int64_t window, int64_t sinks,
                 int32_t* positions, uint64_t* tree, int64_t tree_stride, int32_t* d_status, gptq_stream_t stream) {
  if (!batch || batch->batch < 0 || batch->batch > MAX_DIM || batch->total < 0 || batch->total > MAX_DIM ||
      batch->max_new < 0 || batch->max_new > MAX_DIM || batch->max_kv < 0 || batch->max_kv > MAX_DIM)
    return GPTQ_EINVAL;
  if (window < 0 || sinks < 0 || tree_stride < (batch->max_new + 63) / 64 || !stride_ok(tree_stride) ||
      !aligned(d_status, 4))
    return GPTQ_EINVAL;
  if (batch_empty(batch)) return GPTQ_OK;
  if (!batch->q_start || !batch->kv_len || !parents || !positions || !tree || !aligned(batch->q_start, 4) ||
      !aligned(batch->kv_len, 4) || !aligned(parents, 4) || !aligned(positions, 4) || !aligned(tree, 8) ||
      parents == positions)
    return GPTQ_EINVAL;
  if (!kv_tree_fits(*batch)) return GPTQ_EUNSUPPORTED;
  return kv_tree(*batch, parents, window, sinks, positions, tree, tree_stride, d_status, (hipStream_t)stream) ==
                 hipSuccess
             ? GPTQ_OK
             : GPTQ_EHIP;
}

}  // extern "C"
