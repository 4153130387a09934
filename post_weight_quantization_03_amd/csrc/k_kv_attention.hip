// Attention over the paged 8-bit cache: which kernel takes a call, and how long
// sequences are split.
#include "kv_attend.h"

namespace gptq {
namespace {

struct Plan {
  int tile_rows, nsplit;
  int64_t chunk;
};

Plan make_plan(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  const int64_t rows = b.max_new * (a.q_heads / c.kv_heads);
  Plan p;
  if (rows <= 64)
    p.tile_rows = rows > 16 && c.dim < 256 ? 32 : 16;
  else
    p.tile_rows = rows > 128 && c.dim < 256 ? 256 : 128;
  const int64_t tiles = (rows + p.tile_rows - 1) / p.tile_rows;
  const int64_t base = b.batch * c.kv_heads * tiles;
  // tokens a tile may see, with the rounding of its first
  int64_t span = b.max_kv;
  if (a.window > 0 && a.window + b.max_new < span) span = a.window + b.max_new;
  span += 63;
  const int64_t want = (512 + base - 1) / base;
  int64_t chunk = (span + want - 1) / want;
  chunk = (chunk + 255) / 256 * 256;
  p.chunk = chunk;
  p.nsplit = (int)((span + chunk - 1) / chunk);
  return p;
}

}  // namespace

size_t kv_attention_workspace(const gptq_kv_cache& cache, const gptq_kv_batch& batch, bool, const gptq_attention& a) {
  const Plan p = make_plan(cache, batch, a);
  if (p.nsplit <= 1) return 0;
  return (size_t)batch.total * a.q_heads * p.nsplit * (cache.dim + 1) * sizeof(float);
}

bool kv_attention_fits(const gptq_kv_cache& c, const gptq_kv_batch& b, const gptq_attention& a) {
  const int64_t limit = ((int64_t)1 << 32) - 1;
  const Plan p = make_plan(c, b, a);
  // a workgroup a row and head where splits are joined
  if (p.nsplit > 1 && b.batch * b.max_new > limit / 256 / a.q_heads) return false;
  const int64_t rows = b.max_new * (a.q_heads / c.kv_heads);
  const int64_t tiles = (rows + p.tile_rows - 1) / p.tile_rows;
  return b.batch * c.kv_heads * tiles * p.nsplit <= limit / (p.tile_rows == 256 ? 512 : 256);
}

hipError_t kv_attention(const KvAttention& a, hipStream_t stream) {
  const Plan p = make_plan(a.cache, a.batch, a.a);
  Partials w{nullptr, nullptr, p.nsplit, p.chunk};
  if (p.nsplit > 1) {
    w.out = static_cast<float*>(a.workspace);
    w.lse2 = w.out + (size_t)a.batch.total * a.a.q_heads * p.nsplit * a.cache.dim;
  }
  const hipError_t e = p.tile_rows >= 128 ? kv_prompt_launch(a, w, p.tile_rows, stream)
                                          : kv_rows_launch(a, w, p.tile_rows, stream);
  return e == hipSuccess && p.nsplit > 1 ? kv_join_launch(a, w, p.tile_rows, stream) : e;
}

}  // namespace gptq
