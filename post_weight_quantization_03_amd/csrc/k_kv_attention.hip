// Attention over the paged 8-bit cache: which kernel takes a call, and how long
// sequences are split.  The host knows the sizes of a call but not its sequences'
// lengths (max_kv bounds them), so the rules go by sizes.
#include "kv_attend.h"

namespace gptq {
namespace {

struct Plan {
  int tile_rows, nsplit;
  int64_t chunk, base;  // base: workgroups without splits
};

// a * b, or the largest number where that is larger (a, b >= 0): sizes each in range can have a product past 64 bits.
int64_t product(int64_t a, int64_t b) { return a != 0 && b > INT64_MAX / a ? INT64_MAX : a * b; }

// Rows (query tokens times heads of a key head's group) a workgroup takes.  Measured with groups of 4
// over 4 x 30000, 16 x 2000 and 1 x 8000 tokens, 8 key heads (us, tiles of 16 / 32 / 128 / 256 rows):
//   dim 128 bf16:   32 rows   83 / 93 / 121 / 191     32 / 31 / 52 / 83     18 / 18 / 22 / 25
//                   64       149 / 112 / 128 / 196    47 / 46 / 61 / 93     23 / 25 / 25 / 28
//                  128       284 / 198 / 120 / 175    86 / 64 / 51 / 60     32 / 31 / 27 / 31
//                  200       474 / 419 / 222 / 187   132 / 117 / 76 / 77    54 / 54 / 34 / 34
//   dim 128 fp32:   64       157 / 280 / 260 / 232    49 / 75 / 95 / 107    24 / 32 / 34 / 31
//                  128       292 / 523 / 265 / 235    89 / 124 / 89 / 76    33 / 46 / 38 / 35
//   dim 64 bf16:    64        88 / 68 / 97 / 183      29 / 31 / 50 / 82     16 / 17 / 19 / 23
//                  800       821 / 822 / 386 / 471   224 / 226 / 117 / 155  83 / 82 / 57 / 69
//   dim 256, 4 key heads, tiles of 16 / 128 rows:
//           bf16:  64 rows  167 / 174     66 / 78     34 / 39
//                  80       251 / 176     88 / 79     45 / 40
//                 128       315 / 155     98 / 73     46 / 41
//           fp32:  64       159 / 444     64 / 141    35 / 56
//                 128       297 / 434     95 / 139    46 / 59    four prompts of 1024 tokens 277 / 209
// fp32 keeps two parts of queries and weights in registers: at dim 128 its tiles of 32 rows and its 4 waves of
// 32 spill, and so do forms that are kept, by bytes a lane: 8 waves of dim 128 in fp32 68, 4 waves of dim 128 in
// bf16 20, of dim 256 116 in bf16 and 452 in fp32.  dim 256 fits 16 rows, or 4 waves of 32; in fp32 its rule is bf16's, which
// gains in several short prompts and costs other calls a fifth to a half.
int tile_rows_for(int64_t rows, int dim, bool bf16) {
  if (dim == 256) return rows <= 64 ? 16 : 128;
  if (rows <= 32) return 16;
  if (dim == 128 && !bf16) return rows <= 64 ? 16 : 256;
  if (rows <= 64) return 32;
  return rows <= 128 || dim == 64 ? 128 : 256;
}

Plan make_plan(const gptq_kv_cache& c, const gptq_kv_batch& b, bool bf16, const gptq_attention& a) {
  const int64_t rows = b.max_new * (a.q_heads / c.kv_heads);
  Plan p;
  p.tile_rows = tile_rows_for(rows, c.dim, bf16);
  const int64_t base = product(b.batch * c.kv_heads, (rows + p.tile_rows - 1) / p.tile_rows);
  p.base = base;
  // tokens a tile may see, with the rounding of its first
  int64_t span = b.max_kv;
  if (a.window > 0 && a.window + b.max_new < span) span = a.window + b.max_new;
  span += 63;
  int64_t chunk;
  if (p.tile_rows < 128) {
    // Two workgroups of four waves a CU are resident: one round of 512 (one token over 131035 tokens, 8 key
    // heads, chunks of 1024 / 2048 / 2304 / 4096: 60 / 56 / 60 / 88 us).  From 512 on no split is needed for
    // the chip to be full (64 sequences of up to 8192, 32 heads: 455 to 475 us whole, 521 in two).
    const int64_t want = base >= 512 ? 1 : (512 + base - 1) / base;
    chunk = want == 1 ? span : (span / want + 128) / 256 * 256;
  } else {
    // One workgroup of eight waves a CU.  It starts and ends in the time of 5 tiles of 64 tokens, and its
    // partial results cost a join, so one round of 256 does where chunks stay below 4096 tokens; above, up
    // to three, which even out sequences of different lengths (500 tokens each over 6000 to 12001: 449 us
    // whole, 382 in two, 350 in three, and 25 for the join).  512 tokens each, in 1 / 2 / 3 parts and by this rule:
    //   192 workgroups  6000 tokens 183 / 219 / 223, 278    6000 to 12000  323 / 367 / 290, 289
    //   256             6000        246 / 258 / 258, 279   12000 to 24000  880 / 801 / 739, 739
    //   448             6000        365 / 446 / 471         6000 to 12000  612 / 645 / 673
    //   896             6000        750 / 860 / 920         6000 to 12000 1154 / 1304 / 1325
    // so below 448 it serves unequal sequences, at the cost of equal ones, and from 448 on none is split.
    chunk = base >= 448 ? span : span * base / 256;
    if (base < 448 && chunk > 4096) chunk = span * base / 768 > 4096 ? span * base / 768 : 4096;
  }
  chunk = (chunk + 255) / 256 * 256;
  p.chunk = chunk < 256 ? 256 : chunk;
  p.nsplit = (int)((span + p.chunk - 1) / p.chunk);
  return p;
}

}  // namespace

size_t kv_attention_workspace(const gptq_kv_cache& cache, const gptq_kv_batch& batch, bool bf16,
                              const gptq_attention& a) {
  const Plan p = make_plan(cache, batch, bf16, a);
  if (p.nsplit <= 1) return 0;
  // at most 768 workgroups' splits of 256 rows, times 2^30 tokens: below 2^60
  return (size_t)batch.total * a.q_heads * p.nsplit * (cache.dim + 1) * sizeof(float);
}

bool kv_attention_fits(const gptq_kv_cache& c, const gptq_kv_batch& b, bool bf16, const gptq_attention& a) {
  const int64_t limit = ((int64_t)1 << 32) - 1;
  const Plan p = make_plan(c, b, bf16, a);
  // a workgroup a row and head where splits are joined
  if (p.nsplit > 1 && b.batch * b.max_new > limit / 256 / a.q_heads) return false;
  return p.base <= limit / (p.tile_rows == 256 ? 512 : 256) / p.nsplit;
}

hipError_t kv_attention(const KvAttention& a, hipStream_t stream) {
  const Plan p = make_plan(a.cache, a.batch, a.bf16, a.a);
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
