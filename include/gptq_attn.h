/*
 * gptq_attn.h -- the attention operators of libgptq.so (AMD Instinct MI355X,
 * gfx950): what a decoder layer computes between its packed projections
 * (gptq_dequant_gemv / gptq_dequant_gemm in gptq.h).
 *
 *   gptq_qk_norm_rope, gptq_qk_norm_rope_backward
 *       RMS norm of each query and key head and the position rotation, one pass
 *   gptq_kv_append, gptq_kv_read
 *       new keys and values into a paged cache of 8-bit codes with one scale
 *       for each block of tokens and head (keys normed and rotated on the way);
 *       tokens of the cache back as bf16 or fp32
 *   gptq_kv_attention
 *       attention of new tokens over that cache
 *
 * The conventions of gptq.h hold: device pointers, caller-owned memory, work
 * queued on `stream`, a gptq_status returned, argument errors before any launch.
 *
 * Index data on the device (positions, lengths, tables) is checked by the
 * kernels: a value out of range is never used as an address.  It raises
 * GPTQ_EINVAL in *d_status (a device int32, may be NULL) with an atomic
 * maximum; the caller clears the word, the library never does.  What the call
 * writes for the token, block or sequence concerned is then unspecified; the
 * others are not affected.
 */
#ifndef GPTQ_ATTN_H
#define GPTQ_ATTN_H

#include "gptq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Position rotation and norm.  For a head x[dim] of the token at position p:
 *   n = x * rsqrt(mean(x^2) + eps) * weight      (weight NULL: n = x)
 *   y[a] = n[a] cos[p][i] - n[b] sin[p][i],  y[b] = n[a] sin[p][i] + n[b] cos[p][i]
 * for i < rot / 2, with (a, b) = (i, i + rot / 2), or (2i, 2i + 1) when
 * `interleaved`; y = n from element rot on.  rot 0: no rotation (cos and sin
 * may be NULL, positions are then not read).  fp32 arithmetic, one rounding to
 * the output's type. */
typedef struct {
  const float* cos; /* [max_pos, rot / 2] */
  const float* sin; /* [max_pos, rot / 2] */
  int64_t max_pos;
  int32_t rot;         /* multiple of 16, 0 <= rot <= dim */
  int32_t interleaved; /* 0 or 1 */
  float eps;           /* finite, >= 0 */
} gptq_rope;

/* Heads of every token: element (token, head, d) of x at
 * x[token * x_token + head * x_head + d], the strides in elements.  The same
 * for y.  heads 0: absent, the pointers may be NULL. */
typedef struct {
  const void* x;
  int64_t x_token, x_head;
  void* y;
  int64_t y_token, y_head;
  const void* weight; /* [dim], x's type; NULL: no norm */
  int32_t heads;
} gptq_heads;

/* q->y and k->y as above for `tokens` tokens; positions int32 [tokens], each in
 * [0, max_pos) (max_pos 0 with tokens to rotate: GPTQ_EINVAL).  x, y and weight
 * are all of type dtype (bf16 or fp32).  y may be x with the same strides;
 * otherwise they must not overlap.  dim: a multiple of 16, at most 512.  Vectors
 * of 16 bytes are used where pointers and strides allow, single elements
 * otherwise.  tokens == 0 or no heads: no work. */
int gptq_qk_norm_rope(const gptq_heads* q, const gptq_heads* k, gptq_dtype dtype, int64_t tokens, int32_t dim,
                      const int32_t* positions, const gptq_rope* rope, int32_t* d_status, gptq_stream_t stream);

/* Gradients: dx of type dtype from dy and the forward's x, and, where weight is
 * given, dweight (fp32 [dim], written) summed over tokens and heads in a fixed
 * order (bit-reproducible); heads 0: dweight := 0, the other pointers may be NULL.
 * weight NULL: dx is dy rotated back and x, dweight are not used (may be NULL).
 * dx may be dy with the same strides. */
typedef struct {
  const void* dy;
  int64_t dy_token, dy_head;
  const void* x;
  int64_t x_token, x_head;
  void* dx;
  int64_t dx_token, dx_head;
  const void* weight;
  float* dweight; /* may be NULL */
  int32_t heads;
} gptq_heads_grad;

/* Device bytes for gptq_qk_norm_rope_backward with weights (without any, it takes none). */
size_t gptq_qk_norm_rope_backward_workspace_bytes(int64_t tokens, int32_t dim, int32_t q_heads, int32_t k_heads);

/* tokens == 0: dweight := 0, nothing else.  workspace 4-byte aligned. */
int gptq_qk_norm_rope_backward(const gptq_heads_grad* q, const gptq_heads_grad* k, gptq_dtype dtype, int64_t tokens,
                               int32_t dim, const int32_t* positions, const gptq_rope* rope, void* workspace,
                               size_t workspace_bytes, int32_t* d_status, gptq_stream_t stream);

/* ---------------------------------------------------------------------------
 * The paged cache.  A page holds one block of `block` consecutive tokens of one
 * sequence, for every key head, in 8-bit codes with one scale for the block and
 * head: key element = k_scales[page][head] * code, likewise for values.
 *   k_codes int8 [pages][kv_heads][block][dim]
 *   v_codes int8 [pages][kv_heads][block / 16][dim][16]   (16 tokens of one d
 *           side by side: the order in which the matrix cores take them)
 *   k_scales, v_scales fp32 [pages][kv_heads]
 * block 16, 32, 64 or 128; dim 64, 128 or 256 (else GPTQ_EUNSUPPORTED).
 * Code pointers 16-byte aligned.  Nothing has to be cleared before first use.
 * Scales are not negative and at most 2^122; gptq_kv_append writes powers of two
 * from 2^-100 on, or NaN. */
typedef struct {
  int8_t* k_codes;
  int8_t* v_codes;
  float* k_scales;
  float* v_scales;
  int64_t pages;
  int32_t kv_heads, block, dim;
} gptq_kv_cache;

/* Sequences and their new tokens.  Sequence b has kv_len[b] tokens, the last
 * n_b = q_start[b + 1] - q_start[b] of which are this call's: rows q_start[b]
 * and on of its token tensors (rows that no sequence has are not touched).
 * Token t of the sequence lies in page block_table[b * table_stride + t / block]
 * at place t % block. */
typedef struct {
  const int32_t* q_start;     /* [batch + 1], ascending, within [0, total] */
  const int32_t* kv_len;      /* [batch], each in [0, max_kv] */
  const int32_t* block_table; /* [batch, table_stride]; entries past kv_len are not read */
  int64_t table_stride;       /* >= ceil(max_kv / block) */
  int64_t batch;
  int64_t total;   /* rows of the token tensors */
  int64_t max_new; /* no n_b is larger */
  int64_t max_kv;  /* no kv_len[b] is larger */
} gptq_kv_batch;

/* Stores the new tokens' keys and values (type dtype, [total, kv_heads, dim]
 * with strides as in gptq_heads).  Keys go through the norm (k_weight, NULL:
 * none) and the rotation (rope, NULL: none) at their places in the sequence;
 * values are stored as they are.
 *
 * Scales are powers of two.  For each block that gains tokens, and for keys and
 * values apart: needed = 2^e with the least e >= -100 such that no new element
 * of the block and head exceeds 127 * 2^e in size.  If the block's first token
 * is new, scale := needed and earlier contents are dropped.  Otherwise scale :=
 * max(its scale, needed); where that is larger, the codes of the tokens it
 * already holds are divided by the (power of two) ratio and rounded to nearest,
 * ties to even, so that no number of appends puts an element further than one
 * step of the final scale from its value.  New codes are element / scale,
 * rounded likewise.  A new element that is not finite makes the block's scale
 * NaN (until the block is started afresh): what attends to the block is NaN.
 *
 * Pages that gain tokens must belong to one sequence each.  kv_len[b] >= n_b.
 * No workspace.  total == 0 or batch == 0: no work. */
int gptq_kv_append(const gptq_kv_cache* cache, const gptq_kv_batch* batch, const void* k, int64_t k_token,
                   int64_t k_head, const void* v, int64_t v_token, int64_t v_head, gptq_dtype dtype,
                   const void* k_weight, const gptq_rope* rope, int32_t* d_status, gptq_stream_t stream);

/* The last n_b tokens of each sequence out of the cache: k, v [total, kv_heads,
 * dim] with strides as above, type dtype (bf16 holds them exactly when the
 * scale is a power of two).  k or v may be NULL. */
int gptq_kv_read(const gptq_kv_cache* cache, const gptq_kv_batch* batch, void* k, int64_t k_token, int64_t k_head,
                 void* v, int64_t v_token, int64_t v_head, gptq_dtype dtype, int32_t* d_status,
                 gptq_stream_t stream);

/* ---------------------------------------------------------------------------
 * Attention of each sequence's new tokens over its cache.  With p = kv_len - n_b
 * + i the place of new token i, it sees the tokens j < kv_len, of these only
 * j <= p when `causal`, and only j > p - window when window > 0.  Query head h
 * goes with key head h / (q_heads / kv_heads).
 *   s_j = sm_scale * q . k_j,  out = sum_j exp(s_j) v_j / sum_j exp(s_j),
 *   lse = log sum_j exp(s_j)
 * A query that sees nothing gets out = 0 and lse = -inf.
 *   q, out  [total, q_heads, dim], type dtype, strides as in gptq_heads
 *   lse     fp32 [total, q_heads], contiguous; NULL: not written
 * Products run on the matrix cores with fp32 accumulation.  Codes are exact in
 * fp16.  A bf16 query, scaled by a power of two of its row, is exact in fp16 as
 * far as 2^-22 of the row's largest element; weights times their block's value
 * scale are rounded to fp16 (2^-11) before the second product.  For fp32, query
 * and weights go in two fp16 parts each (about 2^-22).  fp16's range is set, row by
 * row, by the largest product of weight and value scale that the row sees: products
 * are held to 2^-31 of that, whatever is in blocks that the row does not see.
 * Maximum, sum and output are kept in fp32; lse does not depend on values.  Results
 * are bit-reproducible run to run.
 * workspace: gptq_kv_attention_workspace_bytes(...) bytes, 16-byte aligned: the
 * partial results of calls that split long sequences.  out must not overlap q,
 * the cache or the workspace.  q_heads: a multiple of kv_heads. */
typedef struct {
  int32_t q_heads;
  float sm_scale; /* finite */
  int32_t causal; /* 0 or 1 */
  int64_t window; /* 0: no limit */
} gptq_attention;

size_t gptq_kv_attention_workspace_bytes(const gptq_kv_cache* cache, const gptq_kv_batch* batch, gptq_dtype dtype,
                                         const gptq_attention* a);

int gptq_kv_attention(const gptq_kv_cache* cache, const gptq_kv_batch* batch, const gptq_attention* a, const void* q,
                      int64_t q_token, int64_t q_head, void* out, int64_t out_token, int64_t out_head, float* lse,
                      gptq_dtype dtype, void* workspace, size_t workspace_bytes, int32_t* d_status,
                      gptq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_ATTN_H */
