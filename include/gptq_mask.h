/*
 * gptq_mask.h -- attention over the paged 8-bit cache (gptq_attn.h) of tokens that
 * see neither all that came before them nor a plain window of it (libgptq.so, AMD
 * Instinct MI355X, gfx950).
 *
 *   gptq_kv_masked_attention   gptq_kv_attention with a few first tokens that a window
 *                              leaves visible, and with the new tokens as a tree
 *   gptq_kv_tree               positions and masks of a tree of drafted tokens from
 *                              their parents
 *
 * The conventions of gptq_attn.h hold, those for index data on the device and
 * d_status among them.
 */
#ifndef GPTQ_MASK_H
#define GPTQ_MASK_H

#include "gptq_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What a row sees, beside gptq_attention's own limits.  With p the place of new token
 * i, kv_len - n_b + i, it sees the tokens j < kv_len (only j <= p when `causal`) with
 *     window == 0  or  j > p - window  or  j < sinks.
 * With a tree (causal must be 1) its place is not its position: with before = kv_len -
 * n_b and p = positions[row of i], it sees the tokens j < before as above, and of the
 * new tokens those whose bit its mask has set: token before + a where bit a % 64 of
 * word a / 64 is 1, in any pattern (bits from n_b on are not used).
 * sinks has no effect without a window.  Blocks of which no token of a sequence sees
 * anything (between the first tokens and the window) are not read, neither their
 * table entries nor their pages: they may be given away. */
typedef struct {
  int64_t sinks;            /* >= 0 */
  const uint64_t* tree;     /* [total][tree_stride]; NULL: no tree */
  int64_t tree_stride;      /* words, >= ceil(max_new / 64) */
  const int32_t* positions; /* [total], each in [before, before + n_b); read with a tree and a window only */
} gptq_kv_mask;

/* gptq_kv_attention with a mask: the same arguments, types, numbers, workspace rules and
 * results for rows that see nothing. */
size_t gptq_kv_masked_attention_workspace_bytes(const gptq_kv_cache* cache, const gptq_kv_batch* batch,
                                                gptq_dtype dtype, const gptq_attention* a, const gptq_kv_mask* mask);

int gptq_kv_masked_attention(const gptq_kv_cache* cache, const gptq_kv_batch* batch, const gptq_attention* a,
                             const gptq_kv_mask* mask, const void* q, int64_t q_token, int64_t q_head, void* out,
                             int64_t out_token, int64_t out_head, float* lse, gptq_dtype dtype, void* workspace,
                             size_t workspace_bytes, int32_t* d_status, gptq_stream_t stream);

/* The new tokens of each sequence as trees.  parents int32 [total]: of new token i the
 * new token (of its sequence, counted from 0) that it follows, less than i, or -1 where it follows
 * the cache's last token.  Written, for every row that a sequence has:
 *   positions int32 [total]               before + the number of new tokens on the path to it
 *   tree uint64 [total][tree_stride]      words 0 .. ceil(max_new / 64) - 1: the new tokens on
 *        that path and itself, those at positions that `window` and `sinks` leave visible
 * positions are those for gptq_qk_norm_rope and for gptq_kv_mask.  A parent out of range is raised and
 * taken for -1; kv_len < n_b is raised and the sequence's rows are left.  The outputs must not overlap the inputs.
 * The time grows with the longest path (a chain of 8192: 67 us).  The batch's block_table is not used. */
int gptq_kv_tree(const gptq_kv_batch* batch, const int32_t* parents, int64_t window, int64_t sinks,
                 int32_t* positions, uint64_t* tree, int64_t tree_stride, int32_t* d_status, gptq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_MASK_H */
