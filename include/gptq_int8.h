/*
 * gptq_int8.h -- the 8-bit integer product of libgptq.so (AMD Instinct MI355X,
 * gfx950): a layer of 8-bit codes with one scale and zero point for each output
 * channel (gptq_quantize_layer with bits 8 and groupsize -1, packed by gptq_pack),
 * applied to tokens that are rounded to 8 bits with one scale each.
 *
 *   gptq_quantize_tokens   tokens to int8 codes, a scale and the codes' sum each
 *   gptq_int8_gemm         those tokens through a layer, products and sums in
 *                          integers, for one token or whole prompts
 *
 * gptq_dequant_gemm (gptq.h) keeps the activations' precision and reads the codes
 * once for every 16 vectors; this product rounds activations and reads them once
 * for up to 256.
 *
 * The conventions of gptq.h hold: device pointers, caller-owned memory, work
 * queued on `stream`, a gptq_status returned, argument errors before any launch.
 */
#ifndef GPTQ_INT8_H
#define GPTQ_INT8_H

#include "gptq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Quantized tokens: x[t][k] ~ scales[t] * codes[t * stride + k].  A token's codes
 * are followed by zeros up to gptq_token_stride(cols), which gptq_quantize_tokens
 * writes and gptq_int8_gemm relies on. */
typedef struct {
  int8_t* codes;  /* [tokens][stride], 16-byte aligned */
  float* scales;  /* [tokens] */
  int32_t* sums;  /* [tokens]: of a token's codes */
  int64_t tokens;
  int64_t cols;   /* 1 <= cols <= 65536 */
  int64_t stride; /* >= gptq_token_stride(cols), a multiple of 16, at most 2^22 */
} gptq_tokens;

/* cols rounded up to a multiple of 128; 0 when cols is out of range. */
int64_t gptq_token_stride(int64_t cols);

/* For each token x of X [tokens, cols] (row stride ldx >= cols elements; bf16 or fp32):
 *   scale = max(m / 127, 2^-120), rounded to fp32, m the largest |x[k]|
 *   code[k] = the integer nearest to the quotient x[k] / scale, taken exactly, ties to even
 *   sum = the codes' sum
 * so codes lie in [-127, 127].  A token with an element that is not finite gets scale NaN
 * and codes 0 (what it is multiplied to is NaN).  X may have any alignment of its
 * elements; 16-byte-aligned X with rows of whole 16 bytes takes the vector path.  X must not
 * overlap the outputs.  tokens == 0: no work. */
int gptq_quantize_tokens(const void* X, gptq_dtype x_dtype, int64_t ldx, const gptq_tokens* out,
                         gptq_stream_t stream);

/* Y[t, r] = x->scales[t] * scales[r] * sum_k (code[r, k] - zeros[r]) x->codes[t, k] for
 * t < x->tokens, r < rows: Y of type y_dtype (bf16 or fp32), row stride ldy >= rows elements.
 *   packed  uint32 [rows, cols / 4]  8-bit codes as written by gptq_pack, dword aligned;
 *           cols = x->cols a multiple of 4
 *   scales  float [rows], zeros uint8 [rows]
 * The sum is exact in 32-bit integers (|sum| < 2^31 for every cols allowed); it is
 * rounded to fp32, multiplied by the token's scale, then the row's, and rounded to
 * y_dtype: the order of the sum does not matter, so results do not depend on how a
 * call is split, and are bit-reproducible.
 * No workspace.  Y must not overlap the inputs.  tokens == 0 or rows == 0: no work. */
int gptq_int8_gemm(const uint32_t* packed, const float* scales, const uint8_t* zeros, int64_t rows,
                   const gptq_tokens* x, void* Y, gptq_dtype y_dtype, int64_t ldy, gptq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_INT8_H */
