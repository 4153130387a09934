// C ABI of the 8-bit integer product: argument checks on the host and the launch of
// each entry point.  Every declaration is documented in include/gptq_int8.h.
#include "int8.h"

namespace {

using namespace gptq;

constexpr int64_t MAX_DIM = (int64_t)1 << 30;

bool dtype_ok(gptq_dtype dt) { return dt == GPTQ_BF16 || dt == GPTQ_F32; }
int64_t elem_size(gptq_dtype dt) { return dt == GPTQ_BF16 ? 2 : 4; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int tokens_check(const gptq_tokens* x) {
  if (!x || x->tokens < 0 || x->tokens > MAX_DIM || x->cols < 1) return GPTQ_EINVAL;
  if (x->cols > INT8_MAX_COLS) return GPTQ_EUNSUPPORTED;
  if (x->stride < gptq_token_stride(x->cols) || x->stride % 16 != 0) return GPTQ_EINVAL;
  if (x->stride > INT8_MAX_STRIDE) return GPTQ_EUNSUPPORTED;
  return GPTQ_OK;
}
bool tokens_pointers(const gptq_tokens* x) {
  return x->codes && x->scales && x->sums && aligned(x->codes, 16) && aligned(x->scales, 4) && aligned(x->sums, 4);
}

}  // namespace

extern "C" {

int64_t gptq_token_stride(int64_t cols) {
  if (cols < 1 || cols > INT8_MAX_COLS) return 0;
  return (cols + INT8_PAD - 1) / INT8_PAD * INT8_PAD;
}

int gptq_quantize_tokens(const void* X, gptq_dtype x_dtype, int64_t ldx, const gptq_tokens* out,
                         gptq_stream_t stream) {
  const int st = tokens_check(out);
  if (st != GPTQ_OK) return st;
  if (!dtype_ok(x_dtype) || ldx < out->cols || ldx > ((int64_t)1 << 40)) return GPTQ_EINVAL;
  if (out->tokens == 0) return GPTQ_OK;
  if (!X || !aligned(X, (uintptr_t)elem_size(x_dtype)) || !tokens_pointers(out)) return GPTQ_EINVAL;
  if (!quantize_tokens_fits(out->tokens, gptq_token_stride(out->cols))) return GPTQ_EUNSUPPORTED;
  QuantTokens a{};
  a.X = X;
  a.ldx = ldx;
  a.out = *out;
  a.bf16 = x_dtype == GPTQ_BF16;
  a.vec = aligned(X, 16) && ldx * elem_size(x_dtype) % 16 == 0;
  return quantize_tokens(a, (hipStream_t)stream) == hipSuccess ? GPTQ_OK : GPTQ_EHIP;
}

int gptq_int8_gemm(const uint32_t* packed, const float* scales, const uint8_t* zeros, int64_t rows,
                   const gptq_tokens* x, void* Y, gptq_dtype y_dtype, int64_t ldy, gptq_stream_t stream) {
  const int st = tokens_check(x);
  if (st != GPTQ_OK) return st;
  if (rows < 0 || rows > MAX_DIM || !dtype_ok(y_dtype) || x->cols % 4 != 0 || ldy < rows || ldy > ((int64_t)1 << 40))
    return GPTQ_EINVAL;
  if (x->tokens == 0 || rows == 0) return GPTQ_OK;
  if (!packed || !scales || !zeros || !Y || !aligned(packed, 4) || !aligned(scales, 4) ||
      !aligned(Y, (uintptr_t)elem_size(y_dtype)) || !tokens_pointers(x))
    return GPTQ_EINVAL;
  if (!int8_gemm_fits(rows, x->cols, x->tokens)) return GPTQ_EUNSUPPORTED;
  const Int8Gemm a{packed, scales, zeros, rows, *x, Y, ldy, y_dtype == GPTQ_BF16};
  return int8_gemm(a, (hipStream_t)stream) == hipSuccess ? GPTQ_OK : GPTQ_EHIP;
}

}  // extern "C"
