// The 8-bit product: the launch of the kernel that int8_plan.h chooses.
#include "int8.h"

namespace gptq {

bool int8_gemm_fits(int64_t rows, int64_t cols, int64_t tokens) {
  // at most 512 threads a workgroup
  return int8_by_rows(rows, tokens) ||
         int8_tiles_of(int8_best(rows, cols, tokens), rows, tokens) <= ((int64_t)1 << 23) - 8;
}

hipError_t int8_gemm(const Int8Gemm& a, hipStream_t stream) {
  if (int8_by_rows(a.rows, a.x.tokens)) return int8_rows_launch(a, stream);
  return int8_tile_launch(a, int8_best(a.rows, a.x.cols, a.x.tokens).form, stream);
}

}  // namespace gptq
