// Internal declarations of the 8-bit integer product (gptq_int8.h).
#pragma once

#include "common.h"
#include "gptq_int8.h"
#include "int8_plan.h"

namespace gptq {

constexpr int64_t INT8_MAX_COLS = 65536;  // 255 * 127 * 65536 < 2^31
constexpr int64_t INT8_MAX_STRIDE = (int64_t)1 << 22;  // 256 tokens lie within 2^30 bytes
constexpr int64_t INT8_PAD = 128;         // codes of a token are padded with zeros to a multiple of this

struct QuantTokens {
  const void* X;
  int64_t ldx;
  gptq_tokens out;
  int bf16, vec;
};
// Whether the launch stays below 2^32 threads.
bool quantize_tokens_fits(int64_t tokens, int64_t stride);
hipError_t quantize_tokens(const QuantTokens& a, hipStream_t stream);

struct Int8Gemm {
  const uint32_t* packed;
  const float* scales;
  const uint8_t* zeros;
  int64_t rows;
  gptq_tokens x;
  void* Y;
  int64_t ldy;
  int bf16;
};
// Whether the launch stays below 2^32 threads.
bool int8_gemm_fits(int64_t rows, int64_t cols, int64_t tokens);
hipError_t int8_gemm(const Int8Gemm& a, hipStream_t stream);
// k_int8_rows.hip: up to 16 tokens.  k_int8_tile.hip: tiles of rows x tokens.
hipError_t int8_rows_launch(const Int8Gemm& a, hipStream_t stream);
hipError_t int8_tile_launch(const Int8Gemm& a, Int8Form form, hipStream_t stream);

#ifdef __HIPCC__
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4i __attribute__((ext_vector_type(4)));

// Buffer over `bytes` bytes from p on: loads past them give 0, dword by dword.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}
constexpr uint32_t NOWHERE = 0x7ffffff0u;  // an offset past every buffer here

// Codes of a layer, 0 to 255, as int8: code - 128.
__device__ __forceinline__ i32x4 signed_codes(i32x4 w) { return w ^ (int32_t)0x80808080; }

// Sum of (code - 128) * x to a value: what the zero point adds (rest = 128 - zero point, and a token's sum is
// below 2^23), then the scales.
__device__ __forceinline__ float int8_value(int32_t sum, int32_t rest, int32_t token_sum, float token_scale,
                                            float scale) {
  return (float)(sum + __mul24(rest, token_sum)) * token_scale * scale;
}
__device__ __forceinline__ void int8_store(void* Y, int64_t at, float y, bool bf16) {
  if (bf16)
    static_cast<__bf16*>(Y)[at] = (__bf16)y;
  else
    static_cast<float*>(Y)[at] = y;
}
#endif

}  // namespace gptq
