// The 8-bit product of up to 16 tokens and a few thousand rows: 16 rows a workgroup, straight from memory.
//
// v_mfma_i32_16x16x64_i8 takes 16 rows and 16 tokens, lane l the codes 16 (l / 16) .. + 15
// of row l % 16 and of token l % 16, so both operands are 16-byte loads as they lie in
// memory: no LDS and no barrier in the loop.  The four waves go through the columns 128 at a time in turn,
// each with three chunks on their way; their sums are added in LDS at the end (integers: in any order).
//
// One token (times of calls in a row): 4096 columns x 4096 rows 6.1 us, 11008 x 4096 10.3 (4.4 TB/s), where tiles of
// 32 x 16 take 7.1 and 12.8; 4096 x 11008 12.5, where they take 10.1 (int8_plan.h goes by the rows).  With eight
// waves and four chunks 6.2, 11.2 and 14.1; eight chunks 10.5, 17.3 and 20.4: fewer workgroups are resident.
#include "int8.h"

namespace gptq {
namespace {

constexpr int NW = 4;  // waves
constexpr int U = 3;   // chunks of a wave on their way

__global__ __launch_bounds__(64 * NW, 4) void k_int8_rows(Int8Gemm A) {
  __shared__ int32_t part[NW][16][20];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n16 = lane & 15, g = lane >> 4;
  const int64_t r0 = (int64_t)blockIdx.x * 16;
  const int rows = A.rows - r0 < 16 ? (int)(A.rows - r0) : 16, tokens = (int)A.x.tokens;
  const int cols = (int)A.x.cols;
  // rows and tokens past the end read 0
  const auto wb = buffer_of(reinterpret_cast<const char*>(A.packed) + r0 * cols, (int64_t)rows * cols);
  const auto xb = buffer_of(A.x.codes, tokens * A.x.stride);
  const uint32_t w_off = (uint32_t)(n16 * cols + 16 * g + 128 * wave);
  const uint32_t x_off = (uint32_t)(n16 * (uint32_t)A.x.stride + 16 * g + 128 * wave);
  i32x4 acc = {0, 0, 0, 0};

  const int chunks = ((cols + 127) / 128 - wave + NW - 1) / NW;  // this wave's
  i32x4 w[U][2], x[U][2];
  auto load = [&](int u, int c) __attribute__((always_inline)) {
    const bool in = c < chunks;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t o = (uint32_t)(128 * NW * c + 64 * h);
      w[u][h] = (i32x4)__builtin_amdgcn_raw_buffer_load_b128(wb, in ? w_off + o : NOWHERE, 0, 0);
      x[u][h] = (i32x4)__builtin_amdgcn_raw_buffer_load_b128(xb, in ? x_off + o : NOWHERE, 0, 0);
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(u, u);
  for (int c = 0; c < chunks; c += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(signed_codes(w[u][h]), x[u][h], acc, 0, 0, 0);
      load(u, c + u + U);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  *reinterpret_cast<i32x4*>(&part[wave][n16][4 * g]) = acc;
  __syncthreads();
  const int r = threadIdx.x & 15, t = threadIdx.x >> 4;
  if (r >= rows || t >= tokens) return;
  int32_t sum = 0;
#pragma unroll
  for (int k = 0; k < NW; ++k) sum += part[k][t][r];
  const float y = int8_value(sum, 128 - (int)A.zeros[r0 + r], A.x.sums[t], A.x.scales[t], A.scales[r0 + r]);
  int8_store(A.Y, t * A.ldy + r0 + r, y, A.bf16);
}

}  // namespace

hipError_t int8_rows_launch(const Int8Gemm& a, hipStream_t stream) {
  k_int8_rows<<<(uint32_t)((a.rows + 15) / 16), 64 * NW, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace gptq
