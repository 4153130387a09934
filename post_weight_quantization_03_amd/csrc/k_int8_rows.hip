// The 8-bit product of few tokens: 16 rows of the layer a workgroup, straight from HBM.
//
// v_mfma_i32_16x16x64_i8 takes 16 rows and 16 tokens, lane l the codes 16 (l / 16) .. + 15
// of row l % 16 and of token l % 16, so both operands are 16-byte loads as they lie in
// memory.  The waves of a workgroup go through the columns 128 at a time in turn; their sums
// are added in LDS at the end (integers: in any order).
#include "int8.h"

namespace gptq {
namespace {

constexpr int NW = 8;  // waves
constexpr int U = 4;   // column chunks a wave has on their way

template <int CT>
__global__ __launch_bounds__(64 * NW) void k_int8_rows(Int8Gemm A, uint32_t row_blocks) {
  __shared__ int32_t part[NW][16 * CT][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n16 = lane & 15, g = lane >> 4;
  const int64_t r0 = (int64_t)(blockIdx.x % row_blocks) * 16;
  const int64_t t0 = (int64_t)(blockIdx.x / row_blocks) * (16 * CT);
  const int64_t rows = A.rows - r0 < 16 ? A.rows - r0 : 16;
  const int64_t tokens = A.x.tokens - t0 < 16 * CT ? A.x.tokens - t0 : 16 * CT;
  const int cols = (int)A.x.cols;
  const auto wb = buffer_of(reinterpret_cast<const char*>(A.packed) + r0 * cols, rows * cols);
  const int8_t* xp[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int64_t t = 16 * c + n16 < tokens ? 16 * c + n16 : tokens - 1;
    xp[c] = A.x.codes + (t0 + t) * A.x.stride + 16 * g;
  }
  const uint32_t w_off = (uint32_t)(n16 * cols + 16 * g);
  i32x4 acc[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) acc[c] = (i32x4){0, 0, 0, 0};

  const int chunks = (cols + 127) / 128;
  for (int k0 = wave; k0 < chunks; k0 += NW * U) {
    i32x4 w[U][2], x[U][CT][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + NW * u;
      const bool in = k < chunks;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        w[u][h] = (i32x4)__builtin_amdgcn_raw_buffer_load_b128(wb, in ? w_off + 128 * k + 64 * h : NOWHERE, 0, 0);
#pragma unroll
        for (int c = 0; c < CT; ++c)
          x[u][c][h] = in ? *reinterpret_cast<const i32x4*>(xp[c] + 128 * k + 64 * h) : (i32x4){0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const i32x4 a = signed_codes(w[u][h]);
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, x[u][c][h], acc[c], 0, 0, 0);
      }
  }
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int r = 0; r < 4; ++r) part[wave][16 * c + n16][4 * g + r] = acc[c][r];
  __syncthreads();
  for (int i = threadIdx.x; i < 256 * CT; i += 64 * NW) {
    const int r = i & 15, t = i >> 4;
    if (r >= rows || t >= tokens) continue;
    int32_t sum = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += part[w][t][r];
    const float y = int8_value(sum, A.zeros[r0 + r], A.x.sums[t0 + t], A.x.scales[t0 + t], A.scales[r0 + r]);
    int8_store(A.Y, (t0 + t) * A.ldy + r0 + r, y, A.bf16);
  }
}

}  // namespace

size_t int8_gemm_workspace(int64_t, int64_t, int64_t) { return 0; }

bool int8_gemm_fits(int64_t rows, int64_t, int64_t tokens) {
  return (rows + 15) / 16 <= (((int64_t)1 << 32) - 1) / (64 * NW) / ((tokens + 63) / 64);
}

hipError_t int8_gemm(const Int8Gemm& a, hipStream_t stream) {
  const uint32_t blocks = (uint32_t)((a.rows + 15) / 16);
  const uint32_t grid = blocks * (uint32_t)((a.x.tokens + 63) / 64);
  if (a.x.tokens <= 16)
    k_int8_rows<1><<<grid, 64 * NW, 0, stream>>>(a, blocks);
  else if (a.x.tokens <= 32)
    k_int8_rows<2><<<grid, 64 * NW, 0, stream>>>(a, blocks);
  else
    k_int8_rows<4><<<grid, 64 * NW, 0, stream>>>(a, blocks);
  return hipGetLastError();
}

}  // namespace gptq
