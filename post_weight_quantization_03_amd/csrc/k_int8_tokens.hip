// Tokens to int8 codes with one scale each (gptq_quantize_tokens).
//
// A token is held in registers between its two passes, largest element and codes, by
// a wave (up to 512 elements), 256 or 1024 threads, so X is read once.  The largest element is
// taken over the bits without the sign, as integers: infinity and NaN come out above every number.
//
// The code is the nearest integer to x / s, exactly.  x * (1 / s) + 1.5 * 2^23 rounds to a number whose last
// byte is it or its neighbour across a half, and the rest e = x - q s (one fma, exact where |e| is near s / 2:
// a multiple of the smaller of x's and s's last places, and at most s) tells: below s / 2 it is the nearest.  The
// largest |e| of a thread's eight elements is looked at, so only those with one on a half or across it are
// done over: 4 VALU instructions an element beside the packing, which with 11 (every element decided for itself)
// took 19 us for 4096 x 4096 in bf16.  Now 12 to 16 us there (3.1 to 4.2 TB/s; a copy moves 5.1), one token 2.9.
#include "int8.h"

namespace gptq {
namespace {

constexpr float LEAST_SCALE = 7.52316384526264e-37f;  // 2^-120

template <bool BF16>
__device__ __forceinline__ uint32_t element(const void* p, int64_t i) {
  if constexpr (BF16)
    return (uint32_t) static_cast<const uint16_t*>(p)[i] << 16;
  else
    return static_cast<const uint32_t*>(p)[i];
}

constexpr float MAGIC = 12582912.0f;  // 1.5 * 2^23

// Four codes out of the last bytes.
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x00000400u), __builtin_amdgcn_perm(b, a, 0x00000400u),
                               0x05040100u);
}

// Eight codes of x / scale, inv near 1 / scale.
__device__ __forceinline__ uint2 codes_of(const uint32_t (&x)[8], float scale, float inv) {
  float q[8], most = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float v = __uint_as_float(x[j]);
    q[j] = fmaf(v, inv, MAGIC);
    most = fmaxf(most, fabsf(fmaf(-(q[j] - MAGIC), scale, v)));
  }
  if (2.0f * most >= scale) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float e = fmaf(-(q[j] - MAGIC), scale, __uint_as_float(x[j])), twice = 2.0f * fabsf(e);
      const bool odd = (__float_as_uint(q[j]) & 1) != 0;
      if (twice > scale || (twice == scale && odd)) q[j] += __builtin_copysignf(1.0f, e);
    }
  }
  uint32_t u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(q[j]);
  return make_uint2(pack4(u[0], u[1], u[2], u[3]), pack4(u[4], u[5], u[6], u[7]));
}

// NT threads a token, 8 NI elements a thread.
template <bool BF16, bool VEC, int NT, int NI>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_quantize_tokens(QuantTokens A) {
  constexpr int PER = NT < 256 ? 256 / NT : 1;  // tokens a workgroup
  constexpr int NW = NT / 64;
  __shared__ uint32_t most_of[16];
  __shared__ int32_t sum_of[16];
  const int tid = threadIdx.x % NT;
  const int64_t t = (int64_t)blockIdx.x * PER + threadIdx.x / NT;
  if (NT < 256 && t >= A.out.tokens) return;
  const int cols = (int)A.out.cols;
  const int64_t row = t * A.ldx;
  uint32_t x[NI][8], most = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int k = 8 * (tid + NT * i);
    if (VEC && k + 8 <= cols) {
      if constexpr (BF16) {
        const u32x4i u = *reinterpret_cast<const u32x4i*>(static_cast<const uint16_t*>(A.X) + row + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][2 * j] = u[j] << 16, x[i][2 * j + 1] = u[j] & 0xffff0000u;
      } else {
        const u32x4i* p = reinterpret_cast<const u32x4i*>(static_cast<const uint32_t*>(A.X) + row + k);
        const u32x4i u = p[0], v = p[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = u[j], x[i][4 + j] = v[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = k + j < cols ? element<BF16>(A.X, row + k + j) : 0u;
    }
  }
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) most = max(most, x[i][j] & 0x7fffffffu);
#pragma unroll
  for (int m = 1; m < 64; m *= 2) most = max(most, (uint32_t)__shfl_xor((int)most, m));
  if constexpr (NW > 1) {
    if ((tid & 63) == 0) most_of[tid >> 6] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) most = max(most, most_of[w]);
  }
  const bool finite = most < 0x7f800000u;
  const float scale = fmaxf(__uint_as_float(most) / 127.0f, LEAST_SCALE);
  const float inv = finite ? 1.0f / scale : 0.0f;
  const int stride = (cols + (int)INT8_PAD - 1) / (int)INT8_PAD * (int)INT8_PAD;
  int8_t* out = A.out.codes + t * A.out.stride;
  int32_t sum = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int k = 8 * (tid + NT * i);
    const uint2 w = finite ? codes_of(x[i], scale, inv) : make_uint2(0, 0);
    sum = __builtin_amdgcn_sdot4((int)w.x, 0x01010101, sum, false);
    sum = __builtin_amdgcn_sdot4((int)w.y, 0x01010101, sum, false);
    if (k < stride) *reinterpret_cast<uint2*>(out + k) = w;
  }
#pragma unroll
  for (int m = 1; m < 64; m *= 2) sum += __shfl_xor(sum, m);
  if constexpr (NW > 1) {
    if ((tid & 63) == 0) sum_of[tid >> 6] = sum;
    __syncthreads();
  }
  if (tid == 0) {
#pragma unroll
    for (int w = 1; w < NW; ++w) sum += sum_of[w];
    A.out.scales[t] = finite ? scale : __uint_as_float(0x7fc00000u);
    A.out.sums[t] = sum;
  }
}

template <bool BF16, bool VEC>
hipError_t launch(const QuantTokens& a, hipStream_t stream) {
  const int64_t stride = (a.out.cols + INT8_PAD - 1) / INT8_PAD * INT8_PAD;
  const unsigned n = (unsigned)a.out.tokens;
  if (stride <= 512)
    k_quantize_tokens<BF16, VEC, 64, 1><<<(n + 3) / 4, 256, 0, stream>>>(a);
  else if (stride <= 2048)
    k_quantize_tokens<BF16, VEC, 256, 1><<<n, 256, 0, stream>>>(a);
  else if (stride <= 4096)
    k_quantize_tokens<BF16, VEC, 256, 2><<<n, 256, 0, stream>>>(a);
  else if (stride <= 8192)
    k_quantize_tokens<BF16, VEC, 256, 4><<<n, 256, 0, stream>>>(a);
  else if (stride <= 16384)
    k_quantize_tokens<BF16, VEC, 1024, 2><<<n, 1024, 0, stream>>>(a);
  else if (stride <= 32768)
    k_quantize_tokens<BF16, VEC, 1024, 4><<<n, 1024, 0, stream>>>(a);
  else
    k_quantize_tokens<BF16, VEC, 1024, 8><<<n, 1024, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

bool quantize_tokens_fits(int64_t tokens, int64_t stride) {
  return tokens <= (((int64_t)1 << 32) - 1) / (stride <= 8192 ? 256 : 1024);
}

hipError_t quantize_tokens(const QuantTokens& a, hipStream_t stream) {
  if (a.bf16) return a.vec ? launch<true, true>(a, stream) : launch<true, false>(a, stream);
  return a.vec ? launch<false, true>(a, stream) : launch<false, false>(a, stream);
}

}  // namespace gptq
