// What the attention kernels over the paged 8-bit cache share.
#pragma once

#include "attn.h"

namespace gptq {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// A block's value scale v, of size 2^lv, goes into the exponent of its weights: with s the scores (log2) a weight
// enters the second product, in fp16, as p = v 2^(P + s - ref), where ref goes with the largest s + lv that the row
// has seen.  So fp16's range holds what the row's output is made of, whatever the scales of blocks that the row does
// not see, or sees with no weight to speak of.
constexpr float KV_LV_MIN = -100.0f, KV_LV_MAX = 122.0f;  // what an append writes

// lv; 0 for a scale that is not finite (p is then not finite, l is the scores' as always); the end for a scale of 0
// or any outside the two.
__device__ __forceinline__ float value_exponent(float scale) {
  const int e = (int)(__float_as_uint(scale) >> 23 & 0xff) - 127;
  return e == 128 ? 0.0f : fminf(fmaxf((float)e, KV_LV_MIN), KV_LV_MAX);
}

// Tokens of the cache that rows [r0, r0 + rows) of a sequence see, the first
// rounded down to a multiple of 64.  A row is a query token and head of one key
// head's group: row r is token r / group, head r % group.
struct Span {
  int64_t begin, end;
};
__device__ __forceinline__ Span row_span(const KvAttention& A, const Seq& s, int r0, int rows, int group) {
  const int i0 = r0 / group, last = (r0 + rows < s.n * group ? r0 + rows : s.n * group) - 1;
  const int64_t p0 = (int64_t)s.len - s.n + i0, p1 = (int64_t)s.len - s.n + last / group;
  Span v;
  v.end = A.a.causal && p1 + 1 < s.len ? p1 + 1 : s.len;
  v.begin = A.a.window > 0 && p0 - A.a.window + 1 > 0 ? p0 - A.a.window + 1 : 0;
  v.begin &= ~(int64_t)63;
  if (v.end < v.begin) v.end = v.begin;
  return v;
}

// The tokens [lo, hi) that one row sees.
struct Sees {
  int lo, hi;
};
__device__ __forceinline__ Sees row_sees(const KvAttention& A, const Seq& s, int r, int group) {
  if (r >= s.n * group) return {0, 0};
  const int64_t p = (int64_t)s.len - s.n + r / group;
  int64_t hi = A.a.causal && p + 1 < s.len ? p + 1 : s.len;
  int64_t lo = A.a.window > 0 && p - A.a.window + 1 > 0 ? p - A.a.window + 1 : 0;
  if (hi < lo) hi = lo;
  return {(int)lo, (int)hi};
}

// 8 codes (two dwords) as fp16, exact: code + 128 = u becomes the low byte of the
// fp16 number 1024 + u, and 1152 is taken off.
__device__ __forceinline__ f16x8 codes_to_f16(uint32_t x, uint32_t y) {
  union {
    uint32_t u[4];
    f16x2 h[4];
    f16x8 v;
  } r;
  x ^= 0x80808080u;
  y ^= 0x80808080u;
  r.u[0] = __builtin_amdgcn_perm(0x64646464u, x, 0x04010400u);
  r.u[1] = __builtin_amdgcn_perm(0x64646464u, x, 0x04030402u);
  r.u[2] = __builtin_amdgcn_perm(0x64646464u, y, 0x04010400u);
  r.u[3] = __builtin_amdgcn_perm(0x64646464u, y, 0x04030402u);
  const f16x2 off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) r.h[i] += off;
  return r.v;
}

// x = hi + lo to about 22 bits.
__device__ __forceinline__ void split16(const float (&x)[8], f16x8& hi, f16x8& lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi[i] = (_Float16)x[i];
    lo[i] = (_Float16)(x[i] - (float)hi[i]);
  }
}

// The power of two that brings a row whose largest magnitude is `most` into
// [2^7, 2^8), and its inverse.
__device__ __forceinline__ void row_scale(float most, float& up, float& down) {
  int e = (int)(__float_as_uint(most) >> 23) - 127 - 7;
  if (e < -120) e = -120;
  if (e > 120) e = 120;
  up = __uint_as_float((uint32_t)(127 - e) << 23);
  down = __uint_as_float((uint32_t)(127 + e) << 23);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }


// Partial results of split sequences: per row and head, `nsplit` rows of dim fp32
// (normalised) and their log2 sums.
struct Partials {
  float* out;   // [total * q_heads][nsplit][dim]
  float* lse2;  // [total * q_heads][nsplit]
  int nsplit;   // allotted; a row tile uses the first ceil(span / chunk)
  int64_t chunk;
};

// k_kv_rows.hip: row tiles of 16, or of 32 for dim 64 and for bf16 of dim 128.
hipError_t kv_rows_launch(const KvAttention& a, const Partials& p, int tile_rows, hipStream_t stream);
// Joins the splits (k_kv_rows.hip).
hipError_t kv_join_launch(const KvAttention& a, const Partials& p, int tile_rows, hipStream_t stream);
// k_kv_prompt.hip: row tiles of 128, or of 256 for dim 128 (always for fp32 of dim 128).
hipError_t kv_prompt_launch(const KvAttention& a, const Partials& p, int tile_rows, hipStream_t stream);

}  // namespace gptq
