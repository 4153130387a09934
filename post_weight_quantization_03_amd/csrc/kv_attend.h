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
// MASKED: the first tokens that stay visible, up to a multiple of 64 (head), and the window follow each other
// without what lies between: the span counts from 0, and count v stands for token v + (v >= head ? gap : 0).
// Blocks are looked up only for tokens below `sinks` and from `lo` on.  The head costs a tile of 64 tokens however few
// are visible in it: a prompt of 8195 tokens with a window of 1024 (18 tiles a workgroup) takes 205 us with 4 first
// tokens and 189 without; one token of each of 16 sequences over a window of 4096, 37 us with the join.
struct Span {
  int64_t begin, end;
  int head, gap, sinks, lo;
  __device__ __forceinline__ int token(int v) const { return v + (v >= head ? gap : 0); }
  __device__ __forceinline__ int looked_up(int v) const {
    const int t = token(v);
    return t < sinks ? t : max(t, lo);
  }
};
template <bool MASKED>
__device__ __forceinline__ Span row_span(const KvAttention& A, const Seq& s, int r0, int rows, int group);
template <>
__device__ __forceinline__ Span row_span<true>(const KvAttention& A, const Seq& s, int r0, int rows, int group) {
  const int i0 = r0 / group, last = (r0 + rows < s.n * group ? r0 + rows : s.n * group) - 1;
  const bool tree = A.mask.tree != nullptr;
  const int before = s.len - s.n, p0 = tree ? before : before + i0, p1 = before + last / group;
  int end = !tree && A.a.causal && p1 + 1 < s.len ? p1 + 1 : s.len;
  if (end < 0) end = 0;
  const int64_t lo = A.a.window > 0 ? p0 - A.a.window + 1 : 0;
  const int sinks = (int)(A.mask.sinks < end ? A.mask.sinks : end), head = (sinks + 63) & ~63;
  Span v{0, end, 0, 0, sinks, (int)(lo > 0 ? lo : 0)};
  if (v.lo > head) {
    v.head = head;
    v.gap = (v.lo & ~63) - head;
    v.end = end - v.gap > head ? end - v.gap : head;
  }
  return v;
}
template <>
__device__ __forceinline__ Span row_span<false>(const KvAttention& A, const Seq& s, int r0, int rows, int group) {
  const int i0 = r0 / group, last = (r0 + rows < s.n * group ? r0 + rows : s.n * group) - 1;
  const int64_t p0 = (int64_t)s.len - s.n + i0, p1 = (int64_t)s.len - s.n + last / group;
  Span v;
  v.end = A.a.causal && p1 + 1 < s.len ? p1 + 1 : s.len;
  v.begin = A.a.window > 0 && p0 - A.a.window + 1 > 0 ? p0 - A.a.window + 1 : 0;
  v.begin &= ~(int64_t)63;
  if (v.end < v.begin) v.end = v.begin;
  v.head = v.gap = v.sinks = v.lo = 0;
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

// MASKED: tokens from lo to hi - 1 and below sinks (and hi) are seen by the row, and of the new tokens, from
// hi = before on, those of its mask.  A word of 64 bits is made of that for a row and tile of which not all is seen
// (the mask's two words are read then); other tiles take the plain path.  With a tree of 64 tokens over 16 sequences of
// 8192 the call takes what the causal one does, 171 us.
struct RowMask {
  int lo, hi, sinks;
  const uint64_t* words;  // null without a tree
};
__device__ __forceinline__ RowMask row_mask(const KvAttention& A, const Seq& s, int r, int group, int32_t* st) {
  if (r >= s.n * group) return {0, 0, 0, nullptr};
  const int i = r / group, before = s.len - s.n;
  const bool tree = A.mask.tree != nullptr;
  int p = before + i;
  if (tree && A.a.window > 0) {
    p = A.mask.positions[s.row + i];
    if (p < before || p >= s.len) {
      raise_einval(st);
      p = before;
    }
  }
  const int hi = tree ? before : A.a.causal && p + 1 < s.len ? p + 1 : s.len;
  const int64_t lo = A.a.window > 0 ? p - A.a.window + 1 : 0;
  return {(int)(lo > 0 ? lo : 0), hi, (int)A.mask.sinks,
          tree ? A.mask.tree + (s.row + i) * A.mask.tree_stride : nullptr};
}
// The lowest n bits, for any n.
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n <= 0 ? 0 : n >= 64 ? ~(uint64_t)0 : ((uint64_t)1 << n) - 1;
}
// Bit j: the row sees token t + j.
__device__ __forceinline__ uint64_t row_word(const RowMask& m, int n, int t) {
  uint64_t v = low_bits(m.hi - t) & (~low_bits(m.lo - t) | low_bits(m.sinks - t));
  const int d = t - m.hi;
  if (m.words && d > -64 && d < n) {
    const int w = d >> 6, sh = d & 63;
    uint64_t x = w >= 0 ? m.words[w] >> sh : 0;
    if (sh > 0 && 64 * (w + 1) < n) x |= m.words[w + 1] << (64 - sh);
    v |= x & low_bits(n - d);
  }
  return v;
}
// Tokens that every row of [r0, last] sees: from lo to hi - 1 and below sinks (and hi).
struct Full {
  int lo, hi, sinks;
  __device__ __forceinline__ bool has(int t) const { return (t >= lo || t + 64 <= sinks) && t + 64 <= hi; }
};
__device__ __forceinline__ Full full_span(const KvAttention& A, const Seq& s, int r0, int last, int group) {
  const int before = s.len - s.n;
  const bool tree = A.mask.tree != nullptr;
  const int p0 = before + r0 / group, p1 = tree ? s.len - 1 : before + last / group;
  const int64_t lo = A.a.window > 0 ? p1 - A.a.window + 1 : 0;
  return {(int)(lo > 0 ? lo : 0), tree ? before : A.a.causal && p0 + 1 < s.len ? p0 + 1 : s.len, (int)A.mask.sinks};
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
