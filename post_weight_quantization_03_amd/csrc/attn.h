// Internal declarations of the attention operators (gptq_attn.h).
#pragma once

#include "common.h"
#include "gptq_attn.h"

namespace gptq {

// One side (queries or keys) of the norm and rotation, forward or backward.
struct HeadSide {
  const void* x;
  int64_t x_token, x_head;
  void* y;  // forward: y; backward: dx
  int64_t y_token, y_head;
  const void* dy;  // backward only
  int64_t dy_token, dy_head;
  const void* weight;  // null: no norm
  int heads;
};

struct NormRope {
  HeadSide q, k;
  int bf16;
  int vec;  // every pointer and stride allows 16-byte vectors
  int64_t tokens;
  int dim;
  const int32_t* positions;
  gptq_rope rope;
  int32_t* d_status;
};
hipError_t qk_norm_rope(const NormRope& a, hipStream_t stream);
// Partial sums of the weights' gradients: rows of dim floats for q, then for k.
int64_t norm_rope_partials(int64_t tokens, int dim, int heads);
hipError_t qk_norm_rope_backward(const NormRope& a, float* dq_weight, float* dk_weight, float* partials,
                                 hipStream_t stream);

struct KvAppend {
  gptq_kv_cache cache;
  gptq_kv_batch batch;
  const void *k, *v;
  int64_t k_token, k_head, v_token, v_head;
  int bf16, vec;
  const void* k_weight;
  gptq_rope rope;
  int32_t* d_status;
};
hipError_t kv_append(const KvAppend& a, hipStream_t stream);

struct KvRead {
  gptq_kv_cache cache;
  gptq_kv_batch batch;
  void *k, *v;
  int64_t k_token, k_head, v_token, v_head;
  int bf16, vec;
  int32_t* d_status;
};
hipError_t kv_read(const KvRead& a, hipStream_t stream);

struct KvAttention {
  gptq_kv_cache cache;
  gptq_kv_batch batch;
  gptq_attention a;
  const void* q;
  int64_t q_token, q_head;
  void* out;
  int64_t out_token, out_head;
  float* lse;
  int bf16, vec;
  void* workspace;
  int32_t* d_status;
};
size_t kv_attention_workspace(const gptq_kv_cache& cache, const gptq_kv_batch& batch, bool bf16,
                              const gptq_attention& a);
// Whether the call's launches stay below 2^32 threads each.
bool kv_attention_fits(const gptq_kv_cache& cache, const gptq_kv_batch& batch, bool bf16, const gptq_attention& a);
hipError_t kv_attention(const KvAttention& a, hipStream_t stream);

inline bool kv_block_ok(int32_t block) { return block == 16 || block == 32 || block == 64 || block == 128; }
inline bool kv_dim_ok(int32_t dim) { return dim == 64 || dim == 128 || dim == 256; }

#ifdef __HIPCC__
// ---------------------------------------------------------------------------
// Elements of a head.  A lane holds 16 of them as two runs of 8: the rotation's
// two halves of 8 pairs, or, beyond the rotated part, 16 in a row.
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef float f32x8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (BF16)
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else
    return static_cast<const float*>(p)[i];
}

template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (!VEC) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = load1<BF16>(p, i + j);
  } else if constexpr (BF16) {
    const u32x4v u = *reinterpret_cast<const u32x4v*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(u[j] << 16);
      v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  } else {
    const f32x4v a = *reinterpret_cast<const f32x4v*>(static_cast<const float*>(p) + i);
    const f32x4v b = *reinterpret_cast<const f32x4v*>(static_cast<const float*>(p) + i + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
  }
}

template <bool BF16, bool VEC>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (BF16) {
    f32x8v f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = v[j];
    const bf16x8v b = __builtin_convertvector(f, bf16x8v);
    if constexpr (VEC) {
      *reinterpret_cast<bf16x8v*>(static_cast<uint16_t*>(p) + i) = b;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) static_cast<__bf16*>(p)[i + j] = b[j];
    }
  } else if constexpr (VEC) {
    f32x4v a, b;
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = v[j], b[j] = v[4 + j];
    *reinterpret_cast<f32x4v*>(static_cast<float*>(p) + i) = a;
    *reinterpret_cast<f32x4v*>(static_cast<float*>(p) + i + 4) = b;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) static_cast<float*>(p)[i + j] = v[j];
  }
}

// Lanes that share a head: the power of two >= dim / 16 (lanes past dim / 16
// hold nothing).
__host__ __device__ inline int head_lanes(int dim) {
  int l = 1;
  while (16 * l < dim) l *= 2;
  return l;
}

// First element of lane l's two runs, and the rotation's first pair (-1: the
// lane's elements are not rotated).
struct Runs {
  int a, b, pair;
};
__device__ __forceinline__ Runs head_runs(int l, int rot, int interleaved) {
  if (16 * l >= rot) return {16 * l, 16 * l + 8, -1};
  if (interleaved) return {16 * l, 16 * l + 8, 8 * l};
  return {8 * l, rot / 2 + 8 * l, 8 * l};
}

// cos and sin of the lane's 8 pairs; the rotation by their angle (back: by its
// negative).
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ void load_turn(const gptq_rope& r, int64_t p, int pair, Turn& t) {
  const int64_t o = p * (r.rot / 2) + pair;
  load8<false, true>(r.cos, o, t.c);
  load8<false, true>(r.sin, o, t.s);
}
__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
  const float a = x, b = y;
  x = a * c - b * s;
  y = a * s + b * c;
}
__device__ __forceinline__ void turn16(float (&a)[8], float (&b)[8], const Turn& t, int interleaved, bool back) {
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      turn_pair(a[2 * j], a[2 * j + 1], t.c[j], back ? -t.s[j] : t.s[j]);
      turn_pair(b[2 * j], b[2 * j + 1], t.c[4 + j], back ? -t.s[4 + j] : t.s[4 + j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) turn_pair(a[j], b[j], t.c[j], back ? -t.s[j] : t.s[j]);
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
// Sum over the L lanes (a power of two, aligned) that share a head; the same
// value, from the same order, in each.
__device__ __forceinline__ float head_sum(float x, int L) {
  if (L > 1) x += dpp<0xB1>(x);   // lane ^ 1
  if (L > 2) x += dpp<0x4E>(x);   // lane ^ 2
  if (L > 4) x += dpp<0x141>(x);  // the other quad of 8: mirrored, and quads are uniform
  if (L > 8) x += dpp<0x140>(x);  // the other half of 16
  if (L > 16) x += __shfl_xor(x, 16);
  return x;
}
__device__ __forceinline__ void raise_einval(int32_t* st) {
  if (st) atomicMax(st, (int)GPTQ_EINVAL);
}

// A sequence of a batch: rows [row, row + n) are its tokens [len - n, len).
// Lengths out of range are raised and cut to what the grid and tables cover.
struct Seq {
  int64_t row;
  int n, len;
};
__device__ __forceinline__ Seq load_seq(const gptq_kv_batch& B, int b, int32_t* st) {
  const int64_t s0 = B.q_start[b], s1 = B.q_start[b + 1];
  const int64_t len = B.kv_len[b];
  Seq s{s0, 0, 0};
  if (s0 < 0 || s1 < s0 || s1 > B.total || s1 - s0 > B.max_new || len < 0 || len > B.max_kv) {
    raise_einval(st);
    return s;
  }
  s.n = (int)(s1 - s0);
  s.len = (int)len;
  return s;
}
#endif

}  // namespace gptq
