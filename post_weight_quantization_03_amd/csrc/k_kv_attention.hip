// Attention of new tokens over the paged 8-bit cache.
//
//   s_j = sm_scale sk_j (q . kc_j),  out = sum_j e^(s_j - m) sv_j vc_j / sum_j e^(s_j - m)
//
// One wave a query token and head: 64 tokens at a time, a lane a token for the
// scores and a lane an element for the output, in fp32, with the running maximum
// and sum of the softmax.
#include "attn.h"

namespace gptq {
namespace {

__device__ __forceinline__ int code_at(const int8_t* p) { return *p; }

template <bool BF16>
__global__ __launch_bounds__(64) void k_kv_attend(KvAttention A, uint32_t max_new) {
  __shared__ float q[256];
  __shared__ float w[64];
  uint32_t id = blockIdx.x;
  const int h = (int)(id % (uint32_t)A.a.q_heads);
  id /= (uint32_t)A.a.q_heads;
  const int i = (int)(id % max_new), b = (int)(id / max_new);
  const Seq s = load_seq(A.batch, b, A.d_status);
  if (i >= s.n) return;
  const int lane = threadIdx.x, dim = A.cache.dim, block = A.cache.block;
  const int hk = h / (A.a.q_heads / A.cache.kv_heads);
  const int64_t row = s.row + i;
  for (int d = lane; d < dim; d += 64) q[d] = load1<BF16>(A.q, row * A.q_token + h * A.q_head + d);
  __syncthreads();
  const int64_t p = (int64_t)s.len - s.n + i;
  int64_t end = A.a.causal && p + 1 < s.len ? p + 1 : s.len;
  int64_t begin = A.a.window > 0 && p - A.a.window + 1 > 0 ? p - A.a.window + 1 : 0;
  float m = -INFINITY, sum = 0.0f, acc[4] = {0, 0, 0, 0};
  const int32_t* table = A.batch.block_table + b * A.batch.table_stride;
  for (int64_t t0 = begin & ~63ll; t0 < end; t0 += 64) {
    const int64_t j = t0 + lane;
    float x = -INFINITY, vs = 0.0f;
    int64_t page = 0;
    if (j < end) {
      page = table[j / block];
      if (page < 0 || page >= A.cache.pages) {
        raise_einval(A.d_status);
        page = 0;
      }
    }
    const int64_t slot = page * A.cache.kv_heads + hk;
    if (j >= begin && j < end) {
      const int8_t* k = A.cache.k_codes + (slot * block + j % block) * dim;
      x = 0.0f;
      for (int d = 0; d < dim; ++d) x = fmaf(q[d], (float)code_at(k + d), x);
      x *= A.cache.k_scales[slot] * A.a.sm_scale;
      vs = A.cache.v_scales[slot];
    }
    float mt = x;
    for (int k = 1; k < 64; k *= 2) mt = fmaxf(mt, __shfl_xor(mt, k));
    const float mn = fmaxf(m, mt);
    const float e = j >= begin && j < end ? expf(x - mn) : 0.0f;
    const float f = m == -INFINITY ? 0.0f : expf(m - mn);
    float es = e;
    for (int k = 1; k < 64; k *= 2) es += __shfl_xor(es, k);
    sum = sum * f + es;
    m = mn;
    w[lane] = j >= begin && j < end ? e * vs : 0.0f;
    __syncthreads();
    for (int c = 0; c < 4; ++c) acc[c] *= f;
    for (int64_t g = t0; g < t0 + 64 && g < end; g += 16) {
      const int64_t pg = __shfl((int)page, (int)(g - t0));
      const int8_t* v = A.cache.v_codes + (pg * A.cache.kv_heads + hk) * block * dim + g % block * dim;
      for (int c = 0; 64 * c + lane < dim; ++c)
        for (int k = 0; k < 16; ++k)
          acc[c] = fmaf(w[g - t0 + k], (float)code_at(v + (64 * c + lane) * 16 + k), acc[c]);
    }
    __syncthreads();
  }
  for (int c = 0; 64 * c + lane < dim; ++c) {
    const float o = sum > 0.0f || sum != sum ? acc[c] / sum : 0.0f;
    const int64_t at = row * A.out_token + h * A.out_head + 64 * c + lane;
    if (BF16)
      static_cast<__bf16*>(A.out)[at] = (__bf16)o;
    else
      static_cast<float*>(A.out)[at] = o;
  }
  if (A.lse && lane == 0) A.lse[row * A.a.q_heads + h] = m + logf(sum);
}

}  // namespace

size_t kv_attention_workspace(const gptq_kv_cache&, const gptq_kv_batch&, bool, const gptq_attention&) { return 0; }

hipError_t kv_attention(const KvAttention& a, hipStream_t stream) {
  const uint32_t grid = (uint32_t)(a.batch.batch * a.batch.max_new * a.a.q_heads);
  if (a.bf16)
    k_kv_attend<true><<<grid, 64, 0, stream>>>(a, (uint32_t)a.batch.max_new);
  else
    k_kv_attend<false><<<grid, 64, 0, stream>>>(a, (uint32_t)a.batch.max_new);
  return hipGetLastError();
}

}  // namespace gptq
