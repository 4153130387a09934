// RMS norm of every query and key head with the position rotation, in one pass,
// and its gradients.
//
//   r = (mean x^2 + eps)^-1/2,  n = x r w,  y = R(p) n
//   dn = R(p)^T dy,  g = dn w,  dx = r (g - x r mean(g x r)),  dw = sum dn x r
//
// Every element is read once and written once (backward: two read, one
// written) and some ten operations are done on it, so HBM bounds both.  A lane
// takes 16 elements of a head, 8 pairs of the rotation: both halves of the
// pairs are 16-byte vectors (bf16) with no exchange between lanes, and a 128-
// wide head is 8 lanes, one DPP butterfly of three steps for its sum of
// squares.  In place is safe: a lane writes just what it has read.
//
// cos and sin (fp32) are as many bytes as a bf16 head, from the caches.  A lane
// group keeps them in registers over HPT heads of one token; HPT is 4 where
// that still leaves the chip several waves a SIMD, 1 below.
//
// 8195 tokens of 32 and 32 heads of 128 in bf16: 273 MB in 56 to 61 us, 4.5 to 4.9 TB/s, the rate of a large
// copy; in fp32 546 MB in 102 us (5.3 TB/s).  Gradients of 4096 tokens, 32 and 8 heads: 128 MB in 30 us (4.2 TB/s)
// and 4 for the weights' sums, in fp32 252 MB in 50.  One token: 3 us.  1531 tokens of 14 and 2 heads of 64 in fp32,
// 19 MB: 10 us and 4, latency: a pass of dependent loads, the groups' sums through LDS, a second launch.
#include "attn.h"

namespace gptq {
namespace {

constexpr int NR_THREADS = 256;
constexpr int NR_MAX_WG = 512;  // workgroups a side of the backward pass (partial sums of dw)

__device__ __forceinline__ float lane_sq(const float (&a)[8], const float (&b)[8]) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) s = fmaf(a[j], a[j], s);
#pragma unroll
  for (int j = 0; j < 8; ++j) s = fmaf(b[j], b[j], s);
  return s;
}

__device__ __forceinline__ int64_t checked_position(const NormRope& A, int64_t t) {
  if (A.rope.rot == 0) return 0;
  const int64_t p = A.positions[t];
  if (p >= 0 && p < A.rope.max_pos) return p;
  raise_einval(A.d_status);
  return 0;
}

// Item = one token and up to HPT heads of one side; items of q come first.
template <bool BF16, bool VEC, int HPT>
__global__ __launch_bounds__(NR_THREADS) void k_norm_rope(NormRope A, int L, uint32_t q_chunks, uint32_t chunks,
                                                          uint32_t items) {
  const int l = threadIdx.x & (L - 1);
  const uint32_t item = (blockIdx.x * NR_THREADS + threadIdx.x) / (uint32_t)L;
  if (item >= items) return;  // whole lane groups leave together
  const int64_t t = item / chunks;
  const uint32_t c = item - (uint32_t)t * chunks;
  const bool is_k = c >= q_chunks;
  const HeadSide S = is_k ? A.k : A.q;
  const int h0 = (int)(is_k ? c - q_chunks : c) * HPT;
  const Runs u = head_runs(l, A.rope.rot, A.rope.interleaved);
  const bool live = 16 * l < A.dim;

  float xa[HPT][8], xb[HPT][8];
#pragma unroll
  for (int i = 0; i < HPT; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) xa[i][j] = xb[i][j] = 0.0f;
    if (live && h0 + i < S.heads) {
      const int64_t o = t * S.x_token + (h0 + i) * S.x_head;
      load8<BF16, VEC>(S.x, o + u.a, xa[i]);
      load8<BF16, VEC>(S.x, o + u.b, xb[i]);
    }
  }
  const int64_t p = checked_position(A, t);
  Turn turn;
  const bool turned = live && u.pair >= 0;
  if (turned) load_turn(A.rope, p, u.pair, turn);
  float wa[8], wb[8];
  if (S.weight && live) {
    load8<BF16, VEC>(S.weight, u.a, wa);
    load8<BF16, VEC>(S.weight, u.b, wb);
  }
#pragma unroll
  for (int i = 0; i < HPT; ++i) {
    if (S.weight) {
      const float r = rsqrtf(head_sum(lane_sq(xa[i], xb[i]), L) / (float)A.dim + A.rope.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) xa[i][j] *= r * wa[j], xb[i][j] *= r * wb[j];
    }
    if (turned) turn16(xa[i], xb[i], turn, A.rope.interleaved, false);
    if (live && h0 + i < S.heads) {
      const int64_t o = t * S.y_token + (h0 + i) * S.y_head;
      store8<BF16, VEC>(S.y, o + u.a, xa[i]);
      store8<BF16, VEC>(S.y, o + u.b, xb[i]);
    }
  }
}

// Items = (token, head) of one side (blockIdx.y), taken in turn by the lane
// groups of a fixed number of workgroups, so that each lane sums dw for its 16
// elements in registers; then the workgroup's groups are added in LDS in a fixed
// order and one partial row goes out.
template <bool BF16, bool VEC>
__global__ __launch_bounds__(NR_THREADS) void k_norm_rope_bwd(NormRope A, int L, int nwg_q, int nwg_k,
                                                              float* partials) {
  __shared__ float red[NR_THREADS / 64][512];
  const HeadSide S = blockIdx.y ? A.k : A.q;
  const int nwg = blockIdx.y ? nwg_k : nwg_q;
  if ((int)blockIdx.x >= nwg) return;
  const int l = threadIdx.x & (L - 1);
  const int groups = NR_THREADS / L;
  const Runs u = head_runs(l, A.rope.rot, A.rope.interleaved);
  const bool live = 16 * l < A.dim;
  const bool turned = live && u.pair >= 0;
  const bool norm = S.weight != nullptr;
  const float inv_dim = 1.0f / (float)A.dim;
  float wa[8], wb[8], da[8], db[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) wa[j] = wb[j] = da[j] = db[j] = 0.0f;
  if (norm && live) {
    load8<BF16, VEC>(S.weight, u.a, wa);
    load8<BF16, VEC>(S.weight, u.b, wb);
  }
  const uint32_t items = (uint32_t)(A.tokens * S.heads);
  const uint32_t stride = (uint32_t)(nwg * groups);
  for (uint32_t item = blockIdx.x * groups + threadIdx.x / L; item < items; item += stride) {
    const int64_t t = item / (uint32_t)S.heads;
    const int64_t h = item - (uint32_t)t * (uint32_t)S.heads;
    float ga[8], gb[8], xa[8], xb[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) ga[j] = gb[j] = xa[j] = xb[j] = 0.0f;
    if (live) {
      const int64_t o = t * S.dy_token + h * S.dy_head;
      load8<BF16, VEC>(S.dy, o + u.a, ga);
      load8<BF16, VEC>(S.dy, o + u.b, gb);
      if (norm) {
        const int64_t ox = t * S.x_token + h * S.x_head;
        load8<BF16, VEC>(S.x, ox + u.a, xa);
        load8<BF16, VEC>(S.x, ox + u.b, xb);
      }
    }
    const int64_t p = checked_position(A, t);
    if (turned) {
      Turn turn;
      load_turn(A.rope, p, u.pair, turn);
      turn16(ga, gb, turn, A.rope.interleaved, true);
    }
    if (norm) {
      const float r = rsqrtf(head_sum(lane_sq(xa, xb), L) / (float)A.dim + A.rope.eps);
      float gx = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xa[j] *= r, xb[j] *= r;  // of size 1 from here on: r^3 leaves fp32's range long before dx does
        da[j] = fmaf(ga[j], xa[j], da[j]);
        db[j] = fmaf(gb[j], xb[j], db[j]);
        ga[j] *= wa[j];
        gb[j] *= wb[j];
        gx = fmaf(ga[j], xa[j], fmaf(gb[j], xb[j], gx));
      }
      const float c = head_sum(gx, L) * inv_dim;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ga[j] = r * fmaf(-xa[j], c, ga[j]);
        gb[j] = r * fmaf(-xb[j], c, gb[j]);
      }
    }
    if (live) {
      const int64_t o = t * S.y_token + h * S.y_head;
      store8<BF16, VEC>(S.y, o + u.a, ga);
      store8<BF16, VEC>(S.y, o + u.b, gb);
    }
  }
  if (!norm) return;
  // the wave's lane groups, then the waves
#pragma unroll
  for (int j = 0; j < 8; ++j)
    for (int m = L; m < 64; m *= 2) da[j] += __shfl_xor(da[j], m), db[j] += __shfl_xor(db[j], m);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (lane < L && live) {
#pragma unroll
    for (int j = 0; j < 8; ++j) red[wave][u.a + j] = da[j], red[wave][u.b + j] = db[j];
  }
  __syncthreads();
  float* out = partials + ((int64_t)(blockIdx.y ? nwg_q : 0) + blockIdx.x) * A.dim;
  for (int d = threadIdx.x; d < A.dim; d += NR_THREADS) out[d] = (red[0][d] + red[1][d]) + (red[2][d] + red[3][d]);
}

// dw = sum of the partial rows of one side (blockIdx.y), 16 columns a workgroup,
// rows taken in turn by 16 threads a column.
__global__ __launch_bounds__(256) void k_weight_grad(const float* partials, int dim, int nwg_q, int nwg_k,
                                                     float* dq_weight, float* dk_weight) {
  __shared__ float red[16][17];
  float* dst = blockIdx.y ? dk_weight : dq_weight;
  if (!dst) return;
  const int rows = blockIdx.y ? nwg_k : nwg_q;
  const float* src = partials + (blockIdx.y ? (int64_t)nwg_q * dim : 0);
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
  float s = 0.0f;
#pragma unroll 8
  for (int r = g; r < rows; r += 16) s += src[(int64_t)r * dim + 16 * blockIdx.x + c];
  red[g][c] = s;
  __syncthreads();
  if (g == 0) {
    s = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) s += red[r][c];
    dst[16 * blockIdx.x + c] = s;
  }
}

template <bool BF16, bool VEC>
hipError_t launch_forward(const NormRope& a, hipStream_t stream) {
  const int L = head_lanes(a.dim);
  const int64_t heads = (int64_t)a.tokens * (a.q.heads + a.k.heads);
  auto chunks = [](int h, int per) { return (uint32_t)((h + per - 1) / per); };
  auto grid = [&](uint32_t per_token) {
    return (uint32_t)((a.tokens * per_token * L + NR_THREADS - 1) / NR_THREADS);
  };
  // 4 heads a lane group from 16 waves a CU on (256 CUs); fewer heads spread over more waves below
  if (heads * L >= (int64_t)4 * 64 * 16 * 256) {
    const uint32_t qc = chunks(a.q.heads, 4), n = qc + chunks(a.k.heads, 4);
    k_norm_rope<BF16, VEC, 4><<<grid(n), NR_THREADS, 0, stream>>>(a, L, qc, n, (uint32_t)(a.tokens * n));
  } else {
    const uint32_t qc = a.q.heads, n = qc + a.k.heads;
    k_norm_rope<BF16, VEC, 1><<<grid(n), NR_THREADS, 0, stream>>>(a, L, qc, n, (uint32_t)(a.tokens * n));
  }
  return hipGetLastError();
}

int backward_wgs(int64_t tokens, int dim, int heads) {
  const int64_t need = (tokens * heads * head_lanes(dim) + NR_THREADS - 1) / NR_THREADS;
  return (int)(need < NR_MAX_WG ? need : NR_MAX_WG);
}

template <bool BF16, bool VEC>
hipError_t launch_backward(const NormRope& a, float* dqw, float* dkw, float* partials, hipStream_t stream) {
  const int L = head_lanes(a.dim);
  const int nq = backward_wgs(a.tokens, a.dim, a.q.heads), nk = backward_wgs(a.tokens, a.dim, a.k.heads);
  if (a.tokens > 0 && nq + nk > 0)
    k_norm_rope_bwd<BF16, VEC><<<dim3(nq > nk ? nq : nk, 2), NR_THREADS, 0, stream>>>(a, L, nq, nk, partials);
  if (dqw || dkw) k_weight_grad<<<dim3(a.dim / 16, 2), 256, 0, stream>>>(partials, a.dim, nq, nk, dqw, dkw);
  return hipGetLastError();
}

}  // namespace

hipError_t qk_norm_rope(const NormRope& a, hipStream_t stream) {
  if (a.bf16) return a.vec ? launch_forward<true, true>(a, stream) : launch_forward<true, false>(a, stream);
  return a.vec ? launch_forward<false, true>(a, stream) : launch_forward<false, false>(a, stream);
}

int64_t norm_rope_partials(int64_t tokens, int dim, int heads) { return backward_wgs(tokens, dim, heads); }

hipError_t qk_norm_rope_backward(const NormRope& a, float* dqw, float* dkw, float* partials, hipStream_t stream) {
  if (a.bf16)
    return a.vec ? launch_backward<true, true>(a, dqw, dkw, partials, stream)
                 : launch_backward<true, false>(a, dqw, dkw, partials, stream);
  return a.vec ? launch_backward<false, true>(a, dqw, dkw, partials, stream)
               : launch_backward<false, false>(a, dqw, dkw, partials, stream);
}

}  // namespace gptq
