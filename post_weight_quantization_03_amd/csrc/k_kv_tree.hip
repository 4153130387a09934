// Positions and masks of trees of drafted tokens from their parents (gptq_kv_tree).
//
// Parents lie before their children, so a path meets the mask's words from the last to the first and
// each is written once.  The part of a token's path within its 64 tokens is a word, and one lane a token finds
// it in six doublings: a lane takes over the path of the token that it has come to.  The tokens' words, and the ones
// where they leave their 64, are put in LDS for the first LOCAL tokens; then a thread a token goes up the path, a
// word at a time (from LOCAL on a token at a time), twice: for the depth, and for the mask.
//
// 13 tokens 2.4 us, 16 sequences of 64 4.7, chains of 512 / 8192 7 / 67 (a token at a time 139 / 2215; so from LOCAL
// on, a chain of 20000 takes 5.5 ms): latencies, of lengths, parents and the path in turn.  It is made once a step,
// for all layers.
#include "attn.h"
#include "gptq_mask.h"

namespace gptq {
namespace {

constexpr int LOCAL = 8192;  // a multiple of 64, at most 2^15

// Without the lowest n bits that are set.
__device__ __forceinline__ uint64_t without(uint64_t m, int n) {
  for (; n > 0; --n) m &= m - 1;
  return m;
}

__global__ __launch_bounds__(256) void k_kv_tree(gptq_kv_batch B, const int32_t* parents, int64_t window,
                                                 int64_t sinks, int32_t* positions, uint64_t* tree, int64_t stride,
                                                 int32_t* d_status) {
  __shared__ uint64_t path[LOCAL];
  __shared__ int16_t leaves[LOCAL];  // to: a token before the 64, or -1
  const Seq s = load_seq(B, (int)blockIdx.x, d_status);
  const int n = s.n, before = s.len - n, words = (int)((B.max_new + 63) / 64);
  const int first = (int)blockIdx.y * 256, end = n - first < 256 ? n : first + 256;
  if (first >= n) return;
  if (before < 0) {
    if (threadIdx.x == 0) raise_einval(d_status);
    return;
  }
  const int32_t* up = parents + s.row;
  auto checked = [&](int i) {
    const int p = up[i];
    const bool ok = p < i && p >= -1;
    if (!ok) raise_einval(d_status);
    return ok ? p : -1;
  };
  const int lane = threadIdx.x & 63;
  for (int k = (int)threadIdx.x & ~63; k < end && k < LOCAL; k += 256) {
    int at = k + lane < n ? checked(k + lane) : -1;
    uint64_t m = (uint64_t)1 << lane;
    while (__any(at >= k)) {
      const uint64_t more = __shfl(m, at & 63);
      const int next = __shfl(at, at & 63);
      if (at >= k) m |= more, at = next;
    }
    path[k + lane] = m;
    leaves[k + lane] = (int16_t)at;
  }
  __syncthreads();
  const int i = first + (int)threadIdx.x;
  if (i >= end) return;
  auto part = [&](int a) { return a < LOCAL ? path[a] : (uint64_t)1 << (a & 63); };
  auto next = [&](int a) { return a < LOCAL ? (int)leaves[a] : checked(a); };
  int depth = -1;
  for (int a = i; a >= 0; a = next(a)) depth += __popcll(part(a));
  positions[s.row + i] = before + depth;
  uint64_t* row = tree + (s.row + i) * stride;
  int w = words - 1, steps = 0;
  uint64_t bits = 0;
  for (int a = i; a >= 0; a = next(a)) {
    if (window > 0 && steps >= window && before >= sinks) break;
    uint64_t m = part(a);
    const int c = __popcll(m);
    if (window > 0) {
      // the last `near` of these are within the window, the first `seen` below sinks
      const int64_t left = window - steps, low = sinks - (before + depth - steps - c + 1);
      const int near = left <= 0 ? 0 : left < c ? (int)left : c, seen = low <= 0 ? 0 : low < c ? (int)low : c;
      if (near + seen < c) m = without(m, c - near) | (m & ~without(m, seen));
    }
    for (; w > a >> 6; --w, bits = 0) row[w] = bits;
    bits |= m;
    steps += c;
  }
  for (; w >= 0; --w, bits = 0) row[w] = bits;
}

}  // namespace

bool kv_tree_fits(const gptq_kv_batch& b) {
  const int64_t groups = (b.max_new + 255) / 256;
  return groups <= 65535 && b.batch <= (((int64_t)1 << 32) - 1) / 256 / groups;
}

hipError_t kv_tree(const gptq_kv_batch& b, const int32_t* parents, int64_t window, int64_t sinks, int32_t* positions,
                   uint64_t* tree, int64_t stride, int32_t* d_status, hipStream_t stream) {
  const dim3 grid((uint32_t)b.batch, (uint32_t)((b.max_new + 255) / 256));
  k_kv_tree<<<grid, 256, 0, stream>>>(b, parents, window, sinks, positions, tree, stride, d_status);
  return hipGetLastError();
}

}  // namespace gptq
