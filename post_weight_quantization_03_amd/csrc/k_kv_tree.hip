// Positions and masks of trees of drafted tokens from their parents (gptq_kv_tree).
//
// A workgroup takes a sequence, a thread a token: it goes up the path twice, for the depth and for
// the bits.  Parents lie before their children, so a path meets the mask's words from the last to the
// first and each is written once.  The parents of up to LOCAL tokens are in LDS, as a step up the
// path waits for the one before.  13 tokens 3.2 us, 16 sequences of 64 5.7: latencies, of lengths, parents and the path
// in turn.  It is made once a step, for all layers.
#include "attn.h"
#include "gptq_mask.h"

namespace gptq {
namespace {

constexpr int LOCAL = 8192;

__global__ __launch_bounds__(256) void k_kv_tree(gptq_kv_batch B, const int32_t* parents, int64_t window,
                                                 int64_t sinks, int32_t* positions, uint64_t* tree, int64_t stride,
                                                 int32_t* d_status) {
  __shared__ int32_t local[LOCAL];
  const Seq s = load_seq(B, (int)blockIdx.x, d_status);
  const int n = s.n, before = s.len - n, words = (int)((B.max_new + 63) / 64);
  if (n == 0) return;
  if (before < 0) {
    if (threadIdx.x == 0) raise_einval(d_status);
    return;
  }
  const int32_t* up = parents + s.row;
  auto checked = [&](int i) {
    const int p = up[i];
    return p < i && p >= -1 ? p : -1;
  };
  for (int i = threadIdx.x; i < n; i += 256) {
    const int p = checked(i);
    if (p != up[i]) raise_einval(d_status);
    if (i < LOCAL) local[i] = p;
  }
  __syncthreads();
  auto parent = [&](int i) { return i < LOCAL ? local[i] : checked(i); };
  for (int i = threadIdx.x; i < n; i += 256) {
    int depth = 0;
    for (int a = parent(i); a >= 0; a = parent(a)) ++depth;
    positions[s.row + i] = before + depth;
    uint64_t* row = tree + (s.row + i) * stride;
    int w = words - 1, steps = 0;
    uint64_t bits = 0;
    for (int a = i; a >= 0; a = parent(a), ++steps) {
      const bool near = window == 0 || steps < window;
      if (!near && before + depth - steps >= sinks && before >= sinks) break;
      for (; w > a >> 6; --w, bits = 0) row[w] = bits;
      if (near || before + depth - steps < sinks) bits |= (uint64_t)1 << (a & 63);
    }
    for (; w >= 0; --w, bits = 0) row[w] = bits;
  }
}

}  // namespace

hipError_t kv_tree(const gptq_kv_batch& b, const int32_t* parents, int64_t window, int64_t sinks, int32_t* positions,
                   uint64_t* tree, int64_t stride, int32_t* d_status, hipStream_t stream) {
  k_kv_tree<<<(uint32_t)b.batch, 256, 0, stream>>>(b, parents, window, sinks, positions, tree, stride, d_status);
  return hipGetLastError();
}

}  // namespace gptq
