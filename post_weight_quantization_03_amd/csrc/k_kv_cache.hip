// The paged 8-bit cache: appending keys and values, and reading them back.
//
// A block of tokens and a head share one power-of-two scale s = 2^e.  Appending
// to a block that already holds tokens may need a larger scale; the old codes
// are then divided by 2^k and rounded to even.  An element goes through at most
// the roundings 1/2 (s_1 + s_2 + ... + s) with s_i doubling at least, so it stays
// within one step s of its value; with scales amax / 127 the sum has no such
// bound.  Powers of two cost half a bit of step on average, and make the codes'
// values exact in bf16.
//
// Append: one workgroup owns one block (page), one head, keys or values, so
// nothing is atomic: it takes all of the block's new tokens into registers
// (keys through norm and rotation), reduces their largest magnitude as an
// integer maximum of the bits (in which anything not finite exceeds all
// numbers), fixes the scale and writes codes.  Values go through LDS to their
// 16-tokens-of-one-d order and out in 16-byte pieces; a piece that holds old
// tokens is read, merged and written, by the one thread that owns it.
//
// Three prompts of 8608 tokens in all, 32 heads of 128, bf16 with norm and rotation: 211 MB in 61 to 67 us,
// 3.2 to 3.5 TB/s of the 4.9 of a copy; in fp32 353 MB in 85 us, 4.1 TB/s.  What bounds it has not been found:
// fewer VALU instructions (14 to 9 an element) and more or fewer resident waves changed nothing, and of the
// 12672 workgroups of 16 KB, longer-lived ones that take 8 heads in turn are slower (75 us).  One token of
// each of 64 sequences, 8 heads: 7 us, five dependent accesses.  Reading 214 MB of them back as bf16 takes 36 us,
// 6 TB/s.
#include "attn.h"

namespace gptq {
namespace {

constexpr int KV_THREADS = 256;
constexpr int KV_MIN_EXP = -100;  // of a scale

typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));

// The scale that a largest magnitude (fp32 bits) needs: the least 2^e with
// amax <= 127 * 2^e.  127 = 1.984375 * 2^6.
__device__ __forceinline__ float needed_scale(uint32_t m) {
  if (m >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  int e = (int)(m >> 23) - 127 - ((m & 0x7fffffu) <= 0x7e0000u ? 6 : 5);
  if (e < KV_MIN_EXP) e = KV_MIN_EXP;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Four codes from elements and the factor 1 / scale: x * factor + 1.5 * 2^23 is rounded to an integer, ties to
// even, whose two's complement is the number's low byte (|x * factor| <= 127; otherwise the scale is NaN and
// the codes are of no use).
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float factor) {
  const float magic = 12582912.0f;
  const uint32_t x = __float_as_uint(fmaf(a, factor, magic)), y = __float_as_uint(fmaf(b, factor, magic));
  const uint32_t z = __float_as_uint(fmaf(c, factor, magic)), w = __float_as_uint(fmaf(d, factor, magic));
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(w, z, 0x0c0c0400u), __builtin_amdgcn_perm(y, x, 0x0c0c0400u),
                               0x05040100u);
}
__device__ __forceinline__ int byte_of(uint32_t w, int i) { return (int)(w << (24 - 8 * i)) >> 24; }

__device__ __forceinline__ u32x4v rescaled(u32x4v w, float ratio) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = w[i];
    w[i] = codes4((float)byte_of(x, 0), (float)byte_of(x, 1), (float)byte_of(x, 2), (float)byte_of(x, 3), ratio);
  }
  return w;
}

// IT: rounds of tokens a lane group takes (the block's tokens over the groups).
template <bool BF16, bool VEC, int IT>
__global__ __launch_bounds__(KV_THREADS) void k_kv_append(KvAppend A, uint32_t nblk) {
  extern __shared__ __align__(16) int8_t staged[];  // values: [block][dim]
  __shared__ uint32_t wave_max[KV_THREADS / 64];
  uint32_t id = blockIdx.x;
  const bool is_v = id & 1;
  id >>= 1;
  const int h = (int)(id % (uint32_t)A.cache.kv_heads);
  id /= (uint32_t)A.cache.kv_heads;
  const int j = (int)(id % nblk), b = (int)(id / nblk);

  const Seq s = load_seq(A.batch, b, A.d_status);
  if (s.n == 0) return;
  const int block = A.cache.block, dim = A.cache.dim;
  const int before = s.len - s.n;
  if (before < 0) {
    raise_einval(A.d_status);
    return;
  }
  const int blk = before / block + j;
  const int64_t start = (int64_t)blk * block;
  if (start >= s.len) return;
  const int lo = (int)((before > start ? before : start) - start);
  const int hi = (int)((s.len < start + block ? s.len : start + block) - start);
  const int64_t page = A.batch.block_table[b * A.batch.table_stride + blk];  // on its way beside the elements
  const int L = dim / 16;
  const int l = threadIdx.x & (L - 1), group = threadIdx.x / L, groups = KV_THREADS / L;
  const Runs u = is_v ? Runs{16 * l, 16 * l + 8, -1} : head_runs(l, A.rope.rot, A.rope.interleaved);
  const void* src = is_v ? A.v : A.k;
  const int64_t st = is_v ? A.v_token : A.k_token, sh = is_v ? A.v_head : A.k_head;
  // cos and sin come with the elements where registers allow, else when they are needed
  constexpr bool EARLY = IT <= 1;
  const bool turned = u.pair >= 0 && start + hi <= A.rope.max_pos;
  float xa[IT][8], xb[IT][8];
  Turn turn[EARLY ? IT : 1];
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int tok = it * groups + group;
#pragma unroll
    for (int i = 0; i < 8; ++i) xa[it][i] = xb[it][i] = 0.0f;
    if (tok >= lo && tok < hi) {
      const int64_t o = (s.row + (start + tok - before)) * st + h * sh;
      load8<BF16, VEC>(src, o + u.a, xa[it]);
      load8<BF16, VEC>(src, o + u.b, xb[it]);
      if (EARLY && turned) load_turn(A.rope, start + tok, u.pair, turn[it]);
    }
  }
  if (page < 0 || page >= A.cache.pages || (!is_v && A.rope.rot > 0 && start + hi > A.rope.max_pos)) {
    raise_einval(A.d_status);
    return;
  }
  const int64_t slot = page * A.cache.kv_heads + h;
  int8_t* codes = (is_v ? A.cache.v_codes : A.cache.k_codes) + slot * block * dim;
  float* scale_at = (is_v ? A.cache.v_scales : A.cache.k_scales) + slot;
  const float was = lo > 0 ? *scale_at : 0.0f;  // only a block that holds tokens has one
  if (!is_v) {
    if (A.k_weight) {
      float wa[8], wb[8];
      load8<BF16, VEC>(A.k_weight, u.a, wa);
      load8<BF16, VEC>(A.k_weight, u.b, wb);
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        float sq = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fmaf(xa[it][i], xa[it][i], sq);
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fmaf(xb[it][i], xb[it][i], sq);
        const float r = rsqrtf(head_sum(sq, L) / (float)dim + A.rope.eps);
        const int tok = it * groups + group;
        if (tok >= lo && tok < hi) {  // a place without a token keeps its zeros
#pragma unroll
          for (int i = 0; i < 8; ++i) xa[it][i] *= r * wa[i], xb[it][i] *= r * wb[i];
        }
      }
    }
    if (turned) {
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const int tok = it * groups + group;
        if (tok >= lo && tok < hi) {
          if (!EARLY) load_turn(A.rope, start + tok, u.pair, turn[0]);
          turn16(xa[it], xb[it], turn[EARLY ? it : 0], A.rope.interleaved, false);
        }
      }
    }
  }

  uint32_t m = 0;
#pragma unroll
  for (int it = 0; it < IT; ++it)
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // the bits without the sign
      m = max(m, max(__float_as_uint(xa[it][i]) << 1, __float_as_uint(xb[it][i]) << 1));
    }
#pragma unroll
  for (int k = 1; k < 64; k *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, k));
  if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(wave_max[0], wave_max[1]), max(wave_max[2], wave_max[3]));

  const float need = needed_scale(m >> 1);
  const bool carried = lo > 0;
  const float scale = !carried ? need : was != was ? was : need <= was ? was : need;
  const bool grown = carried && scale > was;
  const float ratio = was / scale, inv = 1.0f / scale;
  if (threadIdx.x == 0) *scale_at = scale;

#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int tok = it * groups + group;
    if (tok < lo || tok >= hi) continue;
    const u32x2v a = {codes4(xa[it][0], xa[it][1], xa[it][2], xa[it][3], inv),
                      codes4(xa[it][4], xa[it][5], xa[it][6], xa[it][7], inv)};
    const u32x2v c = {codes4(xb[it][0], xb[it][1], xb[it][2], xb[it][3], inv),
                      codes4(xb[it][4], xb[it][5], xb[it][6], xb[it][7], inv)};
    int8_t* dst = (is_v ? staged : codes) + tok * dim;
    *reinterpret_cast<u32x2v*>(dst + u.a) = a;
    *reinterpret_cast<u32x2v*>(dst + u.b) = c;
  }

  if (!is_v) {
    if (grown)
      for (int i = threadIdx.x; i < lo * dim / 16; i += KV_THREADS) {
        u32x4v* p = reinterpret_cast<u32x4v*>(codes) + i;
        *p = rescaled(*p, ratio);
      }
    return;
  }
  __syncthreads();
  // A thread takes 16 tokens of 4 neighbouring elements: 16 dwords of LDS, transposed byte by byte (4 x 4
  // at a time, 8 v_perm) into the four pieces.
  const int g0 = grown ? 0 : lo / 16, g1 = (hi + 15) / 16, quads = dim / 4;
  for (int i = g0 * quads + threadIdx.x; i < g1 * quads; i += KV_THREADS) {
    const int g = i / quads, d = 4 * (i - g * quads);
    u32x4v* p = reinterpret_cast<u32x4v*>(codes + (g * dim + d) * 16);
    u32x4v w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int tok = 16 * g + 4 * k + j;
        r[j] = tok >= lo && tok < hi ? *reinterpret_cast<const uint32_t*>(staged + tok * dim + d) : 0u;
      }
      const uint32_t a = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u), c = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u);
      const uint32_t e = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u), f = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
      w[0][k] = __builtin_amdgcn_perm(e, a, 0x05040100u);
      w[1][k] = __builtin_amdgcn_perm(e, a, 0x07060302u);
      w[2][k] = __builtin_amdgcn_perm(f, c, 0x05040100u);
      w[3][k] = __builtin_amdgcn_perm(f, c, 0x07060302u);
    }
    if (16 * g < lo) {  // the piece holds old tokens too
      const int old = lo - 16 * g < 16 ? lo - 16 * g : 16;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4v x = p[j];
        if (grown) x = rescaled(x, ratio);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int n = old - 4 * k;
          const uint32_t mask = n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1;
          w[j][k] = (x[k] & mask) | (w[j][k] & ~mask);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = w[j];
  }
}

constexpr int KR_TOKENS = 64;  // tokens a workgroup reads back

// One workgroup: up to 64 tokens (from a multiple of 16 on) of one head, keys or
// values.  A value thread takes 16 tokens of two neighbouring elements.
template <bool BF16, bool VEC>
__global__ __launch_bounds__(KV_THREADS) void k_kv_read(KvRead A, uint32_t ntile) {
  uint32_t id = blockIdx.x;
  const bool is_v = id & 1;
  id >>= 1;
  if (!(is_v ? A.v : A.k)) return;
  const int h = (int)(id % (uint32_t)A.cache.kv_heads);
  id /= (uint32_t)A.cache.kv_heads;
  const int j = (int)(id % ntile), b = (int)(id / ntile);
  const Seq s = load_seq(A.batch, b, A.d_status);
  if (s.n == 0) return;
  const int before = s.len - s.n;
  if (before < 0) {
    raise_einval(A.d_status);
    return;
  }
  const int block = A.cache.block, dim = A.cache.dim;
  const int64_t t0 = (int64_t)(before & ~15) + (int64_t)j * KR_TOKENS;
  const int32_t* table = A.batch.block_table + b * A.batch.table_stride;
  auto slot_of = [&](int64_t tok, int64_t& slot) {
    const int64_t page = table[tok / block];
    if (page < 0 || page >= A.cache.pages) {
      raise_einval(A.d_status);
      return false;
    }
    slot = page * A.cache.kv_heads + h;
    return true;
  };
  if (!is_v) {
    const int L = dim / 16;
    const int l = threadIdx.x & (L - 1);
    for (int i = threadIdx.x / L; i < KR_TOKENS; i += KV_THREADS / L) {
      const int64_t tok = t0 + i;
      int64_t slot;
      if (tok < before || tok >= s.len || !slot_of(tok, slot)) continue;
      const u32x4v w = *reinterpret_cast<const u32x4v*>(A.cache.k_codes + (slot * block + tok % block) * dim + 16 * l);
      const float scale = A.cache.k_scales[slot];
      float a[8], c[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = (float)byte_of(w[e >> 2], e & 3) * scale;
        c[e] = (float)byte_of(w[2 + (e >> 2)], e & 3) * scale;
      }
      const int64_t o = (s.row + tok - before) * A.k_token + h * A.k_head + 16 * l;
      store8<BF16, VEC>(A.k, o, a);
      store8<BF16, VEC>(A.k, o + 8, c);
    }
    return;
  }
  const int pairs = dim / 2;
  for (int i = threadIdx.x; i < KR_TOKENS / 16 * pairs; i += KV_THREADS) {
    const int g = i / pairs, d = 2 * (i - g * pairs);
    const int64_t base = t0 + 16 * g;
    int64_t slot;
    if (base + 16 <= before || base >= s.len || !slot_of(base, slot)) continue;
    const u32x4v* p =
        reinterpret_cast<const u32x4v*>(A.cache.v_codes + slot * block * dim + (base % block * dim + 16 * d));
    const u32x4v w0 = p[0], w1 = p[1];
    const float scale = A.cache.v_scales[slot];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int64_t tok = base + k;
      if (tok < before || tok >= s.len) continue;
      const float x = (float)byte_of(w0[k >> 2], k & 3) * scale, y = (float)byte_of(w1[k >> 2], k & 3) * scale;
      const int64_t o = (s.row + tok - before) * A.v_token + h * A.v_head + d;
      if constexpr (BF16) {
        typedef float f2 __attribute__((ext_vector_type(2)));
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        const b2 r = __builtin_convertvector((f2){x, y}, b2);
        if constexpr (VEC) {
          *reinterpret_cast<b2*>(static_cast<__bf16*>(A.v) + o) = r;
        } else {
          static_cast<__bf16*>(A.v)[o] = r[0];
          static_cast<__bf16*>(A.v)[o + 1] = r[1];
        }
      } else {
        static_cast<float*>(A.v)[o] = x;
        static_cast<float*>(A.v)[o + 1] = y;
      }
    }
  }
}

template <bool BF16, bool VEC>
hipError_t append_launch(const KvAppend& a, hipStream_t stream) {
  const int64_t block = a.cache.block, dim = a.cache.dim;
  // n tokens reach at most (n + block - 2) / block + 1 blocks
  const int64_t nblk = (a.batch.max_new + block - 2) / block + 1;
  const uint32_t grid = (uint32_t)(a.batch.batch * nblk * a.cache.kv_heads * 2);
  const int groups = KV_THREADS / (int)(dim / 16);
  const int it = ((int)block + groups - 1) / groups;
  const size_t lds = (size_t)(block * dim);
#define GPTQ_APPEND(IT) k_kv_append<BF16, VEC, IT><<<grid, KV_THREADS, lds, stream>>>(a, (uint32_t)nblk)
  switch (it) {
    case 1: GPTQ_APPEND(1); break;
    case 2: GPTQ_APPEND(2); break;
    case 4: GPTQ_APPEND(4); break;
    default: GPTQ_APPEND(8); break;
  }
#undef GPTQ_APPEND
  return hipGetLastError();
}

}  // namespace

hipError_t kv_append(const KvAppend& a, hipStream_t stream) {
  if (a.bf16) return a.vec ? append_launch<true, true>(a, stream) : append_launch<true, false>(a, stream);
  return a.vec ? append_launch<false, true>(a, stream) : append_launch<false, false>(a, stream);
}

hipError_t kv_read(const KvRead& a, hipStream_t stream) {
  const int64_t ntile = (a.batch.max_new + 15 + KR_TOKENS - 1) / KR_TOKENS;
  const uint32_t grid = (uint32_t)(a.batch.batch * ntile * a.cache.kv_heads * 2);
  if (a.bf16) {
    if (a.vec)
      k_kv_read<true, true><<<grid, KV_THREADS, 0, stream>>>(a, (uint32_t)ntile);
    else
      k_kv_read<true, false><<<grid, KV_THREADS, 0, stream>>>(a, (uint32_t)ntile);
  } else if (a.vec) {
    k_kv_read<false, true><<<grid, KV_THREADS, 0, stream>>>(a, (uint32_t)ntile);
  } else {
    k_kv_read<false, false><<<grid, KV_THREADS, 0, stream>>>(a, (uint32_t)ntile);
  }
  return hipGetLastError();
}

}  // namespace gptq
