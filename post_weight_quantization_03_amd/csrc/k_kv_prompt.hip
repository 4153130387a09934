// Attention of many query rows over the paged 8-bit cache: prompts and chunks.
//
// S^T = K Q^T and O^T += V^T P^T on v_mfma_f32_32x32x16_f16.  A wave keeps 32 rows
// (query token and head of one key head's group) as the columns: queries and
// output in registers, keys and values of 64 tokens in LDS, shared by the
// workgroup's waves.  Codes are widened to fp16 once, on their way into LDS (a
// thread loads 16 of them while the tile before is worked on), because widening
// them in every wave would cost as many VALU cycles as the softmax.
//
// Column q of S^T lies in lanes q and q + 32, which hold tokens 8 (r / 4) + 4 half +
// r % 4; the values' 16 tokens are stored in LDS in the order (0-3, 8-11, 4-7,
// 12-15), so that a lane's weights are its operand of the second product where
// they are.  LDS rows are XOR-swizzled in 16-byte pieces; reads and writes are
// 16-byte and conflict-free.
//
// What bounds it: per wave and tile the two products take 1024 cycles (dim 128),
// the softmax about as many VALU cycles (32 exponentials a lane at a quarter of
// the rate are half of it), and the LDS reads of the CU's 8 waves 2048 at 128 bytes
// a cycle against 2048 of a SIMD's two waves of products.  The softmax is therefore
// kept to an fma, an exponential and an addition a score: the key scale times the
// row's constant is one factor, the maximum is taken before it (it is not
// negative), the value scale is added to the exponent (log2 of its ratio to the
// largest so far) and taken back out of the sum once for 16 tokens, and output and
// sum are rescaled only when a row's maximum has grown by more than 2^8.
#include "kv_attend.h"

namespace gptq {
namespace {

constexpr int PT = 64;                // tokens a tile
constexpr float P_EXP = 6.0f;         // weights are 2^P_EXP e^(s - m), m up to 2^P_SLACK behind the maximum
constexpr float P_SLACK = 8.0f;
constexpr float P_LOG_MIN = -200.0f;  // log2 of a value scale, at least
constexpr float P_RATIO_MIN = -60.0f; // log2 of its ratio to the largest, at least: below, fp16 weights are 0

__device__ __forceinline__ float keep_nan_max(float x, float lo) { return x != x ? x : fmaxf(x, lo); }

// the other half's value of the same column
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

template <int DIM, bool BF16, int NW>
__global__ __launch_bounds__(64 * NW, DIM == 256 ? 1 : 2) void k_kv_prompt(KvAttention A, Partials P, uint32_t pairs,
                                                                           uint32_t row_tiles) {
  constexpr int NK = DIM / 16;         // MFMA steps of the first product
  constexpr int ND = DIM / 32;         // d tiles
  constexpr int NT = 64 * NW;          // threads
  constexpr int PIECES = PT * DIM / 16;  // 16-code pieces of K (and of V) a tile
  constexpr int PER = (PIECES + NT - 1) / NT;
  constexpr int KROW = DIM * 2, VROW = PT * 2;  // bytes
  constexpr int KC = KROW / 16;        // 16-byte pieces a K row
  constexpr int KB = PT * KROW, VB = DIM * VROW;
  __shared__ __align__(16) char lds[2 * (KB + VB)];  // [2][KB], [2][VB]
  // of a tile's four groups of 16 tokens: key scale, log2 of the value scale's ratio to the
  // largest so far and the inverse of that ratio; log2 of the largest so far
  struct Scales {
    float ks[4], lr[4], ir[4], lref, pad[3];
  };
  __shared__ __align__(16) Scales sc[2];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 31, half = lane >> 5;
  uint32_t id = blockIdx.x;
  const uint32_t pair = id % pairs;  // workgroups of one sequence and key head: the same XCD where pairs is a multiple of 8
  id /= pairs;
  const int split = (int)(id % (uint32_t)P.nsplit);
  const int rt = (int)(row_tiles - 1 - id / (uint32_t)P.nsplit);  // the longest of a causal call first
  const int hk = (int)(pair % (uint32_t)A.cache.kv_heads), b = (int)(pair / (uint32_t)A.cache.kv_heads);
  const Seq s = load_seq(A.batch, b, A.d_status);
  const int group = A.a.q_heads / A.cache.kv_heads;
  const int rows = s.n * group, r0 = rt * 32 * NW;
  if (r0 >= rows) return;
  const Span span = row_span(A, s, r0, 32 * NW, group);
  const int64_t first = span.begin + split * P.chunk;
  if (split > 0 && first >= span.end) return;
  const bool whole = span.end - span.begin <= P.chunk;
  const int64_t stop = first + P.chunk < span.end ? first + P.chunk : span.end;
  const int32_t* table = A.batch.block_table + b * A.batch.table_stride;
  const int shift = __builtin_ctz((unsigned)A.cache.block);
  const int block = A.cache.block;

  // queries
  const int wr0 = r0 + 32 * wave, r = wr0 + col;
  f16x8 qh[NK], ql[BF16 ? 1 : NK];
  float qs;
  {
    float x[NK][8];
    float most = 0.0f;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[k][j] = 0.0f;
      if (r < rows) {
        const int64_t o = (s.row + r / group) * A.q_token + (hk * group + r % group) * A.q_head + 16 * k + 8 * half;
        if (A.vec)
          load8<BF16, true>(A.q, o, x[k]);
        else
          load8<BF16, false>(A.q, o, x[k]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(x[k][j]));
    }
    most = fmaxf(most, other_half(most));
    float up, down;
    row_scale(most, up, down);
    qs = fabsf(A.a.sm_scale) * 1.44269504088896340736f * down;
    if (A.a.sm_scale < 0.0f) up = -up;  // the factor of a score is not negative
#pragma unroll
    for (int k = 0; k < NK; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[k][j] *= up;
      if constexpr (BF16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) qh[k][j] = (_Float16)x[k][j];
      } else {
        split16(x[k], qh[k], ql[k]);
      }
    }
  }
  const Sees see = row_sees(A, s, r, group);
  // this wave's tokens: some row sees them; every row sees those of full_lo .. full_hi
  int wave_lo = 0, wave_hi = 0, full_lo = 0, full_hi = 0;
  if (wr0 < rows) {
    const int last = (wr0 + 32 < rows ? wr0 + 32 : rows) - 1;
    const Sees a = row_sees(A, s, wr0, group), z = row_sees(A, s, last, group);
    wave_lo = a.lo, wave_hi = z.hi, full_lo = z.lo, full_hi = a.hi;
  }

  f32x16 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = -INFINITY, l = 0.0f, lref = P_LOG_MIN;

  // a thread's pieces of the next tile
  u32x4v kp[PER], vp[PER];
  float next_ks = 0.0f, next_vs = 0.0f, run_ref = P_LOG_MIN;
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int p = threadIdx.x + i * NT;
      if (PIECES % NT == 0 || p < PIECES) {
        const int tok = p / (DIM / 16), c = p % (DIM / 16);
        const int64_t sk = slot_at(A, table, t + (tok & ~15), stop, shift, hk);
        kp[i] = *reinterpret_cast<const u32x4v*>(A.cache.k_codes +
                                                 (sk * block + ((t + tok) & (block - 1))) * DIM + 16 * c);
        const int g = p / DIM, d = p % DIM;
        const int64_t sv = slot_at(A, table, t + 16 * g, stop, shift, hk);
        vp[i] = *reinterpret_cast<const u32x4v*>(A.cache.v_codes + (sv * block + ((t + 16 * g) & (block - 1))) * DIM +
                                                 16 * d);
      }
    }
    if (threadIdx.x < 4) {
      const int64_t sg = slot_at(A, table, t + 16 * threadIdx.x, stop, shift, hk);
      next_ks = A.cache.k_scales[sg];
      next_vs = t + 16 * threadIdx.x < stop ? A.cache.v_scales[sg] : 0.0f;
    }
  };
  auto place = [&](int buf) {
    char* kb = lds + buf * KB;
    char* vb = lds + 2 * KB + buf * VB;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int p = threadIdx.x + i * NT;
      if (PIECES % NT == 0 || p < PIECES) {
        const int tok = p / (DIM / 16), c = p % (DIM / 16);
        char* row = kb + tok * KROW;
        *reinterpret_cast<f16x8*>(row + 16 * ((2 * c) ^ (tok & (KC - 1)))) = codes_to_f16(kp[i][0], kp[i][1]);
        *reinterpret_cast<f16x8*>(row + 16 * ((2 * c + 1) ^ (tok & (KC - 1)))) = codes_to_f16(kp[i][2], kp[i][3]);
        const int g = p / DIM, d = p % DIM;
        row = vb + d * VROW;
        *reinterpret_cast<f16x8*>(row + 16 * ((2 * g) ^ (d & 7))) = codes_to_f16(vp[i][0], vp[i][2]);
        *reinterpret_cast<f16x8*>(row + 16 * ((2 * g + 1) ^ (d & 7))) = codes_to_f16(vp[i][1], vp[i][3]);
      }
    }
    if (threadIdx.x < 4) {
      const float lv = keep_nan_max(__log2f(next_vs), P_LOG_MIN);
      float top = fmaxf(lv, P_LOG_MIN);
      top = fmaxf(top, dpp<0xB1>(top));
      top = fmaxf(top, dpp<0x4E>(top));
      run_ref = fmaxf(run_ref, top);
      const float lr = keep_nan_max(lv - run_ref, P_RATIO_MIN);
      sc[buf].ks[threadIdx.x] = next_ks;
      sc[buf].lr[threadIdx.x] = lr;
      // with a scale of NaN the weights that see it are NaN; the sums of rows that do not are 0
      sc[buf].ir[threadIdx.x] = lr != lr ? 1.0f : exp2_fast(-lr);
      if (threadIdx.x == 0) sc[buf].lref = run_ref;
    }
  };

  if (first < stop) {
    fetch(first);
    place(0);
  }
  __syncthreads();
  int buf = 0;
  for (int64_t t = first; t < stop; t += PT, buf ^= 1) {
    const bool more = t + PT < stop;
    if (more) fetch(t + PT);
    if (t + PT > wave_lo && t < wave_hi) {
      const char* kb = lds + buf * KB;
      const char* vb = lds + 2 * KB + buf * VB;
      f32x16 x[2];
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[tt][i] = 0.0f;
        const int tok = 32 * tt + col;
        const char* row = kb + tok * KROW;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          const f16x8 a = *reinterpret_cast<const f16x8*>(row + 16 * ((2 * k + half) ^ (tok & (KC - 1))));
          x[tt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, qh[k], x[tt], 0, 0, 0);
          if constexpr (!BF16) x[tt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, ql[k], x[tt], 0, 0, 0);
        }
      }
      const Scales S = sc[buf];
      const bool full = t >= full_lo && t + PT <= full_hi;
      if (!full) {
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int j = (int)t + 32 * tt + 8 * (i >> 2) + 4 * half + (i & 3);
            x[tt][i] = j >= see.lo && j < see.hi ? x[tt][i] : -INFINITY;
          }
      }
      float f[4], most = -INFINITY;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f[g] = S.ks[g] * qs;
        float y = x[g >> 1][8 * (g & 1)];
#pragma unroll
        for (int i = 1; i < 8; ++i) y = fmaxf(y, x[g >> 1][8 * (g & 1) + i]);
        // a masked group stays out whatever its factor is (0, infinite or NaN)
        most = fmaxf(most, y == -INFINITY ? y : y * f[g]);
      }
      most = fmaxf(most, other_half(most));
      const float mn = fmaxf(m, most);
      if (__any(mn > m + P_SLACK || (m == -INFINITY && mn != m)) || S.lref != lref) {
        const float base = mn == -INFINITY ? 0.0f : mn;
        const float alpha = exp2_fast(m - base);
        l *= alpha;
        const float turn = alpha * exp2_fast(lref - S.lref);
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d] *= turn;
        m = mn;
        lref = S.lref;
      }
      const float base = m == -INFINITY ? 0.0f : m;
      f16x8 ph[4], pl[BF16 ? 1 : 4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float add = (P_EXP - base) + S.lr[g];
        float p[8], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y = x[g >> 1][8 * (g & 1) + i];
          float e = exp2_fast(fmaf(y, f[g], add));
          if (!full) e = y == -INFINITY ? 0.0f : e;
          p[i] = e;
          sum += e;
        }
        l = fmaf(sum, S.ir[g], l);
        if constexpr (BF16) {
#pragma unroll
          for (int i = 0; i < 8; ++i) ph[g][i] = (_Float16)p[i];
        } else {
          split16(p, ph[g], pl[g]);
        }
      }
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const int dd = 32 * d + col;
        const char* row = vb + dd * VROW;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f16x8 a = *reinterpret_cast<const f16x8*>(row + 16 * ((2 * g + half) ^ (dd & 7)));
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, ph[g], o[d], 0, 0, 0);
          if constexpr (!BF16) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, pl[g], o[d], 0, 0, 0);
        }
      }
    }
    if (more) place(buf ^ 1);
    __syncthreads();
  }

  l += other_half(l);
  if (r >= rows) return;
  const float inv = l == 0.0f ? 0.0f : exp2_fast(lref) / l;
  const float lse2 = l == 0.0f ? -INFINITY : m + __log2f(l) - P_EXP;
  const int64_t token = s.row + r / group;
  const int head = hk * group + r % group;
  const int64_t at = (token * A.a.q_heads + head) * P.nsplit + split;
  const int64_t oat = token * A.out_token + head * A.out_head;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 32 * d + 8 * i + 4 * half;
      const f32x4 y = {o[d][4 * i] * inv, o[d][4 * i + 1] * inv, o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv};
      if (!whole) {
        *reinterpret_cast<f32x4*>(P.out + at * DIM + e) = y;
      } else if constexpr (BF16) {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        const bf16x4 w = __builtin_convertvector(y, bf16x4);
        __bf16* p = static_cast<__bf16*>(A.out) + oat + e;
        if (A.vec) {
          *reinterpret_cast<bf16x4*>(p) = w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = w[j];
        }
      } else {
        float* p = static_cast<float*>(A.out) + oat + e;
        if (A.vec) {
          *reinterpret_cast<f32x4*>(p) = y;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = y[j];
        }
      }
    }
  if (half == 0) {
    if (!whole)
      P.lse2[at] = lse2;
    else if (A.lse)
      A.lse[token * A.a.q_heads + head] = lse2 * 0.69314718055994530942f;
  }
}

template <int DIM, bool BF16, int NW>
hipError_t launch(const KvAttention& a, const Partials& p, hipStream_t stream) {
  const int64_t rows = a.batch.max_new * (a.a.q_heads / a.cache.kv_heads);
  const uint32_t tiles = (uint32_t)((rows + 32 * NW - 1) / (32 * NW));
  const uint32_t pairs = (uint32_t)(a.batch.batch * a.cache.kv_heads);
  k_kv_prompt<DIM, BF16, NW><<<pairs * tiles * (uint32_t)p.nsplit, 64 * NW, 0, stream>>>(a, p, pairs, tiles);
  return hipGetLastError();
}

template <int DIM>
hipError_t launch(const KvAttention& a, const Partials& p, int tile_rows, hipStream_t stream) {
  if constexpr (DIM < 256) {
    if (tile_rows == 256) return a.bf16 ? launch<DIM, true, 8>(a, p, stream) : launch<DIM, false, 8>(a, p, stream);
  }
  return a.bf16 ? launch<DIM, true, 4>(a, p, stream) : launch<DIM, false, 4>(a, p, stream);
}

}  // namespace

hipError_t kv_prompt_launch(const KvAttention& a, const Partials& p, int tile_rows, hipStream_t stream) {
  switch (a.cache.dim) {
    case 64: return launch<64>(a, p, tile_rows, stream);
    case 128: return launch<128>(a, p, tile_rows, stream);
    default: return launch<256>(a, p, tile_rows, stream);
  }
}

}  // namespace gptq
