// Attention of many query rows over the paged 8-bit cache: prompts and chunks.
//
// S^T = K Q^T and O^T += V^T P^T on v_mfma_f32_32x32x16_f16.  A wave keeps 32 rows
// (query token and head of one key head's group) as the columns: queries and
// output in registers, keys and values of 64 tokens in LDS, shared by the
// workgroup's waves.  Codes are widened to fp16 once, on their way into LDS;
// widening them in every wave would cost as many VALU cycles as the softmax.
//
// Column q of S^T lies in lanes q and q + 32, which hold tokens 8 (r / 4) + 4 half +
// r % 4; the values' 16 tokens are stored in LDS in the order (0-3, 8-11, 4-7,
// 12-15), so that a lane's weights are its operand of the second product where
// they are.  LDS rows are XOR-swizzled in 16-byte pieces for 64 banks (swizzled
// for 32, reads of V took twice the cycles).
//
// What bounds it (dim 128, 256 rows, 64 tokens a turn): per wave and turn 32
// products of 32 cycles and some 190 VALU instructions of the softmax, 34 of them
// exponentials at a quarter of the rate, and 70 of the widening.  Run one after the
// other these took 7000 cycles a turn of the SIMD's two waves.  So the two waves
// of a SIMD run half a turn apart, one's products beside the other's softmax, with a
// barrier where they change over, LDS operands are read 8 products ahead in an order
// that is written out, and addresses, page look-ups and the scales of 8 tiles at a
// time stay out of the softmax: 4300 cycles.  Counters over a whole call (3.8e5 cycles):
// matrix cores busy 36 % of a SIMD's cycles, vector instructions 53 %, some instruction of
// any kind 75 %, so products and softmax run side by side only in part; what holds the
// rest has not been traced.  Sustained, the clock is near 2.0 GHz.  A causal prompt of
// 4096 tokens and 32 heads takes 160 to 164 us (172 to 186 in a loop of its own), 740 to 860 TFLOP/s
// of the products that it needs, 0.63 to 0.73 of a large library product's rate; starting and
// ending a workgroup costs 11 us each, a tenth of it.  In fp32, with twice the products and 68 bytes
// a lane of scratch, 260 to 290 us.
//
// The softmax is an fma, an exponential and an addition a score: the key scale
// times the row's constant is one factor, the maximum is taken before it (it is not
// negative), the value scale is added to the exponent (kv_attend.h) and taken back
// out of the sum once for 16 tokens, and output and sum are rescaled only when a
// row's maximum has grown by more than 2^7.  Tiles with a value scale that is no power of two, not finite or 2^80
// below the largest take one more multiplication a score, as do those with masked places or scores that
// may be large.  Sums are of the unrounded weights (of the rounded ones, two at a time, lse lost 1e-4).
//
// The reference of a row's weights is an integer m from the largest s + lv on: as a rule differences with it are
// exact.  The sum of weights is kept to the same m, l = sum 2^(KV_C + s - m): its largest s - m lies between -123 and
// 100 (and the slack of m), so fp32 has room for it with 2^20 tokens of the least scale, and 2^-24 of it in subnormal
// numbers.  Both come from one exponential e = 2^(k + s - m), p = e v 2^(P - k), l += e 2^(KV_C - k), with any
// integer k for which e neither vanishes nor overflows:
//   k = m less the largest s of the lane's 8 tokens    always does: e is up to 2;
//   k = P + lv    takes no multiplication where v = 2^lv; it does unless scales lie 2^KV_NEAR apart (e could vanish
//                 and still count in l).
// Scores of 2^23 and more leave m no digits for lv: m is then the row's largest score and an integer d beside it, 0
// else, has the rest.
#include "kv_attend.h"

// The kernel's parts are lambdas over its registers: a call left in place would put those in memory.
#define INLINE __attribute__((always_inline))

namespace gptq {
namespace {

constexpr int PT = 64;                // tokens a tile
constexpr int SB = 8;                 // tiles whose scales are brought in together
constexpr float KV_C = -2.0f;
constexpr float KV_NEAR = 80.0f;
constexpr float LARGE = 8388608.0f;   // 2^23
constexpr float P_EXP = 7.0f;         // weights are up to 2^P_EXP in fp16, or
constexpr float P_SLACK = 7.0f;       // 2^(P_EXP + P_SLACK) while m is up to P_SLACK behind the row's maximum

// Maximum and sum over the two lanes of a column: v_permlane32_swap of x with itself leaves the lower
// half's values in one register and the upper half's in the other (VALU; a shuffle would wait behind the
// other waves' LDS reads).
__device__ __forceinline__ float column_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float column_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

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
  // Of a tile's four groups of 16 tokens: key scale, the value scale's exponent lv and 2^(KV_C - P_EXP - lv); a bit
  // for each group of value scale 2^lv, near the largest; the largest key scale.  Beside it the value scales, for
  // tiles in which not all are so.
  struct Scales {
    float ks[4], lv[4], zl[4];
    int plain;
    float ks_most, pad[2];
  };
  __shared__ __align__(16) Scales sc[2 * SB];
  __shared__ __align__(16) f32x4 value_scales[2 * SB];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 31, half = lane >> 5;
  // Workgroups go to the XCDs in turn, and within one to its four shader engines in turn, waiting for the
  // engine whose turn it is.  A sequence and key head (pair) stays on one XCD where pairs is a multiple of 8,
  // and the pairs are shifted by 8 from one (row tile, split) to the next: else a long sequence's workgroups
  // would all wait for one engine (a chunk of four prompts: 96 of 256 CUs busy at first).  The longest row
  // tiles of a causal call come first.
  const uint32_t rest = blockIdx.x / pairs, pair = (blockIdx.x + 8 * rest) % pairs;
  const int split = (int)(rest % (uint32_t)P.nsplit);
  const int rt = (int)(row_tiles - 1 - rest / (uint32_t)P.nsplit);
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

  // Queries, scaled to [2^7, 2^8) by row; the tokens a row sees, and those from full_lo to full_hi that every
  // row of this wave sees.
  const int wr0 = r0 + 32 * wave, r = wr0 + col;
  f16x8 qh[NK], ql[BF16 ? 1 : NK];
  float qs = 0.0f;
  Sees see = {0, 0};
  int full_lo = 0, full_hi = 0;
  auto load_queries = [&]() INLINE {
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
    most = column_max(most);
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
    see = row_sees(A, s, r, group);
    if (wr0 < rows) {
      const int last = (wr0 + 32 < rows ? wr0 + 32 : rows) - 1;
      full_lo = row_sees(A, s, last, group).lo, full_hi = row_sees(A, s, wr0, group).hi;
    }
  };

  f32x16 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = -INFINITY, md = 0.0f, l = 0.0f;

  // A thread's pieces of the tiles to come.  The 64 pieces of a wave lie in one group of 16 tokens, for K
  // and for V, so their page is one number a wave, read a tile ahead of the pieces, which thus never wait for
  // the table, and the address is scalar work but for a lane's own offset, which does not change: with t a
  // multiple of 64, place (t + j) % block is t % block + j % block.  Past the end the pieces are those of the
  // last token's page: in bounds, of no use.
  u32x4v kp[PER], vp[PER];
  int page_k[PER], page_v[PER], bad = 0;
  const int wave0 = __builtin_amdgcn_readfirstlane((int)threadIdx.x) & ~63;
  const int t0 = (int)first, t1 = (int)stop;
  const uint32_t page_bytes = (uint32_t)A.cache.kv_heads * (uint32_t)(block * DIM);  // at most 2^31
  const int8_t* k_base = A.cache.k_codes + (int64_t)hk * block * DIM;
  const int8_t* v_base = A.cache.v_codes + (int64_t)hk * block * DIM;
  // piece i of thread x
  auto piece = [&](int x, int i) INLINE { return (x + i * NT) & (PIECES - 1); };
  uint32_t off_k[PER], off_v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int p = piece(threadIdx.x, i);
    off_k[i] = (uint32_t)((p / (DIM / 16) & (block - 1)) * DIM + p % (DIM / 16) * 16);
    off_v[i] = (uint32_t)((16 * (p / DIM) & (block - 1)) * DIM + p % DIM * 16);
  }
  auto entry = [&](int tok) INLINE { return table[(tok < t1 ? tok : t1 - 1) >> shift]; };
  auto checked = [&](int page) INLINE {
    const bool ok = (uint32_t)page < (uint32_t)A.cache.pages;
    bad |= !ok;
    return ok ? (uint32_t)page : 0u;
  };
  auto pages = [&](int t_k, int t_v) INLINE {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      page_k[i] = entry(t_k + piece(wave0, i) / (DIM / 16));
      page_v[i] = entry(t_v + 16 * (piece(wave0, i) / DIM));
    }
  };
  auto fetch_k = [&](int t) INLINE {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t page = checked(__builtin_amdgcn_readfirstlane(page_k[i]));
      kp[i] = *reinterpret_cast<const u32x4v*>(k_base + ((uint64_t)page * page_bytes + (uint32_t)((t & (block - 1)) * DIM)) +
                                               off_k[i]);
    }
  };
  auto fetch_v = [&](int t) INLINE {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t page = checked(__builtin_amdgcn_readfirstlane(page_v[i]));
      vp[i] = *reinterpret_cast<const u32x4v*>(v_base + ((uint64_t)page * page_bytes + (uint32_t)((t & (block - 1)) * DIM)) +
                                               off_v[i]);
    }
  };
  // Quarter q of piece i, 8 codes widened and written: q 0, 1 of K's piece (to buffer bk), 2, 3 of V's (bv).
  auto place = [&](int i, int q, int bk, int bv) INLINE {
    const int p = piece(threadIdx.x, i);
    if (q < 2) {
      const int tok = p / (DIM / 16), c = 2 * (p % (DIM / 16)) + q;
      *reinterpret_cast<f16x8*>(lds + bk * KB + tok * KROW + 16 * (c ^ (tok & (KC - 1)))) =
          codes_to_f16(kp[i][2 * q], kp[i][2 * q + 1]);
    } else {
      const int c = 2 * (p / DIM) + q - 2, d = p % DIM;
      *reinterpret_cast<f16x8*>(lds + 2 * KB + bv * VB + d * VROW + 16 * (c ^ (d >> 1 & 7))) =
          codes_to_f16(vp[i][q - 2], vp[i][q]);
    }
  };

  // The scales of SB tiles at a time, by the first wave (lane 4 j + g: group g of the batch's tile j): pages
  // looked up, scales read and the result placed in different turns, a batch ahead of its use.  The largest
  // value scale so far is taken over the whole batch.
  int page_s = 0;
  float next_ks = 0.0f, next_vs = 0.0f, lv_most = KV_LV_MIN;
  auto look_s = [&](int batch) INLINE { page_s = entry(t0 + PT * SB * batch + 16 * (lane & (4 * SB - 1))); };
  auto fetch_s = [&](int batch) INLINE {
    const bool ok = (uint32_t)page_s < (uint32_t)A.cache.pages;
    if (!ok) bad = 1;
    const int64_t sg = (int64_t)(ok ? page_s : 0) * A.cache.kv_heads + hk;
    next_ks = A.cache.k_scales[sg];
    next_vs = A.cache.v_scales[sg];
    if (t0 + PT * SB * batch + 16 * (lane & (4 * SB - 1)) >= t1) next_vs = 0.0f;
  };
  auto place_s = [&](int batch) INLINE {
    const float lv = value_exponent(next_vs);
    lv_most = fmaxf(lv_most, lv);
#pragma unroll
    for (int k = 1; k < 4 * SB; k *= 2) lv_most = fmaxf(lv_most, __shfl_xor(lv_most, k));
    const int g = lane & 3, at = SB * (batch & 1) + (lane >> 2 & (SB - 1));
    int plain = lv >= lv_most - KV_NEAR && next_vs == ldexpf(1.0f, (int)lv) ? 1 << g : 0;
    plain |= __shfl_xor(plain, 1);
    plain |= __shfl_xor(plain, 2);
    float ks_most = fmaxf(next_ks, __shfl_xor(next_ks, 1));
    ks_most = fmaxf(ks_most, __shfl_xor(ks_most, 2));
    if (lane < 4 * SB) {
      sc[at].ks[g] = next_ks;
      sc[at].lv[g] = lv;
      sc[at].zl[g] = ldexpf(1.0f, (int)(KV_C - P_EXP - lv));
      sc[at].plain = plain;
      sc[at].ks_most = ks_most;
      value_scales[at][g] = next_vs;
    }
  };

  f16x8 ph[4], pl[BF16 ? 1 : 4];  // a tile's weights, from its softmax to its output
  Scales S;                       // its scales, read with the last operands of its scores
  // A score is at most 2^23 times its factor: 2^22 in size where this holds.
  auto are_small = [&]() INLINE { return S.ks_most * qs < 0.5f; };
  // ANY: with masked places or scales of any kind
  auto softmax = [&]<bool ANY>(int tile, f32x16 (&x)[2]) INLINE {
    f32x4 vs;
    if constexpr (ANY) {
      vs = value_scales[tile & (2 * SB - 1)];
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = t0 + PT * tile + 32 * tt + 8 * (i >> 2) + 4 * half + (i & 3);
          x[tt][i] = j >= see.lo && j < see.hi ? x[tt][i] : -INFINITY;
        }
    }
    float f[4], top[4], most = -INFINITY;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      f[g] = S.ks[g] * qs;
      const int e = 8 * (g & 1);
      const f32x16& z = x[g >> 1];
      const float y = fmaxf(fmaxf(fmaxf(fmaxf(z[e], z[e + 1]), z[e + 2]), fmaxf(fmaxf(z[e + 3], z[e + 4]), z[e + 5])),
                            fmaxf(z[e + 6], z[e + 7]));
      // a masked group stays out whatever its factor is (0, infinite or NaN)
      if constexpr (ANY) top[g] = y == -INFINITY ? y : y * f[g];
      most = fmaxf(most, ANY ? top[g] + S.lv[g] : fmaf(y, f[g], S.lv[g]));
    }
    most = column_max(most);
    // to a new reference; 2^by in two steps, as l 2^by may be a number where 2^by is none
    auto turn = [&](float by) INLINE {
      const float half_way = exp2_fast(0.5f * by);
      l = l * half_way * half_way;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d] *= half_way * half_way;
    };
    if (ANY && __any(!are_small() || m >= LARGE)) {
      float first = fmaxf(m, column_max(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]))));
      const bool large = fabsf(first) >= LARGE && first != -INFINITY;
      first = large ? first : m;
      float d = KV_LV_MIN;
#pragma unroll
      for (int g = 0; g < 4; ++g) d = fmaxf(d, S.lv[g] - (first - top[g]));
      d = ceilf(fmaxf(column_max(d), md + (m - first)));
      d = large ? d : md;
      turn(large ? (m - first) + (md - d) : 0.0f);
      m = first, md = d;
      most = large ? m : most;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        // a score for itself: with m taken off in one step it would not be exact
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y = x[g >> 1][8 * (g & 1) + i];
          x[g >> 1][8 * (g & 1) + i] = y == -INFINITY ? y : y * f[g];
        }
        f[g] = 1.0f;
      }
    }
    if (__any(most > m + P_SLACK)) {
      const float mn = fmaxf(m, ceilf(most));
      turn(mn > m ? (m - mn) + md : 0.0f);
      md = mn > m ? 0.0f : md;
      m = mn;
    }
    const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float k = !ANY ? P_EXP + S.lv[g] : top[g] == -INFINITY ? 0.0f : ceilf(fminf(base - top[g], 1024.0f));
      const float add = ANY && fabsf(base) >= LARGE ? -top[g] : k - base;
      float p[8], sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = x[g >> 1][8 * (g & 1) + i];
        float e = exp2_fast(fmaf(y, f[g], add));
        if constexpr (ANY) e = y == -INFINITY ? 0.0f : e;
        p[i] = e;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += p[i];
      if constexpr (ANY) {
        const float zp = ldexpf(vs[g], (int)(P_EXP - md - k));
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = x[g >> 1][8 * (g & 1) + i] == -INFINITY ? 0.0f : p[i] * zp;
      }
      if constexpr (BF16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) ph[g][i] = (_Float16)p[i];
      } else {
        split16(p, ph[g], pl[g]);
      }
      l = ANY ? l + ldexpf(sum, (int)(KV_C - md - k)) : fmaf(sum, S.zl[g], l);
    }
  };
  // The matrix products of a turn: output of the tile before (PV), scores of this one (QK).  Their LDS operands
  // are read AHEAD products before they are used, products that follow each other go to different accumulators,
  // and the tiles to come are widened between them, 8 codes to two products (10 VALU instructions in the 64
  // cycles of two): the order is written out here and kept.
  auto products = [&]<bool PV, bool QK>(int tile, f32x16 (&x)[2]) INLINE {
    constexpr int NPV = PV ? 4 * ND : 0, N = NPV + (QK ? 2 * NK : 0), AHEAD = 8;
    constexpr int SIDES = QK ? 4 * PER + 2 : 0;
    const char* vb = lds + 2 * KB + ((tile - 1) & 1) * VB;
    const char* kb = lds + (tile & 1) * KB;
    const int t = t0 + PT * tile;
    auto operand = [&](int i) INLINE {
      if (i < NPV) {
        const int dd = 32 * (i % ND) + col;
        return *reinterpret_cast<const f16x8*>(vb + dd * VROW + 16 * ((2 * (i / ND) + half) ^ (dd >> 1 & 7)));
      }
      const int k = (i - NPV) >> 1, tok = 32 * ((i - NPV) & 1) + col;
      return *reinterpret_cast<const f16x8*>(kb + tok * KROW + 16 * ((2 * k + half) ^ (tok & (KC - 1))));
    };
    auto product = [&](int i, f16x8 a) INLINE {
      if (i < NPV) {
        const int g = i / ND, d = i % ND;
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, ph[g], o[d], 0, 0, 0);
        if constexpr (!BF16) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, pl[g], o[d], 0, 0, 0);
      } else {
        const int k = (i - NPV) >> 1, tt = (i - NPV) & 1;
        x[tt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, qh[k], x[tt], 0, 0, 0);
        if constexpr (!BF16) x[tt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a, ql[k], x[tt], 0, 0, 0);
      }
    };
    auto side = [&](int j) INLINE {
      if (j < 4 * PER)
        place(j / 4, j % 4, (tile + 1) & 1, tile & 1);
      else if (j == 4 * PER) {
        fetch_k(t + 2 * PT);
        fetch_v(t + PT);
      } else {
        pages(t + 3 * PT, t + 2 * PT);
      }
    };
    f16x8 a[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) a[i] = operand(i);
    if constexpr (QK) {
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 16; ++i) x[tt][i] = 0.0f;
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      product(i, a[i % AHEAD]);
      product(i + 1, a[(i + 1) % AHEAD]);
      if (i + AHEAD < N) {
        a[i % AHEAD] = operand(i + AHEAD);
        a[(i + 1) % AHEAD] = operand(i + 1 + AHEAD);
      }
      if (i / 2 < SIDES) side(i / 2);
      if (QK && i + 4 == N) S = sc[tile & (2 * SB - 1)];
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = N / 2; j < SIDES; ++j) side(j);
    if constexpr (QK) {
      if (wave == 0) {
        const int batch = tile / SB + 1;
        switch (tile & (SB - 1)) {
          case 0: look_s(batch); break;
          case 2: fetch_s(batch); break;
          case 4: place_s(batch); break;
        }
      }
    }
  };
  // Everything a wave has written to LDS is there for all when they pass; loads from HBM stay
  // on their way.
  auto meet = [&]() INLINE {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // A wave's turn i has two phases: matrix products (output of tile i - 1, scores of tile i) with the tiles to
  // come brought in and widened beside them, then the softmax of tile i.  With 8 waves, two on a SIMD, the
  // second four are a phase behind the first, so that one wave's products run beside the other's softmax.
  // In slots (a slot ends where all meet) the first four have their products of turn i in slot 2 i, the
  // second in slot 2 i + 1; in it a wave reads K(i) and V(i - 1) and writes its pieces of K(i + 1) and V(i).
  // The buffers of K(i + 1) and V(i) held K(i - 1) and V(i - 2), last read in slot 2 i - 1, and are first read
  // in slot 2 i + 2.
  const int tiles = (t1 - t0 + PT - 1) / PT;
  const bool late = wave >= 4;
  if (tiles > 0) {
    f32x16 x[2];
    auto weigh = [&](int tile) INLINE {
      const int t = t0 + PT * tile;
      // one condition of vector registers, though it is the same in all lanes: as a scalar branch the compiler reads
      // ahead across it, and spills (188 bytes a lane at dim 128)
      if ((t >= full_lo) & (t + PT <= full_hi) & (S.plain == 15) & are_small())
        softmax.template operator()<false>(tile, x);
      else
        softmax.template operator()<true>(tile, x);
    };
    pages(t0, t0);
    if (wave == 0) look_s(0);
    fetch_k(t0);
    fetch_v(t0);
    pages(t0 + PT, t0);
    if (wave == 0) fetch_s(0);
    load_queries();  // while the first tile is on its way
#pragma unroll
    for (int i = 0; i < PER; ++i) place(i, 0, 0, 0), place(i, 1, 0, 0);
    if (wave == 0) place_s(0);
    fetch_k(t0 + PT);
    pages(t0 + 2 * PT, t0 + PT);
    meet();
    if (late) meet();
    products.template operator()<false, true>(0, x);
    meet();
    for (int tile = 0; tile < tiles - 1; ++tile) {
      weigh(tile);
      meet();
      __builtin_amdgcn_s_setprio(1);
      products.template operator()<true, true>(tile + 1, x);
      __builtin_amdgcn_s_setprio(0);
      meet();
    }
    weigh(tiles - 1);
    meet();
    products.template operator()<true, false>(tiles, x);
    if (NW > 4 && !late) meet();
    if (bad) raise_einval(A.d_status);
  }

  l = column_sum(l);
  if (r >= rows) return;
  const float inv = l == 0.0f ? 0.0f : exp2_fast(KV_C - P_EXP) / l;
  // the exponent of l is added to m's as the integer that it is
  const float lse2 = l == 0.0f ? -INFINITY
                               : m + (md - KV_C + (float)__builtin_amdgcn_frexp_expf(l)) +
                                     __log2f(__builtin_amdgcn_frexp_mantf(l));
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

}  // namespace

hipError_t kv_prompt_launch(const KvAttention& a, const Partials& p, int tile_rows, hipStream_t stream) {
  switch (a.cache.dim) {
    case 64: return a.bf16 ? launch<64, true, 4>(a, p, stream) : launch<64, false, 4>(a, p, stream);
    case 128:
      if (!a.bf16) return launch<128, false, 8>(a, p, stream);
      return tile_rows == 256 ? launch<128, true, 8>(a, p, stream) : launch<128, true, 4>(a, p, stream);
    default: return a.bf16 ? launch<256, true, 4>(a, p, stream) : launch<256, false, 4>(a, p, stream);
  }
}

}  // namespace gptq
