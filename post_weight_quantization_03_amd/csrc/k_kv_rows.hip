// Attention of few query rows over the paged 8-bit cache: single tokens, guessed
// tokens, short chunks.
//
// A row is a query token and head; the rows of a key head's group go together, 16
// (or 32) at a time, as the columns of two matrix products on
// v_mfma_f32_16x16x32_f16:  S^T = K Q^T,  O^T += V^T P^T.  Every cache byte is read
// once a row tile, straight from HBM into the lane that needs it as an operand:
// no LDS, no barrier in the loop.
//   K: row m = lane % 16 of tile t is token 16 (m / 4) + 4 t + m % 4 of 64, so that
//      in the product lane (q = l % 16, g = l / 16) holds tokens 16 g .. 16 g + 15 of
//      row q, one scale group, in order; its 16-byte loads are elements 64 i + 16 g
//      .. + 15, the k-slots of two MFMAs.
//   V: lane (d = l % 16, g) loads tokens 16 g .. 16 g + 15 of element d in one piece
//      (the cache's order), the k-slots of two MFMAs, which meet the same tokens of P
//      in the same lane group: P never moves between lanes.
// A wave goes through 64 tokens a turn, four waves side by side; the loads of the
// next turn's K are issued when the scores are done, those of V when the output is,
// so about 8 to 16 KB a wave is always on its way.  Each keeps its own maximum, sum
// and output; they are joined in LDS at the end, and over the splits of a long
// sequence by k_kv_join.
//
// One token over 64 sequences of 2048 to 8192 tokens, 32 heads of 128: 2.69 GB in 457 us, 5.9 TB/s (a large
// copy moves 4.9 TB/s, read and written); over 131035 tokens, 8 key heads: 268 MB in 52 us, and 5 for
// joining 65 splits; over 43 tokens 7 us, the latencies of lengths, table, cache and output in turn.  fp32:
// 460, 54 to 56 and 7.2 us.  Three waves a SIMD instead of two spill: 707 us for the first.
// With several row tiles each reads the cache: 64 rows over 4 x 30000 tokens, 8 key heads, 246 MB, take 92 to 95 us in bf16
// (one tile of 32 rows twice) and 150 to 155 in fp32 (tiles of 16 rows, four times).
//
// Scales: K's multiplies the score, V's goes into the exponent of the weight (kv_attend.h), whose reference is kept
// in two parts, the largest score r and an integer d: scores of any size leave d its digits.
#include "kv_attend.h"

namespace gptq {
namespace {

constexpr int KW = 4;  // waves
constexpr float P_EXP = 14.0f;  // weights are up to 2^P_EXP in fp16, normal numbers down to 2^-28 of that

template <int DIM, bool BF16, int CT, bool MASKED>
__global__ __launch_bounds__(64 * KW, DIM == 256 ? 1 : 2) void k_kv_rows(KvAttention A, Partials P, uint32_t row_tiles) {
  constexpr int NI = DIM / 64;  // 16-byte K loads a row
  constexpr int NK = DIM / 32;  // MFMA steps of the first product
  constexpr int ND = DIM / 16;  // d tiles
  constexpr int CW = DIM < 128 ? DIM : 128;  // columns joined at a time
  constexpr int LDO = CW + 4;
  __shared__ __align__(16) float so[KW][16 * LDO];
  __shared__ float sm[KW][16 * CT], sd[KW][16 * CT], sl[KW][16 * CT];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n16 = lane & 15, g = lane >> 4;
  // The splits are the slowest index: workgroups go to the XCDs and their shader engines in turn, and the
  // last splits, which short sequences lack, would else leave some of these idle.
  const uint32_t tiles = (uint32_t)A.batch.batch * (uint32_t)A.cache.kv_heads * row_tiles;
  const int split = (int)(blockIdx.x / tiles);
  uint32_t id = blockIdx.x % tiles;
  const int rt = (int)(id % row_tiles);
  id /= row_tiles;
  const int hk = (int)(id % (uint32_t)A.cache.kv_heads), b = (int)(id / (uint32_t)A.cache.kv_heads);
  const Seq s = load_seq(A.batch, b, A.d_status);
  const int group = A.a.q_heads / A.cache.kv_heads;
  const int rows = s.n * group, r0 = rt * 16 * CT;
  if (r0 >= rows) return;
  const Span span = row_span<MASKED>(A, s, r0, 16 * CT, group);
  const int64_t first = span.begin + split * P.chunk;
  if (split > 0 && first >= span.end) return;
  const bool whole = span.end - span.begin <= P.chunk;
  const int64_t stop = first + P.chunk < span.end ? first + P.chunk : span.end;
  const int32_t* table = A.batch.block_table + b * A.batch.table_stride;
  const int shift = __builtin_ctz((unsigned)A.cache.block);
  const int block = A.cache.block;

  // A lane's K rows of a tile lie in group n16 / 4 of its four groups of 16 tokens, its V pieces and its scores'
  // scales in group g.  The pages of both are read a tile ahead of what they hold and looked at only then (a
  // wait for the table would wait for the loads before it, too).  Past the end they are the last token's.
  u32x4v kr[4][NI], vr[ND];
  float ks = 0.0f, vs = 0.0f;
  int page_k = 0, page_v = 0, bad = 0;
  const int gk = n16 >> 2;
  const uint32_t page_bytes = (uint32_t)A.cache.kv_heads * (uint32_t)(block * DIM);  // at most 2^31
  const int8_t* k_base = A.cache.k_codes + (int64_t)hk * block * DIM + (n16 & 3) * DIM + 16 * g;
  const int8_t* v_base = A.cache.v_codes + (int64_t)hk * block * DIM + 16 * n16;
  const int t_stop = (int)stop;
  auto pages = [&](int t) {
    const int tk = t + 16 * gk, tv = t + 16 * g;
    const int ck = tk < t_stop ? tk : t_stop - 1, cv = tv < t_stop ? tv : t_stop - 1;
    page_k = table[(MASKED ? span.looked_up(ck) : ck) >> shift];
    page_v = table[(MASKED ? span.looked_up(cv) : cv) >> shift];
  };
  auto actual = [&](int t) { return MASKED ? span.token(t) : t; };
  auto checked = [&](int page) {
    const bool ok = (uint32_t)page < (uint32_t)A.cache.pages;
    bad |= !ok;
    return ok ? (uint32_t)page : 0u;
  };
  auto load_k = [&](int t) {
    const int8_t* p = k_base + (uint64_t)checked(page_k) * page_bytes + (uint32_t)(((actual(t) + 16 * gk) & (block - 1)) * DIM);
#pragma unroll
    for (int tt = 0; tt < 4; ++tt)
#pragma unroll
      for (int i = 0; i < NI; ++i) kr[tt][i] = *reinterpret_cast<const u32x4v*>(p + 4 * tt * DIM + 64 * i);
    ks = A.cache.k_scales[(int64_t)checked(page_v) * A.cache.kv_heads + hk];
  };
  auto load_v = [&](int t) {
    const uint32_t page = checked(page_v);
    const int8_t* p = v_base + (uint64_t)page * page_bytes + (uint32_t)(((actual(t) + 16 * g) & (block - 1)) * DIM);
#pragma unroll
    for (int d = 0; d < ND; ++d) vr[d] = *reinterpret_cast<const u32x4v*>(p + 256 * d);
    vs = A.cache.v_scales[(int64_t)page * A.cache.kv_heads + hk];
  };

  // the first tile is on its way while the queries are read and scaled
  int t = (int)first + 64 * wave;
  if (t < t_stop) {
    pages(t);
    load_k(t);
    load_v(t);
    pages(t + 64 * KW);
  }

  // queries, scaled to [2^7, 2^8) by row
  f16x8 qh[CT][NK], ql[CT][BF16 ? 1 : NK];
  float qs[CT];
  Sees see[CT];
  RowMask mask[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int r = r0 + 16 * c + n16;
    float x[NK][8];
    float most = 0.0f;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[k][j] = 0.0f;
      if (r < rows) {
        const int64_t o = (s.row + r / group) * A.q_token + (hk * group + r % group) * A.q_head + 64 * (k >> 1) +
                          16 * g + 8 * (k & 1);
        if (A.vec)
          load8<BF16, true>(A.q, o, x[k]);
        else
          load8<BF16, false>(A.q, o, x[k]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(x[k][j]));
    }
    most = fmaxf(most, __shfl_xor(most, 16));
    most = fmaxf(most, __shfl_xor(most, 32));
    float up, down;
    row_scale(most, up, down);
    qs[c] = A.a.sm_scale * 1.44269504088896340736f * down;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[k][j] *= up;
      if constexpr (BF16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) qh[c][k][j] = (_Float16)x[k][j];
      } else {
        split16(x[k], qh[c][k], ql[c][k]);
      }
    }
    if constexpr (MASKED)
      mask[c] = row_mask(A, s, r, group, A.d_status);
    else
      see[c] = row_sees(A, s, r, group);
  }
  // tokens from full_lo to full_hi are seen by every row of the tile
  int full_lo = 0, full_hi = 0;
  Full every;
  if constexpr (MASKED) {
    every = full_span(A, s, r0, (r0 + 16 * CT < rows ? r0 + 16 * CT : rows) - 1, group);
  } else {
    const int last = (r0 + 16 * CT < rows ? r0 + 16 * CT : rows) - 1;
    full_lo = row_sees(A, s, last, group).lo;
    full_hi = row_sees(A, s, r0, group).hi;
  }

  f32x4 o[CT][ND];
  float m[CT], md[CT], l[CT];  // largest score; integer beside it; sum of 2^(s - m)
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    m[c] = -INFINITY;
    md[c] = KV_LV_MIN;
    l[c] = 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[c][d] = (f32x4){0, 0, 0, 0};
  }

  for (; t < t_stop; t += 64 * KW) {
    const int tn = t + 64 * KW;
    // scores
    f32x4 x[CT][4];
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
      for (int c = 0; c < CT; ++c) x[c][tt] = (f32x4){0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const u32x4v w = kr[tt][k >> 1];
        const f16x8 a = (k & 1) ? codes_to_f16(w[2], w[3]) : codes_to_f16(w[0], w[1]);
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          x[c][tt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, qh[c][k], x[c][tt], 0, 0, 0);
          if constexpr (!BF16) x[c][tt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, ql[c][k], x[c][tt], 0, 0, 0);
        }
      }
    }
    const float ks_now = ks;
    const float vs_now = t + 16 * g < t_stop ? vs : 0.0f;
    if (tn < t_stop) load_k(tn);

    const float lv = value_exponent(vs_now);
    const bool full = MASKED ? every.has(actual(t)) : t >= full_lo && t + 64 <= full_hi;
    f16x8 ph[CT][2], pl[CT][BF16 ? 1 : 2];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const float f = ks_now * qs[c];
      uint32_t seen = 0;  // MASKED: of the lane's 16 tokens
      if constexpr (MASKED) {
        if (!full) seen = (uint32_t)(row_word(mask[c], s.n, actual(t)) >> (16 * g));
      }
      float top = -INFINITY;  // of the 16 scores
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float y = x[c][tt][r] * f;
          if (!full) {
            const int j = t + 16 * g + 4 * tt + r;
            y = (MASKED ? (seen >> (4 * tt + r) & 1) != 0 : j >= see[c].lo && j < see[c].hi) ? y : -INFINITY;
          }
          x[c][tt][r] = y;
          top = fmaxf(top, y);
        }
      float mn = fmaxf(top, __shfl_xor(top, 16));
      mn = fmaxf(mn, __shfl_xor(mn, 32));
      mn = fmaxf(m[c], mn);
      const float base = mn == -INFINITY ? 0.0f : mn;
      const float behind = top == -INFINITY ? 0.0f : base - top, k = ceilf(fminf(behind, 1024.0f));
      float dn = top == -INFINITY ? KV_LV_MIN : ceilf(lv - behind);
      dn = fmaxf(dn, __shfl_xor(dn, 16));
      dn = fmaxf(dn, __shfl_xor(dn, 32));
      const float risen = m[c] - base;
      dn = fmaxf(fmaxf(dn, ceilf(md[c] + risen)), KV_LV_MIN);
      const float turn_l = exp2_fast(risen), turn_o = exp2_fast(risen + (md[c] - dn));
      m[c] = mn;
      md[c] = dn;
      // e = 2^(s - top), up to 1; from there to the row's reference by an integer and what is left of it
      const float from = top == -INFINITY ? 0.0f : top, rest = exp2_fast(k - fminf(behind, 1024.0f));
      const float zp = ldexpf(vs_now * rest, (int)(P_EXP - dn - k));
      float sum = 0.0f;
      float p[16];
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float y = x[c][tt][r], e = exp2_fast(y - from);
          sum += e;
          p[4 * tt + r] = full || y != -INFINITY ? e * zp : 0.0f;  // also where the block's scale of values is NaN
        }
      l[c] = fmaf(l[c], turn_l, ldexpf(sum * rest, (int)-k));
#pragma unroll
      for (int d = 0; d < ND; ++d) o[c][d] *= turn_o;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float q8[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) q8[j] = p[8 * u + j];
        if constexpr (BF16) {
#pragma unroll
          for (int j = 0; j < 8; ++j) ph[c][u][j] = (_Float16)q8[j];
        } else {
          split16(q8, ph[c][u], pl[c][u]);
        }
      }
    }
    // output
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f16x8 a = codes_to_f16(vr[d][2 * u], vr[d][2 * u + 1]);
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          o[c][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, ph[c][u], o[c][d], 0, 0, 0);
          if constexpr (!BF16) o[c][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pl[c][u], o[c][d], 0, 0, 0);
        }
      }
    if (tn < t_stop) {
      load_v(tn);
      pages(tn + 64 * KW);
    }
  }
  if (bad) raise_einval(A.d_status);

  // join the waves
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    l[c] += __shfl_xor(l[c], 16);
    l[c] += __shfl_xor(l[c], 32);
    if (g == 0) sm[wave][16 * c + n16] = m[c], sd[wave][16 * c + n16] = md[c], sl[wave][16 * c + n16] = l[c];
  }
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int h = 0; h < DIM / CW; ++h) {
      __syncthreads();
#pragma unroll
      for (int d = 0; d < CW / 16; ++d)
        *reinterpret_cast<f32x4*>(&so[wave][n16 * LDO + 16 * d + 4 * g]) = o[c][h * (CW / 16) + d];
      __syncthreads();
      for (int i = threadIdx.x; i < 16 * CW / 8; i += 64 * KW) {
        const int row = i / (CW / 8), d = 8 * (i % (CW / 8));
        const int r = r0 + 16 * c + row;
        if (r >= rows) continue;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < KW; ++w) mm = fmaxf(mm, sm[w][16 * c + row]);
        const float base = mm == -INFINITY ? 0.0f : mm;
        float dd = KV_LV_MIN;
#pragma unroll
        for (int w = 0; w < KW; ++w) dd = fmaxf(dd, ceilf(sd[w][16 * c + row] + (sm[w][16 * c + row] - base)));
        float sum = 0.0f, y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.0f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const float risen = sm[w][16 * c + row] - base;
          const float fo = exp2_fast(risen + (sd[w][16 * c + row] - dd));
          sum = fmaf(sl[w][16 * c + row], exp2_fast(risen), sum);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = fmaf(fo, so[w][row * LDO + d + j], y[j]);
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // a sum of NaN stays NaN
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = ldexpf(y[j] * inv, (int)(dd - P_EXP));
        const float lse2 = sum == 0.0f ? -INFINITY : mm + __log2f(sum);
        const int64_t token = s.row + r / group;
        const int head = hk * group + r % group;
        // lse first: of a condition that ends where the loop does, the compiler has kept the mask for later copies
        if (whole) {
          if (A.lse && h == 0 && d == 0) A.lse[token * A.a.q_heads + head] = lse2 * 0.69314718055994530942f;
          const int64_t at = token * A.out_token + head * A.out_head + h * CW + d;
          if (A.vec)
            store8<BF16, true>(A.out, at, y);
          else
            store8<BF16, false>(A.out, at, y);
        } else {
          const int64_t at = (token * A.a.q_heads + head) * P.nsplit + split;
          if (h == 0 && d == 0) P.lse2[at] = lse2;
          store8<false, true>(P.out, at * DIM + h * CW + d, y);
        }
      }
    }
}

// Joins the splits of each row that has several: out = sum 2^(lse2_s - max) out_s /
// sum 2^(lse2_s - max).  A workgroup a row and head: the splits' factors go to LDS,
// then each group of dim / 4 threads adds every (1024 / dim)-th split, and the groups
// are added in order.  All loads of a thread are independent.
// A few splits are joined by a wave a row instead: a workgroup a row is bound by the
// workgroups' start (2 splits of 48000 rows: 89 us against 28).
constexpr int JT = 256;
constexpr int JOIN_FEW = 8;

template <int DIM, bool BF16>
__global__ __launch_bounds__(JT) void k_kv_join(KvAttention A, Partials P, uint32_t tile_rows) {
  constexpr int TG = DIM / 4, NG = JT / TG;  // threads a group, groups
  __shared__ float fac[JT];
  __shared__ float red[JT / 64];
  __shared__ __align__(16) float part[NG][DIM];
  __shared__ float psum[NG];
  uint32_t id = blockIdx.x;
  const int h = (int)(id % (uint32_t)A.a.q_heads);
  id /= (uint32_t)A.a.q_heads;
  const int i = (int)(id % (uint32_t)A.batch.max_new);
  const int b = (int)(id / (uint32_t)A.batch.max_new);
  const Seq s = load_seq(A.batch, b, nullptr);
  if (i >= s.n) return;
  const int group = A.a.q_heads / A.cache.kv_heads;
  const int r = i * group + h % group;
  const int first_row = r / (int)tile_rows * (int)tile_rows;
  const Span span = A.masked ? row_span<true>(A, s, first_row, (int)tile_rows, group)
                             : row_span<false>(A, s, first_row, (int)tile_rows, group);
  const int ns = (int)((span.end - span.begin + P.chunk - 1) / P.chunk);
  if (ns <= 1) return;
  const int64_t token = s.row + i, at = (token * A.a.q_heads + h) * P.nsplit;
  const int tid = threadIdx.x, tg = tid / TG, td = tid % TG;
  float mm = -INFINITY;
  for (int k = tid; k < ns; k += JT) mm = fmaxf(mm, P.lse2[at + k]);
#pragma unroll
  for (int k = 1; k < 64; k *= 2) mm = fmaxf(mm, __shfl_xor(mm, k));
  if ((tid & 63) == 0) red[tid >> 6] = mm;
  __syncthreads();
  mm = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float base = mm == -INFINITY ? 0.0f : mm;
  float sum = 0.0f;
  f32x4 y = {0, 0, 0, 0};
  for (int k0 = 0; k0 < ns; k0 += JT) {
    __syncthreads();
    fac[tid] = k0 + tid < ns ? exp2_fast(P.lse2[at + k0 + tid] - base) : 0.0f;
    __syncthreads();
    const int n = ns - k0 < JT ? ns - k0 : JT;
#pragma unroll 4
    for (int k = tg; k < n; k += NG) {
      const float f = fac[k];
      sum += f;
      const f32x4 p = *reinterpret_cast<const f32x4*>(P.out + (at + k0 + k) * DIM + 4 * td);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = fmaf(f, p[e], y[e]);
    }
  }
  *reinterpret_cast<f32x4*>(&part[tg][4 * td]) = y;
  if (td == 0) psum[tg] = sum;
  __syncthreads();
  if (tid >= DIM) return;
  float o = 0.0f;
  sum = 0.0f;
#pragma unroll
  for (int k = 0; k < NG; ++k) o += part[k][tid], sum += psum[k];
  o *= sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t to = token * A.out_token + h * A.out_head + tid;
  if constexpr (BF16)
    static_cast<__bf16*>(A.out)[to] = (__bf16)o;
  else
    static_cast<float*>(A.out)[to] = o;
  if (A.lse && tid == 0)
    A.lse[token * A.a.q_heads + h] = (sum == 0.0f ? -INFINITY : mm + __log2f(sum)) * 0.69314718055994530942f;
}

template <int DIM, bool BF16, bool MASKED>
hipError_t launch(const KvAttention& a, const Partials& p, int tile_rows, hipStream_t stream) {
  const int64_t rows = a.batch.max_new * (a.a.q_heads / a.cache.kv_heads);
  const uint32_t tiles = (uint32_t)((rows + tile_rows - 1) / tile_rows);
  const uint32_t grid = (uint32_t)(a.batch.batch * a.cache.kv_heads * tiles * p.nsplit);
  if constexpr (DIM == 64 || (DIM == 128 && BF16)) {
    if (tile_rows == 32)
      k_kv_rows<DIM, BF16, 2, MASKED><<<grid, 64 * KW, 0, stream>>>(a, p, tiles);
    else
      k_kv_rows<DIM, BF16, 1, MASKED><<<grid, 64 * KW, 0, stream>>>(a, p, tiles);
  } else {
    k_kv_rows<DIM, BF16, 1, MASKED><<<grid, 64 * KW, 0, stream>>>(a, p, tiles);
  }
  return hipGetLastError();
}

template <int DIM>
hipError_t launch(const KvAttention& a, const Partials& p, int tile_rows, hipStream_t stream) {
  if (a.masked)
    return a.bf16 ? launch<DIM, true, true>(a, p, tile_rows, stream) : launch<DIM, false, true>(a, p, tile_rows, stream);
  return a.bf16 ? launch<DIM, true, false>(a, p, tile_rows, stream) : launch<DIM, false, false>(a, p, tile_rows, stream);
}

}  // namespace

hipError_t kv_rows_launch(const KvAttention& a, const Partials& p, int tile_rows, hipStream_t stream) {
  switch (a.cache.dim) {
    case 64: return launch<64>(a, p, tile_rows, stream);
    case 128: return launch<128>(a, p, tile_rows, stream);
    default: return launch<256>(a, p, tile_rows, stream);
  }
}

namespace {

template <int DIM, bool BF16>
__global__ __launch_bounds__(JT) void k_kv_join_few(KvAttention A, Partials P, uint32_t tile_rows) {
  constexpr int TG = DIM / 4 < 64 ? DIM / 4 : 64, NG = 64 / TG;  // lanes a split, splits side by side
  uint32_t id = blockIdx.x * (JT / 64) + (threadIdx.x >> 6);
  const int h = (int)(id % (uint32_t)A.a.q_heads);
  id /= (uint32_t)A.a.q_heads;
  const int i = (int)(id % (uint32_t)A.batch.max_new);
  const int64_t b = id / (uint32_t)A.batch.max_new;
  if (b >= A.batch.batch) return;
  const Seq s = load_seq(A.batch, (int)b, nullptr);
  if (i >= s.n) return;
  const int group = A.a.q_heads / A.cache.kv_heads;
  const int r = i * group + h % group;
  const int first_row = r / (int)tile_rows * (int)tile_rows;
  const Span span = A.masked ? row_span<true>(A, s, first_row, (int)tile_rows, group)
                             : row_span<false>(A, s, first_row, (int)tile_rows, group);
  const int ns = (int)((span.end - span.begin + P.chunk - 1) / P.chunk);
  if (ns <= 1) return;
  const int64_t token = s.row + i, at = (token * A.a.q_heads + h) * P.nsplit;
  const int lane = threadIdx.x & 63, tg = lane / TG, td = lane % TG;
  f32x4 p[JOIN_FEW / NG];
  float e[JOIN_FEW], mm = -INFINITY;
#pragma unroll
  for (int k = 0; k < JOIN_FEW; ++k) e[k] = k < ns ? P.lse2[at + k] : -INFINITY;
#pragma unroll
  for (int k = 0; k < JOIN_FEW / NG; ++k) {
    p[k] = (f32x4){0, 0, 0, 0};
    if (k * NG + tg < ns) p[k] = *reinterpret_cast<const f32x4*>(P.out + (at + k * NG + tg) * DIM + 4 * td);
  }
#pragma unroll
  for (int k = 0; k < JOIN_FEW; ++k) mm = fmaxf(mm, e[k]);
  const float base = mm == -INFINITY ? 0.0f : mm;
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < JOIN_FEW; ++k) sum += e[k] = exp2_fast(e[k] - base);
  f32x4 y = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < JOIN_FEW / NG; ++k) {
    float f = e[k * NG];
#pragma unroll
    for (int g = 1; g < NG; ++g) f = tg == g ? e[k * NG + g] : f;
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = fmaf(f, p[k][j], y[j]);
  }
#pragma unroll
  for (int m = TG; m < 64; m *= 2)
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] += __shfl_xor(y[j], m);
  if (lane >= TG) return;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t to = token * A.out_token + h * A.out_head + 4 * td;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (BF16)
      static_cast<__bf16*>(A.out)[to + j] = (__bf16)(y[j] * inv);
    else
      static_cast<float*>(A.out)[to + j] = y[j] * inv;
  }
  if (A.lse && lane == 0)
    A.lse[token * A.a.q_heads + h] = (sum == 0.0f ? -INFINITY : mm + __log2f(sum)) * 0.69314718055994530942f;
}

}  // namespace

template <int DIM>
static void join(const KvAttention& a, const Partials& p, int tile_rows, hipStream_t stream) {
  const uint32_t grid = (uint32_t)(a.batch.batch * a.batch.max_new * a.a.q_heads);
  if (p.nsplit <= JOIN_FEW) {
    if (a.bf16)
      k_kv_join_few<DIM, true><<<(grid + 3) / 4, JT, 0, stream>>>(a, p, (uint32_t)tile_rows);
    else
      k_kv_join_few<DIM, false><<<(grid + 3) / 4, JT, 0, stream>>>(a, p, (uint32_t)tile_rows);
    return;
  }
  if (a.bf16)
    k_kv_join<DIM, true><<<grid, JT, 0, stream>>>(a, p, (uint32_t)tile_rows);
  else
    k_kv_join<DIM, false><<<grid, JT, 0, stream>>>(a, p, (uint32_t)tile_rows);
}

hipError_t kv_join_launch(const KvAttention& a, const Partials& p, int tile_rows, hipStream_t stream) {
  switch (a.cache.dim) {
    case 64: join<64>(a, p, tile_rows, stream); break;
    case 128: join<128>(a, p, tile_rows, stream); break;
    default: join<256>(a, p, tile_rows, stream); break;
  }
  return hipGetLastError();
}

}  // namespace gptq
