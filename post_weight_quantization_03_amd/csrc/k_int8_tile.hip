// The 8-bit product in tiles of rows x tokens on v_mfma_i32_16x16x64_i8.
//
// WA x WB waves, each with RB x TB blocks of 16 rows by 16 tokens; rows are the first operand, so a lane's
// sums of a block are four rows of one token, side by side in Y.  The codes of KS columns a stage go
// from memory to LDS directly (buffer loads, which give 0 past the end of the layer and of the tokens), some
// stages ahead of their use.  In LDS a row's KS codes are pieces of 16 bytes, permuted by the row so that the
// 16 lanes that a read serves at a time fall on all 64 banks (no conflicts counted).
//
// An operand is replaced, as soon as its last product is on its way, by the one SETS steps of 64 columns on: from the
// second stage on, all of a stage's operands have been read when the barrier before it is passed, and products
// follow each other without a pause.  EARLY: a stage's buffer has then been read (a wait for the wave's own reads goes
// before the barrier), and the stage BUFS on is brought into it at once; else that waits for a stage.
//
// Measured (tokens x columns x rows): 4096 x 11008 x 4096 160 us (2.31 POP/s, 256 x 256 tiles), a library's
// product of the same operands 152 to 161; 8192^3 455 us (2.42), 440 to 462.  What bounds it is power: the first keeps
// the matrix cores busy for 62 % of 2.84e5 cycles at 1.78 GHz (159 us), with operands of zeros for 61 % of 2.89e5 at
// 2.32 GHz (124 us).  So, for that case: products of 16 x 16 (170 us), which move half as many sums as those of 32 x 32 (180); no bank conflicts
// (164); waves of few rows and many tokens, as rows have to be made signed (160); and nothing by a pipeline that
// only saves cycles (177 to 180 with any of four, before these).  A call that leaves places empty is bound otherwise: 1531 x 4100 x 4099
// (204 tiles of 256 x 128 for 256 CUs, 36 to 40 us) runs at 2.5 GHz, the matrix cores of the CUs with a tile busy for
// 37 % of the cycles: a stage takes 1.0 us there, 0.4 of them products, and 49 KB a CU out of the L2s (10 TB/s).  Requests of 128 bytes of a row: with 64-byte ones
// tiles of 256 x 128 took 211 us instead of 177 (256 x 256 has no room in LDS for them).  Small tiles are bound by
// the stage's chain of wait, barrier and LDS reads (0.2 to 0.4 us), so theirs are 256 columns (64 x 4096 x 4096:
// 8.0 us, with 128 9.5), and by what the CUs read out of the L2s, 15 to 20 TB/s: with twice the waves, each half of
// them at half of the columns, products of up to 256 tiles take 3 to 8 % less and larger ones up to 30 % more (not
// kept).
#include "int8.h"

namespace gptq {
namespace {

typedef __attribute__((address_space(3))) char lds_char;
typedef uint32_t u32x4s __attribute__((ext_vector_type(4)));
typedef float f32x8i __attribute__((ext_vector_type(8)));
// of any element alignment
typedef float f32x4e __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 bf16x8e __attribute__((ext_vector_type(8), aligned(2)));

// The lambdas' arguments are constants and registers: a call left in place would put those in memory.
#define INLINE __attribute__((always_inline))

// What brings one operand in: a buffer whose start moves on with the stages.
struct Stream {
  uint64_t base;
  int64_t left;  // bytes from base to the end: below 2^32 (256 rows of 65536 codes) and at least a stage's
  __device__ __forceinline__ u32x4s buffer(bool more) const {
    u32x4s r;
    r[0] = (uint32_t)base;
    r[1] = (uint32_t)(base >> 32) & 0xffffu;
    r[2] = more ? (uint32_t)left : 0u;
    r[3] = 0x00027000u;
    return r;
  }
  __device__ __forceinline__ void advance(int columns) {
    base += columns;
    left -= columns;
  }
};

// With the wait state between the write of M0 and a load that uses it, as in direct_load.
__device__ __forceinline__ void load_to_lds(uint32_t offset, u32x4s buffer, uint32_t lds) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(offset), "s"(buffer), "{m0}"(lds));
}

// All but the wave's N newest loads have come, in every wave.
template <int N>
__device__ __forceinline__ void retire() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

template <int RB, int TB, int WA, int WB, int KS, int BUFS, int SETS, bool EARLY>
__global__ __launch_bounds__(64 * WA * WB, 2) void k_int8_tile(Int8Gemm A, uint32_t row_tiles, uint32_t token_tiles) {
  constexpr int NW = WA * WB;
  constexpr int TR = 16 * RB * WA, TT = 16 * TB * WB;  // rows and tokens of a tile
  constexpr int WR = 16 * RB;                          // rows of a wave
  constexpr int RBYTES = TR * KS, STAGE = (TR + TT) * KS;
  constexpr int PIECES = KS / 16, PER = 64 / PIECES;                    // of a row; rows a load
  constexpr int LR = TR / PER / NW, LT = TT / PER / NW, LPW = LR + LT;  // loads a wave and stage
  static_assert(LR * PER * NW == TR && LT * PER * NW == TT, "loads divide the tile evenly");
  constexpr int STEPS = KS / 64;
  static_assert(SETS <= STEPS && (!EARLY || SETS == STEPS), "a stage's operands fit, and are all held where EARLY");
  constexpr int LD = 4 * WR + 16;  // bytes of a token's sums on their way out
  constexpr int LDS = BUFS * STAGE > NW * 16 * LD ? BUFS * STAGE : NW * 16 * LD;
  __shared__ __align__(1024) char lds[LDS];
  __shared__ float token_scale[TT];
  __shared__ int32_t token_sum[TT];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int col = lane & 15, part = lane >> 4;
  const int wr = wave / WB, wt = wave % WB;

  // Workgroups go to the 8 XCDs in turn.  Each XCD takes a run of tiles in which 4 row tiles go with every token
  // tile before the next 4, so what its 32 CUs read at a time is in its L2 once.
  const uint32_t tiles = row_tiles * token_tiles, per = (tiles + 7) / 8, in = blockIdx.x / 8;
  const uint32_t id = (blockIdx.x % 8) * per + in;
  if (in >= per || id >= tiles) return;
  const uint32_t group = id / (4 * token_tiles), rest = id - group * 4 * token_tiles;
  const uint32_t width = row_tiles - 4 * group < 4 ? row_tiles - 4 * group : 4;
  const int64_t r0 = (int64_t)(4 * group + rest % width) * TR, t0 = (int64_t)(rest / width) * TT;

  const int cols = (int)A.x.cols, stages = (cols + KS - 1) / KS;
  const int64_t rows = A.rows - r0 < TR ? A.rows - r0 : TR, tokens = A.x.tokens - t0 < TT ? A.x.tokens - t0 : TT;
  Stream ws{reinterpret_cast<uint64_t>(A.packed) + r0 * cols, rows * cols};
  Stream xs{reinterpret_cast<uint64_t>(A.x.codes) + t0 * A.x.stride, tokens * A.x.stride};

  // Piece p of a row is at place p ^ (..): rows of 64 bytes share the banks by fours, of 128 by twos.  The 16 lanes
  // that are served at a time are 0 to 3, 12 to 15, 20 to 27 and so on, in two pieces: with row / 4 % 4 itself rows 0
  // and 4 met in a bank (67 thousand of 375 thousand cycles counted as conflicts).
  auto place = [&](int row, int piece) INLINE {
    return 16 * (piece ^ (KS == 64 ? -(row >> 2) & 3 : KS == 128 ? row >> 1 & 7 : row & 15));
  };
  // Lane l of load i brings the piece that belongs at place l % PIECES of row PER (..) + l / PIECES.  Tokens are padded
  // with zeros to a multiple of 128 columns; of a stage of 256 that goes past that (cut) the second half is left
  // out, as what follows is another token's.
  uint32_t row_off[LR], token_off[LT], past[LT];
#pragma unroll
  for (int i = 0; i < LR; ++i) {
    const int r = PER * (wave * LR + i) + lane / PIECES;
    row_off[i] = (uint32_t)r * (uint32_t)cols + place(r, lane % PIECES);
  }
#pragma unroll
  for (int i = 0; i < LT; ++i) {
    const int t = PER * (wave * LT + i) + lane / PIECES;
    token_off[i] = (uint32_t)t * (uint32_t)A.x.stride + place(t, lane % PIECES);
    past[i] = place(t, lane % PIECES) >= (int)INT8_PAD ? NOWHERE : 0u;
  }
  auto cuts = [&](int s) INLINE { return KS > INT8_PAD && s * KS + (int)INT8_PAD >= cols ? ~0u : 0u; };
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char*)lds;
  auto bring_one = [&](int i, uint32_t buf, const u32x4s& wb, const u32x4s& xb, uint32_t cut) INLINE {
    if (i < LR)
      load_to_lds(row_off[i], wb, buf + (wave * LR + i) * 1024);
    else
      load_to_lds(KS > INT8_PAD ? token_off[i - LR] | (past[i - LR] & cut) : token_off[i - LR], xb,
                  buf + RBYTES + (wave * LT + i - LR) * 1024);
  };

  // a lane's 16 codes of a block's row in a step: at piece 4 step + part
  const char* wa = lds + (wr * 16 * RB + col) * KS;
  const char* xa = lds + RBYTES + (wt * 16 * TB + col) * KS;
  int at[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) at[s] = place(col, 4 * s + part);
  i32x4 acc[RB][TB];
  i32x4 w[SETS][RB], x[SETS][TB];
  auto read_rows = [&](int buf, int step, int i) INLINE {
    w[step % SETS][i] = *reinterpret_cast<const i32x4*>(wa + buf + at[step] + i * 16 * KS);
  };
  auto read_tokens = [&](int buf, int step, int j) INLINE {
    x[step % SETS][j] = *reinterpret_cast<const i32x4*>(xa + buf + at[step] + j * 16 * KS);
  };
  // Products of a step.  Between them: each operand, when its last product is on its way, is replaced by the
  // one SETS steps on (in the next stage's buffer where that is over), a share of a stage to come is brought
  // in, and the next row block's codes are made signed (the next step's first at the end), not right before their use.
  auto products = [&]<bool FIRST>(int step, int buf, int next, uint32_t dst, const u32x4s& wb, const u32x4s& xb,
                                  uint32_t cut) INLINE {
    constexpr int N = RB * TB;
    const int set = step % SETS, from = step + SETS < STEPS ? buf : next, to = (step + SETS) % STEPS;
#pragma unroll
    for (int p = 0; p < N; ++p) {
      const int i = p / TB, j = p % TB;
      acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[set][i], x[set][j], FIRST ? i32x4{} : acc[i][j], 0, 0, 0);
      if (j == TB - 1) read_rows(from, to, i);
      if (i == RB - 1) read_tokens(from, to, j);
#pragma unroll
      for (int n = 0; n < LPW; ++n)
        if (STEPS * n * N / LPW - step * N == p) bring_one(n, dst, wb, xb, cut);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((e * TB / 4 < TB - 1 ? e * TB / 4 : TB > 1 ? TB - 2 : 0) == j) {
          if (i + 1 < RB)
            w[set][i + 1][e] ^= (int32_t)0x80808080;
          else
            w[(step + 1) % SETS][0][e] ^= (int32_t)0x80808080;
        }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

#pragma unroll
  for (int s = 0; s < (EARLY ? BUFS : BUFS - 1); ++s) {
    const u32x4s wb = ws.buffer(s < stages), xb = xs.buffer(s < stages);
#pragma unroll
    for (int i = 0; i < LPW; ++i) bring_one(i, lds0 + s * STAGE, wb, xb, cuts(s));
    ws.advance(KS), xs.advance(KS);
  }
  // While they are on their way: what the tokens' and the lane's eight rows' sums are multiplied with at the end.
  const int64_t wave_r0 = r0 + wr * WR;
  const int own = lane % (WR / 8) * 8;
  float scale[8];
  int32_t zero[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int64_t r = wave_r0 + own + e < A.rows ? wave_r0 + own + e : A.rows - 1;
    scale[e] = A.scales[r];
    zero[e] = 128 - (int)A.zeros[r];
  }
  for (int t = threadIdx.x; t < TT; t += 64 * NW) {
    const int64_t tk = t < tokens ? t0 + t : A.x.tokens - 1;
    token_scale[t] = A.x.scales[tk];
    token_sum[t] = A.x.sums[tk];
  }
  retire<0>();
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0), for the compiler to know that no scalar load is left
#pragma unroll
  for (int k = 0; k < SETS; ++k) {
#pragma unroll
    for (int i = 0; i < RB; ++i) read_rows(0, k, i);
#pragma unroll
    for (int j = 0; j < TB; ++j) read_tokens(0, k, j);
  }
  w[0][0] = signed_codes(w[0][0]);
  if constexpr (EARLY) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");

  int buf = 0;  // of the stage, in bytes
  auto stage = [&]<bool FIRST>(int s) INLINE {
    const int coming = s + (EARLY ? BUFS : BUFS - 1);
    const u32x4s wb = ws.buffer(coming < stages), xb = xs.buffer(coming < stages);
    const uint32_t cut = cuts(coming);
    const int next = buf == (BUFS - 1) * STAGE ? 0 : buf + STAGE, before = buf == 0 ? (BUFS - 1) * STAGE : buf - STAGE;
    const uint32_t free = lds0 + (EARLY ? buf : before);
    products.template operator()<FIRST>(0, buf, next, free, wb, xb, cut);
#pragma unroll
    for (int k = 1; k < STEPS; ++k) products.template operator()<false>(k, buf, next, free, wb, xb, cut);
    ws.advance(KS), xs.advance(KS);
    if constexpr (EARLY) __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the next stage's operands have been read
    retire<(EARLY ? BUFS - 2 : BUFS - 3) * LPW>();
    buf = next;
  };
  stage.template operator()<true>(0);
  for (int s = 1; s < stages; ++s) stage.template operator()<false>(s);

  // A wave's sums, 16 tokens at a time, through a part of LDS of its own to rows of Y: as they are on the way
  // in, and in a loop on the way out, a lane its eight rows of every 512 / WR-th token.  A wave's LDS accesses are done
  // in their order; the compiler, to which lanes are strangers, is held to it.
  auto in_order = [] INLINE { asm volatile("" ::: "memory"); };
  retire<0>();
  char* mine = lds + wave * 16 * LD;
  const int64_t left = A.rows - wave_r0 - own;
  const int size = A.bf16 ? 2 : 4;
  char* y0 = static_cast<char*>(A.Y) + (t0 * A.ldy + wave_r0) * size;  // the wave's first row of the tile's first token
#pragma unroll
  for (int j = 0; j < TB; ++j) {
#pragma unroll
    for (int i = 0; i < RB; ++i) *reinterpret_cast<i32x4*>(mine + col * LD + 4 * (16 * i + 4 * part)) = acc[i][j];
    in_order();
    const int first = 16 * (TB * wt + j);
#pragma unroll 1
    for (int k = lane / (WR / 8); k < 16; k += 512 / WR) {
      const int tk = first + k;
      const i32x4* sums = reinterpret_cast<const i32x4*>(mine + k * LD + 4 * own);
      const i32x4 lo = sums[0], hi = sums[1];
      if (tk >= tokens || left <= 0) continue;
      f32x8i y;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        y[e] = int8_value(e < 4 ? lo[e] : hi[e - 4], zero[e], token_sum[tk], token_scale[tk], scale[e]);
      char* to = y0 + ((int64_t)tk * A.ldy + own) * size;
      if (left < 8) {
        for (int e = 0; e < left; ++e) int8_store(to, e, y[e], A.bf16);
      } else if (A.bf16) {
        *reinterpret_cast<bf16x8e*>(to) = __builtin_convertvector(y, bf16x8);
      } else {
        reinterpret_cast<f32x4e*>(to)[0] = (f32x4e){y[0], y[1], y[2], y[3]};
        reinterpret_cast<f32x4e*>(to)[1] = (f32x4e){y[4], y[5], y[6], y[7]};
      }
    }
    in_order();
  }
}

template <int RB, int TB, int WA, int WB, int KS, int BUFS, int SETS, bool EARLY>
hipError_t launch(const Int8Gemm& a, hipStream_t stream) {
  constexpr int TR = 16 * RB * WA, TT = 16 * TB * WB;
  const uint32_t rt = (uint32_t)((a.rows + TR - 1) / TR), tt = (uint32_t)((a.x.tokens + TT - 1) / TT);
  const uint32_t grid = (rt * tt + 7) / 8 * 8;
  k_int8_tile<RB, TB, WA, WB, KS, BUFS, SETS, EARLY><<<grid, 64 * WA * WB, 0, stream>>>(a, rt, tt);
  return hipGetLastError();
}

}  // namespace

hipError_t int8_tile_launch(const Int8Gemm& a, Int8Form form, hipStream_t stream) {
  switch (form) {
    case Int8Form::T256x256: return launch<4, 8, 4, 2, 64, 4, 1, false>(a, stream);
    case Int8Form::T256x128: return launch<2, 8, 8, 1, 128, 3, 2, true>(a, stream);
    case Int8Form::T128x64: return launch<2, 4, 4, 1, 128, 3, 2, true>(a, stream);
    case Int8Form::T64x128: return launch<2, 4, 2, 2, 128, 2, 2, true>(a, stream);
    case Int8Form::T64x64: return launch<2, 2, 2, 2, 256, 3, 4, true>(a, stream);
    case Int8Form::T32x32: return launch<1, 2, 2, 1, 256, 4, 4, true>(a, stream);
    default: return launch<1, 1, 2, 1, 256, 4, 4, true>(a, stream);
  }
}

}  // namespace gptq
