// Which kernel takes a call of the 8-bit product: plain C++, the same on the host with any compiler.
#pragma once

#include <stdint.h>

namespace gptq {

// k_int8_tile.hip's tiles of rows x tokens.
enum class Int8Form { T256x256, T256x128, T128x64, T64x128, T64x64, T32x32, T32x16 };

// A form's time (us) is estimated as INT8_START + for every round of the workgroups that the chip holds at a time (256
// CUs, `held` each): `round` + stages * t, where a stage takes t0 while the round fills at most `knee` of the
// places and t1 when it fills all.  The numbers fit what was measured from 300 x 512 x 512 to 8192^3; tokens x
// columns x rows, us by form (the one that the rule takes last):
//   4096 x 4096 x 11008  256x128 190, 256x256 177
//   4096 x 11008 x 4096  256x128 166, 256x256 160
//   2048 x 4096 x 4096   256x256 48, 128x64 45, 256x128 35
//   1000 x 4096 x 4096   256x128 28, 64x128 25.4, 128x64 24.8
//   777 x 2052 x 5001    256x128 21.4, 128x64 24.6, 64x128 20
//   500 x 4096 x 4096    64x64 20, 256x128 27, 128x64 15
//   256 x 4096 x 4096    128x64 14, 32x32 17, 64x64 11
//   128 x 4096 x 4096    128x64 15, 64x64 10.3, 32x32 9.6
//   64 x 4096 x 4096     64x64 9.9, 32x32 8.0
//   1000 x 1000 x 1000   128x64 7.9, 32x32 10, 64x64 6.4
//   61 x 11008 x 4096    64x64 20, 32x16 17, 32x32 15
struct Int8Tiles {
  Int8Form form;
  int rows, tokens, cols, held;
  float round, t0, t1, knee;
};
constexpr Int8Tiles INT8_FORMS[] = {
    {Int8Form::T256x256, 256, 256, 64, 1, 6.0f, 0.55f, 0.87f, 0.0f},
    {Int8Form::T256x128, 256, 128, 128, 1, 4.0f, 0.62f, 0.92f, 0.0f},
    {Int8Form::T128x64, 128, 64, 128, 2, 4.0f, 0.28f, 0.58f, 0.5f},
    {Int8Form::T64x128, 64, 128, 128, 3, 3.5f, 0.50f, 0.92f, 0.33f},
    {Int8Form::T64x64, 64, 64, 256, 1, 3.5f, 0.36f, 0.39f, 0.0f},
    {Int8Form::T32x32, 32, 32, 256, 2, 2.5f, 0.21f, 0.32f, 0.5f},
    {Int8Form::T32x16, 32, 16, 256, 3, 2.0f, 0.16f, 0.36f, 0.33f},
};
constexpr float INT8_START = 2.5f;
constexpr int INT8_CUS = 256;

inline int64_t int8_tiles_of(const Int8Tiles& f, int64_t rows, int64_t tokens) {
  return (rows + f.rows - 1) / f.rows * ((tokens + f.tokens - 1) / f.tokens);
}

inline float int8_estimate(const Int8Tiles& f, int64_t rows, int64_t cols, int64_t tokens) {
  const int64_t tiles = int8_tiles_of(f, rows, tokens), places = (int64_t)INT8_CUS * f.held, full = tiles / places;
  const float stages = (float)((cols + f.cols - 1) / f.cols);
  const float filled = (float)(tiles % places) / (float)places;
  const float over = filled > f.knee ? (filled - f.knee) / (1.0f - f.knee) : 0.0f;
  const float last = filled > 0.0f ? f.round + stages * (f.t0 + (f.t1 - f.t0) * over) : 0.0f;
  return INT8_START + (float)full * (f.round + stages * f.t1) + last;
}

inline const Int8Tiles& int8_best(int64_t rows, int64_t cols, int64_t tokens) {
  const Int8Tiles* b = &INT8_FORMS[0];
  for (const Int8Tiles& f : INT8_FORMS)
    if (int8_estimate(f, rows, cols, tokens) < int8_estimate(*b, rows, cols, tokens)) b = &f;
  return *b;
}

// Up to two workgroups of k_int8_rows.hip a CU.  Its time and that of tiles of 32 x 16, us, layers in turn that
// together fill no cache:
//   rows              2048          4096          6144          8192         11008         16384
//   1 token
//     1024 columns     3.1 / 4.3     3.2 / 4.5     4.6 / 5.0     4.7 / 5.5     5.9 / 6.8     7.1 / 7.4
//     4096             5.6 / 7.7     6.3 / 8.2     9.0 / 9.0    10.0 / 10.0   13.6 / 13.4   17.0 / 20.2
//     11008           10.0 / 14.7   14.2 / 16.9   20.6 / 22.7   24.2 / 26.8   34.1 / 34.3   46.6 / 45.8
//   16 tokens
//     1024             3.5 / 4.3     3.6 / 4.5     5.2 / 5.2     5.3 / 5.5     6.9 / 6.9     8.4 / 7.4
//     4096             6.5 / 7.9     7.0 / 8.5    11.2 / 9.1    11.8 / 10.1   15.8 / 14.1   20.9 / 19.5
//     11008           12.9 / 14.9   15.4 / 17.1   25.9 / 20.7   27.0 / 24.2   38.2 / 33.1   51.2 / 42.6
// So for one token the two are equal from 8192 rows on, give or take the columns, and with 16 tokens tiles take over
// between 4096 and 6144 rows: the cut goes by one token, and costs 16 up to a quarter between 6144 and 8192 rows.
inline bool int8_by_rows(int64_t rows, int64_t tokens) { return tokens <= 16 && rows <= 8192; }

}  // namespace gptq
