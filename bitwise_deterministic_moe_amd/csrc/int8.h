// Parameter blocks and host-side launchers of the products in 8-bit integers.
#pragma once

#include "dense.h"
#include "kernels.h"

namespace moedet {

// Rows of numbers this small are quantised to zeros: their scale's reciprocal would
// leave float32's range.
constexpr float kInt8Tiny = 0x1p-100f;
// Longest contraction: 2^17 products of at most 127^2 stay below 2^31.
constexpr int kInt8MaxK = 1 << 17;
constexpr int kInt8MaxGroups = 1024;

struct Int8QuantParams {
  const void* x;            // [rows][ldx]
  int64_t rows, ldx;
  int cols, cols16;         // columns, and columns of the codes (a multiple of 16; zeros past cols)
  const int32_t* limit;     // or null: only rows below *limit are read and written
  int8_t* codes;            // [rows][cols16]
  float* scales;            // [rows]
  uint64_t seed;
};
hipError_t launch_int8_quantize(const Int8QuantParams& P, bool bf16, hipStream_t st);

struct Int8QuantTParams {
  const void* w;            // [batch][rows][cols]
  int64_t batch;
  int rows, cols, rows16;
  int8_t* codes;            // [batch][cols][rows16]
  float* scales;            // [batch][cols]
  uint64_t seed;
};
hipError_t launch_int8_quantize_t(const Int8QuantTParams& P, bool bf16, hipStream_t st);

// Few rows that the product itself quantises, into LDS.
constexpr int kInt8FusedRows = 4, kInt8FusedBytes = 32768;

// y[m, n] = act(sa[m] sb[n] sum_k a[m, k] b[n, k] + bias[n]) + add[m, n], in
// groups of rows with matrices of their own when offsets is set.
struct Int8Params {
  // M rows, N, K (bytes of a code row, a multiple of 16), S (chunks of the contraction, one
  // group only), bias, add, ldadd, c[0], ldc, act, seed; the operands' fields are unread
  DenseParams d;
  const int8_t* a;
  int64_t lda;
  const float* sa;
  const void* x;            // few rows, instead of a and sa: x [M][ldx] of y's type, xcols columns
  int64_t ldx;
  int xcols;
  const int8_t* b;          // [groups][N][K]
  const float* sb;          // [groups][N]
  const int32_t* offsets;   // [groups + 1] first rows, or null for one group of all rows
  int groups;
  int32_t* part;            // S > 1: [S][M][part_ld] sums
  int64_t part_ld;
};
struct Int8Shape {
  int bm, bn, bk;           // bk: codes of a K slice
};
// Tiles: 256 x 256 (one workgroup a CU), 128 x 128 (two), 128 x 64 (three), 64 x 64 (five), and 64
// x 64 with a deeper ring (two) for products with a workgroup a CU or less.  Us
// without activation (rows x columns x K), in this order:
//   4096 x 8192 x 2048     92   96  111  128  144
//   8192 x 2048 x 1024     29   33   35   39   48
//   4096 x 2048 x 8192     87   79  111  122  128
//   1000 x 8192 x 2048     34   26   34   37   40
//   1024 x 4096 x 4096     47   35   29   35   36
//   300 x 4096 x 4096      45   32   25   22   19
//   64 x 2048 x 8192       66   55   42   36   20
//   8 experts of 325..2456 rows, 2048 x 1024         51   41   39   44   55
//   64 experts of 2400 rows, 2048 x 2048 (268 MB)    74   80   74   72   76
//   64 experts of 800 rows                           68   60   66   55   60
constexpr int kInt8Tiles = 5;
constexpr Int8Shape kInt8Shapes[kInt8Tiles] = {{256, 256, 64}, {128, 128, 128}, {128, 64, 128}, {64, 64, 128}, {64, 64, 128}};
hipError_t launch_int8_tiles(const Int8Params& P, bool bf16, int tile, hipStream_t st);
// ks: waves that share a contraction (1, 2 or 4)
hipError_t launch_int8_few(const Int8Params& P, bool bf16, int ks, hipStream_t st);

}  // namespace moedet
