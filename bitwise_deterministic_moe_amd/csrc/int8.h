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
int64_t int8_quantize_grid(int64_t rows, int cols16, bool bf16);
hipError_t launch_int8_quantize(const Int8QuantParams& P, bool bf16, hipStream_t st);

struct Int8QuantTParams {
  const void* w;            // [batch][rows][cols]
  int64_t batch;
  int rows, cols, rows16;
  int8_t* codes;            // [batch][cols][rows16]
  float* scales;            // [batch][cols]
  uint64_t seed;
};
int64_t int8_quantize_t_grid(int64_t batch, int cols);   // workgroups of 512 threads
hipError_t launch_int8_quantize_t(const Int8QuantTParams& P, bool bf16, hipStream_t st);

// Rows that the few-row kernel quantises itself, into LDS: of one matrix up to this many (every
// workgroup quantises all of them), of experts a workgroup's up to 16; their codes fit
// kInt8FusedBytes, which leaves room for four workgroups a CU.
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
  int bm, bn;
};
constexpr int kInt8Slice = 128;   // codes of a tile's K slice
// Tiles: 256 x 256 (one workgroup a CU), 128 x 128 (two), 128 x 64 with a ring of three slots
// (two) and of two (three), 64 x 64 with two (five) and with four (two).  The deeper rings
// are for products with few workgroups a CU.  Us without activation (rows x columns x
// K; experts with the squared ReLU), in this order:
//   8192 x 8192 x 8192    450  551  703  690  845  864
//   4096 x 8192 x 2048     73   84  100   98  119  127
//   8192 x 2048 x 1024     23   26   33   31   34   41
//   4096 x 2048 x 8192     79   71   84   93  104  106
//   1000 x 8192 x 2048     33   23   28   29   31   34
//   2048 x 2048 x 2048     28   16   16   15   17   18
//   300 x 4096 x 4096      44   24   14   21   19   16
//   512 x 2048 x 2048      27   15    9   13   11    7
//   64 x 2048 x 8192       75   42   21   36   32   15
//   8 experts of 325..2456 rows, 2048 x 1024         44   33   37   34   41   46
//   64 experts of 2400 rows, 2048 x 2048 (268 MB)    71   58   68   66   63   59
//   64 experts of 800 rows                           69   56   63   62   53   58
constexpr int kInt8Tiles = 6;
constexpr Int8Shape kInt8Shapes[kInt8Tiles] = {{256, 256}, {128, 128}, {128, 64}, {128, 64}, {64, 64}, {64, 64}};
hipError_t launch_int8_tiles(const Int8Params& P, bool bf16, int tile, hipStream_t st);
// ks: waves that share a contraction, 1 or 4
hipError_t launch_int8_few(const Int8Params& P, bool bf16, int ks, hipStream_t st);

}  // namespace moedet
