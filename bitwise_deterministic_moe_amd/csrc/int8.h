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

// y[m, n] = act(sa[m] sb[n] sum_k a[m, k] b[n, k] + bias[n]) + add[m, n], in
// groups of rows with matrices of their own when offsets is set.
struct Int8Params {
  // M rows, N, K (bytes of a code row, a multiple of 16), bias, add, ldadd, c[0], ldc,
  // act, seed; the operands' fields are unread
  DenseParams d;
  const int8_t* a;
  int64_t lda;
  const float* sa;
  const int8_t* b;          // [groups][N][K]
  const float* sb;          // [groups][N]
  const int32_t* offsets;   // [groups + 1] first rows, or null for one group of all rows
  int groups;
};
enum { kInt8Tiles = 4 };    // 256x256, 128x256, 128x128, 64x64 (dense_shape's bf16 numbers)
hipError_t launch_int8_tiles(const Int8Params& P, bool bf16, int tile, hipStream_t st);
// mt: blocks of 16 rows a workgroup multiplies the weights it streams with (1 or 2)
hipError_t launch_int8_few(const Int8Params& P, bool bf16, int mt, hipStream_t st);

}  // namespace moedet
