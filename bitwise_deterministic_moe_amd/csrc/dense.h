// Parameter blocks and host-side launchers of the dense operators (layer
// norm, linear map, gated product).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

namespace moedet {

// Activations (moe_act of the C ABI).
enum { kActNone = 0, kActRelu = 1, kActRelu2 = 2, kActSilu = 3, kActGelu = 4 };

// ------------------------------------------------------- vectors of any address
// 16-byte vectors that may start at any element: gfx950 loads and stores
// them in one instruction at any byte address.
typedef uint32_t u32_any_t __attribute__((aligned(2)));
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any_t __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));

template <typename T>
struct Vec;   // the 16-byte vector of a storage type
template <>
struct Vec<uint16_t> {
  static constexpr int N = 8;
  typedef u32x4_t raw;
  // elements [0, n) of p, n >= 1; the others read as zero
  DEV static raw load(const uint16_t* p, int n) {
    if (n >= N) return *(const u32x4_any_t*)p;
    raw r = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
      if (i < n) r[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    return r;
  }
  DEV static void get(const raw& r, float* v) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      v[2 * w] = __uint_as_float(r[w] << 16);
      v[2 * w + 1] = __uint_as_float(r[w] & 0xffff0000u);
    }
  }
  DEV static void store(uint16_t* p, const float* v, int n) {
    const u32x4_t r = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    if (n >= N) {
      *(u32x4_any_t*)p = r;
      return;
    }
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
      if (i < n) p[i] = (uint16_t)(r[i >> 1] >> (16 * (i & 1)));
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  typedef f32x4_t raw;
  DEV static raw load(const float* p, int n) {
    if (n >= N) return *(const f32x4_any_t*)p;
    raw r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
      if (i < n) r[i] = p[i];
    return r;
  }
  DEV static void get(const raw& r, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = r[i];
  }
  DEV static void store(float* p, const float* v, int n) {
    if (n >= N) {
      *(f32x4_any_t*)p = f32x4_t{v[0], v[1], v[2], v[3]};
      return;
    }
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
      if (i < n) p[i] = v[i];
  }
};

// ---------------------------------------------------------------- layer norm
constexpr int64_t kNormMaxCols = 16384;
constexpr int kNormBlocks = 512;  // most row blocks of the weight gradient's partial sums

struct NormParams {
  const void* x;
  const void* weight;   // or null: 1
  const void* bias;     // or null: 0
  const void* dy;
  const void* add;      // or null
  int64_t rows, ldx, lddy, ldadd;
  int cols;
  float eps;
  void* y;              // forward y, backward dx
  float* mean;
  float* rstd;
  float* part;          // backward: [blocks][2][cols] partial sums of dweight and dbias
  int blocks;
  uint64_t seed;
};

// Row blocks of the backward for a problem (from its sizes and type alone).
int norm_bwd_blocks(int64_t rows, int64_t cols, bool bf16);
hipError_t launch_norm_fwd(const NormParams& P, bool bf16, hipStream_t st);
hipError_t launch_norm_bwd(const NormParams& P, bool bf16, hipStream_t st);
// out[c] = sum over b ascending, in fixed phases, of part[b * stride + c], c <
// cols; out2 the same of the next cols columns.  Either may be null.
hipError_t launch_block_sums(const float* part, int blocks, int64_t stride, int cols, void* out, void* out2,
                             hipStream_t st);

// The column sums of one workgroup of 256 threads: columns 16 block .. 16
// block + 15 in 16 phases; phase p adds blocks [p B / 16, (p + 1) B / 16)
// ascending, then the phases are added in order.  Nothing is written where out is null.
DEV void block_sum16(const float* part, int blocks, int64_t stride, int cols, uint32_t block, void* out, bool out_bf16) {
  __shared__ float s[16][17];
  const int x = threadIdx.x & 15, p = threadIdx.x >> 4;
  const int c = (int)block * 16 + x;
  const int b0 = p * blocks / 16, b1 = (p + 1) * blocks / 16;
  float v = 0.f;
  if (c < cols) {
    const float* q = part + (int64_t)b0 * stride + c;
#pragma unroll 8
    for (int b = b0; b < b1; ++b, q += stride) v = v + *q;
  }
  s[p][x] = v;
  __syncthreads();
  if (p == 0 && c < cols && out) {
    v = s[0][x];
#pragma unroll
    for (int i = 1; i < 16; ++i) v = v + s[i][x];
    if (out_bf16)
      ((uint16_t*)out)[c] = (uint16_t)f32_to_bf16(v);
    else
      ((float*)out)[c] = v;
  }
}

// ------------------------------------------------------------ matrix operators
// One matrix product of a dense operator,
//   C[m, n] = sum_k A[m, k] B[n, k]
// in one of four forms (kForm*), split into S chunks of the contraction when
// S > 1: each chunk then stores its float32 partial and launch_dense_finish
// adds them in chunk order and runs the epilogue.
enum {
  kFormLinear = 0,  // A = x [M][K], B = w [K][N]: z = C + bias, y = act(z) + residual
  kFormGlu = 1,     // A = x, B = wg and wu [K][N]: g, u and act(g) u
  kFormDx = 2,      // A = dz [M][nseg K], B = nseg matrices [N][K]: C + add
  kFormDw = 3       // A = x [K][M], B = dz [K][nseg N]: nseg matrices C
};

struct DenseParams {
  int64_t M;          // rows of C
  int N;              // columns of C (of one matrix)
  int64_t K;          // contraction (of one segment)
  int nseg;           // kFormDx: K segments; kFormDw: matrices C
  const void* a;
  int64_t lda;
  int64_t seg;        // kFormDx: elements between the K segments of a; kFormDw: between the column segments of b
  const void* b[2];
  int64_t ldb;
  int S;              // chunks of the contraction
  float* part;        // [S][M][part_ld] when S > 1
  int64_t part_ld;
  int part_seg;       // columns between the two matrices in a partial row
  // epilogue
  const void* bias;   // or null
  const void* add;    // residual / dx_add, or null
  int64_t ldadd;
  void* c[2];         // y, a, dx or the weight gradients
  int64_t ldc;
  void* z[2];         // z or g and u; null: not stored
  int64_t ldz;
  bool z_f32;         // float32 z whatever the storage type
  int act;
  bool c_f32;         // kFormDw: float32 c whatever the storage type
  uint64_t seed;
};

// Rows of the few-row kernels (weights streamed once), by the number of matrices and
// whether tiles would have to copy the weights first.  Against the tiles, us (kernels
// alone, in a graph):
//   bf16, one matrix  32 rows: 2048^2 9.7 and 9.4, 2048 x 8192 10.6 and 12.5, 1024^2 5.3 and
//                     6.5, 4096^2 16.5 and 12.3; 64 rows: 12.7 and 10.7, 13.2 and 12.5, 7.0 and
//                     6.6, 21.7 and 13.0
//   bf16, gated       48 rows: 15.1 and 14.1, 16.5 and 20.0, 7.1 and 9.0, 28.4 and 19.9
//   bf16, weights to copy, 64 rows: one matrix 13.7 and 18.0, 15.0 and 25.1, 7.7 and 10.2,
//                     23.8 and 24.9; gated 17.7 and 21.1, 23.6 and 45.1, 10.7 and 13.8, 33.6 and 45.9
//   float32           32 rows: one matrix 13.4 and 14.1, 26.2 and 27.1, 8.7 and 9.2, 24.2 and
//                     27.0; gated 17.6 and 21.9, 54.1 and 46.8, 13.5 and 15.1, 49.1 and 50.8
constexpr int few_rows(bool bf16, int nm, bool copies) { return !bf16 ? 32 : copies ? 64 : nm == 2 ? 48 : 32; }
// Rows from which these kernels read a copy of an x whose bf16 rows do not all start on
// 16 bytes: every workgroup reads all of x, and its loads then straddle lines.  In
// place and with the copy, us, one matrix: 12 rows 4096^2 17.4 and 15.6, 2048 x 8192 10.9 and
// 11.7; 16 rows 19.3 and 16.1, 11.7 and 11.8; 32 rows 31.0 and 19.2, 18.0 and 13.5; weights to copy
// too, 64 rows 57.1 and 26.6, 30.8 and 18.0.
constexpr int kFewCopyRows = 13;

// tile: as in dense_shape
hipError_t launch_dense_gemm(const DenseParams& P, int form, bool bf16, int tile, hipStream_t st);
hipError_t launch_dense_few(const DenseParams& P, int form, bool bf16, hipStream_t st);
hipError_t launch_dense_finish(const DenseParams& P, int form, bool bf16, hipStream_t st);
// Rows, columns (of one matrix) and K slice of a tile
struct DenseShape {
  int bm, bn, bk;
};
constexpr int kDenseBf16Tiles = 4, kDenseF32Tiles = 2;
DenseShape dense_shape(int form, bool bf16, int tile);
// Variants of a tile: the 64-row bf16 tile's short ring (at most two slices a
// workgroup), and the float32 tiles' loads of four columns (each operand's
// contiguous direction is whole groups of four).
bool dense_short(const DenseParams& P, int form);
bool dense_v4(const DenseParams& P, int form);

// bf16 matrices [rows][cols] (row distance ld) into [rows][ldo], zeros past cols
struct DensePackParams {
  const void* in[3];
  void* out[3];
  int64_t rows[3], ld[3], ldo[3], first[4];   // first workgroup of each
  int cols[3];
  int n;
  void add(const void* src, int64_t r, int c, int64_t l, void* dst, int64_t lo);
};
hipError_t launch_dense_pack(const DensePackParams& P, hipStream_t st);
// Gradients of the pre-activations, elementwise, with the column sums of dz
// over row blocks.
struct DenseEwParams {
  int64_t rows;
  int cols;
  const void* dy;     // or da
  int64_t lddy;
  const void* z[2];   // z, or g and u
  int64_t ldz;
  bool z_f32;
  int act;
  void* out[2];       // dz, or dg and du; null: not stored
  int64_t ldo;
  int pad;            // columns up to which an output row is written (zeros past cols)
  float* part;        // [blocks][cols] column sums of dz, or null
  int blocks;
  uint64_t seed;
};
int dense_ew_blocks(int64_t rows, int cols, bool bf16, bool sums);
// K: operands to copy in the same launch (K.n may be 0)
hipError_t launch_dense_ew(const DenseEwParams& P, const DensePackParams& K, bool glu, bool bf16, hipStream_t st);
// What a backward call joins at its end: chunks of dx and dw (where S > 1) and
// the bias gradient's column sums (where db is set).
struct DenseJoin {
  DenseParams dx, dw;
  uint32_t nx, nw;     // workgroups of each
  const float* sums;   // [blocks][cols]
  int blocks, cols;
  void* db;
  bool db_bf16;
};
hipError_t launch_dense_join(const DenseParams& dx, const DenseParams& dw, const float* sums, int blocks, int cols,
                             void* db, bool db_bf16, bool bf16, hipStream_t st);
hipError_t launch_dense_zero(void* p, int64_t n16, hipStream_t st);   // n16 16-bit words

}  // namespace moedet
