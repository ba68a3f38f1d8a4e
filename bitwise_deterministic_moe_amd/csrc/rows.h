// Parameter blocks and host-side launchers of the pieces of an expert layer:
// rows sorted by expert, copied for their experts and summed back, and dropout.
#pragma once

#include <cmath>

#include "dense.h"
#include "kernels.h"

namespace moedet {

// ---------------------------------------------------------------------- sort
constexpr int kSortMaxLocal = 1024;   // experts of a sort
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / kWave;
constexpr int kSortMaxChunks = 256;   // workgroups of a sort: one a CU
// Slots that one workgroup sorts in one launch; more take a launch that counts
// the experts of each chunk and one that places the slots (4096 slots of 8, 64 and 512 experts
// 6.6, 7.2 and 8.3 us in one, 6.9, 7.2 and 8.4 in two; 8192: 9.2, 10.4 and 12.2, and 6.9, 7.7
// and 8.5).
constexpr int64_t kSortOne = 4096;

struct SortParams {
  const void* idx;       // [n] expert numbers, int32 or int64
  bool wide;             // int64
  int64_t n;
  int begin, local;
  int64_t chunk;         // slots of a workgroup, a multiple of 64 kSortWaves
  int chunks;
  int32_t* hist;         // [chunks][local], when chunks > 1
  int32_t* slot_row;
  int32_t* offsets;
  int32_t* row_src;      // or null
  uint64_t seed;
};
// Chunks of n slots (a function of n and local alone).  A workgroup walks its chunk, n /
// chunks slots, and adds up chunks * local counts: the sum is least near the root of
// n / local, times 3.2 as measured.  Us with about 30, 60, 120 and 240 chunks: 90112 slots of 512 experts
// 11.5 and (88) 12.4, of 1024 13.7 and (88) 17.1; 360448 of 512 20.4, 16.4, 16.4, of 1024 23.4,
// 20.5, 22.9; 1441792 of 512 58, 36, 27, 27, of 1024 63, 41, 35, 39, of 64 50, 29, 19, 14.
inline void sort_chunks(int64_t n, int local, int64_t* chunk, int* chunks) {
  const int64_t step = kSortThreads;
  int64_t most = n <= kSortOne ? 1 : (int64_t)std::sqrt(10.0 * (double)n / local);
  if (most < 1) most = 1;
  if (most > kSortMaxChunks) most = kSortMaxChunks;
  *chunk = ((n + most - 1) / most + step - 1) / step * step;
  if (*chunk < step) *chunk = step;
  *chunks = n > *chunk ? (int)((n + *chunk - 1) / *chunk) : 1;
}
hipError_t launch_sort(const SortParams& P, hipStream_t st);

// ------------------------------------------------------------ rows of experts
struct RowsParams {
  int64_t tokens;
  int k;
  int cols;
  int64_t nrows;           // rows of the expert-sorted matrices: slots outside [0, nrows) have no row
  const int32_t* slot_row; // [tokens k]
  const float* prob;       // [tokens k] or null: 1
  const void* x;           // permute: [tokens][ldx]; unpermute backward: dy
  int64_t ldx;
  const void* rows;        // [nrows][cols]
  const void* add;         // [tokens][ldadd] or null
  int64_t ldadd;
  void* out;               // [tokens][cols], or rows [nrows][cols]
  float* dprob;            // [tokens k] or null
  uint64_t seed;
};
// Workgroups of a call (*_grid), from its sizes alone: the entry points refuse more than kMaxGrid.
int64_t permute_grid(const RowsParams& P, int elem_bytes);
int64_t unpermute_grid(const RowsParams& P, bool bf16);
int64_t unpermute_bwd_grid(const RowsParams& P, bool bf16);
hipError_t launch_permute(const RowsParams& P, int elem_bytes, hipStream_t st);
hipError_t launch_unpermute(const RowsParams& P, bool bf16, hipStream_t st);
hipError_t launch_unpermute_bwd(const RowsParams& P, bool bf16, hipStream_t st);

// -------------------------------------------------------------------- dropout
struct DropoutParams {
  int64_t rows;
  int cols;
  const void* x;
  int64_t ldx;
  const void* add;         // or null
  int64_t ldadd;
  void* y;                 // contiguous
  const uint64_t* rng;     // {key, first counter}
  uint32_t limit;          // a word below it drops its element
  bool all;                // every element is dropped (a limit of 2^32)
  float scale;
  uint64_t seed;
};
int64_t dropout_grid(const DropoutParams& P, bool bf16);
hipError_t launch_dropout(const DropoutParams& P, bool bf16, hipStream_t st);

}  // namespace moedet
