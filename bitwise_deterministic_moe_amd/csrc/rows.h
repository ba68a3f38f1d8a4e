// Parameter blocks and host-side launchers of the pieces of an expert layer:
// rows sorted by expert, copied for their experts and summed back, and dropout.
#pragma once

#include "dense.h"
#include "kernels.h"

namespace moedet {

// The launchers below return hipErrorInvalidConfiguration, with nothing enqueued, for more
// than kMaxGrid workgroups.

// ---------------------------------------------------------------------- sort
constexpr int kSortMaxLocal = 1024;   // experts of a sort
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / kWave;
constexpr int kSortMaxChunks = 256;   // workgroups of a sort: one a CU
constexpr int kSortMaxHist = 16384;   // counts that each of them adds up
// Slots that one workgroup sorts in one launch; more take a launch that counts
// the experts of each chunk and one that places the slots.
constexpr int64_t kSortOne = 8192;

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
// Chunks of n slots (a function of n and local alone).
inline void sort_chunks(int64_t n, int local, int64_t* chunk, int* chunks) {
  if (n <= kSortOne) {
    *chunk = kSortOne;
    *chunks = 1;
    return;
  }
  int most = kSortMaxHist / local;
  if (most > kSortMaxChunks) most = kSortMaxChunks;
  const int64_t step = kSortThreads;
  *chunk = ((n + most - 1) / most + step - 1) / step * step;
  *chunks = (int)((n + *chunk - 1) / *chunk);
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
hipError_t launch_dropout(const DropoutParams& P, bool bf16, hipStream_t st);

}  // namespace moedet
