// Slots sorted by expert (a stable counting sort), integer-exact.
//
// Slot i of n holds an expert number; the slots whose expert is one of the
// `local` ones are numbered expert by expert, inside an expert by ascending
// slot.  row(i) = offsets[e] + (slots j < i of the same expert).
//
//  sort_count_kernel  histogram of every chunk of slots in LDS (integer
//                     atomics: exact in any order).
//  sort_place_kernel  a workgroup per chunk adds up the histograms itself (all of them
//                     for the experts' offsets, those of earlier chunks for
//                     its own bases), which saves a launch with one workgroup at work;
//                     its 16 waves take consecutive runs of the chunk, count
//                     them, and then walk them 64 slots at a time: a
//                     lane's rank among equal experts comes from ballots.
//                     With one chunk it is the whole sort.
//
// Bound by latency: 22 slots of 512 experts 4.9 us in one launch, 90112 slots 11.3 in two
// (1.1 MB), 1441792 slots 26 (most of it the ballots, one a bit of the expert's number), again and
// again in a graph; 13.3 for the 90112 among other calls, whose indices come from memory.
#include "common.h"
#include "rows.h"

namespace moedet {

namespace {

// The local expert of slot i, -1 if it is none of them or i is past the end.
template <bool WIDE>
DEV int local_expert(const SortParams& P, int64_t i, int64_t end) {
  if (i >= end) return -1;
  const int64_t e = (WIDE ? ((const int64_t*)P.idx)[i] : (int64_t)((const int32_t*)P.idx)[i]);
  // e - begin in unsigned arithmetic: numbers below begin are past `local` too
  const uint64_t le = (uint64_t)e - (uint64_t)P.begin;
  return le < (uint64_t)P.local ? (int)le : -1;
}

}  // namespace

template <bool WIDE>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortParams P) {
  __shared__ int s_hist[kSortMaxLocal];
  const int tid = threadIdx.x;
  const int64_t c = blockIdx.x;
  if (P.seed) shuffle_delay(P.seed, c);
  for (int e = tid; e < P.local; e += kSortThreads) s_hist[e] = 0;
  __syncthreads();
  const int64_t end = min((c + 1) * P.chunk, P.n);
  for (int64_t i = c * P.chunk + tid; i < end; i += kSortThreads) {
    const int e = local_expert<WIDE>(P, i, end);
    if (e >= 0) atomicAdd(&s_hist[e], 1);
  }
  __syncthreads();
  for (int e = tid; e < P.local; e += kSortThreads) P.hist[c * P.local + e] = s_hist[e];
}

template <bool WIDE>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortParams P) {
  __shared__ int s_cnt[kSortWaves * kSortMaxLocal];   // [wave][expert]: counts, then next rows
  __shared__ int s_tot[kSortMaxLocal], s_before[kSortMaxLocal];
  __shared__ int s_off[kSortMaxLocal + 1];
  __shared__ int s_tmp[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int El = P.local;
  const int64_t c = blockIdx.x;
  if (P.seed) shuffle_delay(P.seed, c);
  for (int i = tid; i < kSortWaves * El; i += kSortThreads) s_cnt[i] = 0;
  for (int e = tid; e < El; e += kSortThreads) s_tot[e] = s_before[e] = 0;
  __syncthreads();
  // this wave's run of the chunk
  const int64_t run = P.chunk / kSortWaves;
  const int64_t i0 = c * P.chunk + w * run, end = min(i0 + run, P.n);
  int* cnt = s_cnt + w * El;
  for (int64_t i = i0; i < end; i += 64) {
    const int e = local_expert<WIDE>(P, i + lane, end);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  if (P.chunks > 1) {
    // thread (part, e): chunks part, part + parts, ...
    int span = 1;
    while (span < El) span <<= 1;
    const int e = tid & (span - 1), part = tid / span, parts = kSortThreads / span;
    if (e < El) {
      int tot = 0, before = 0;
      // loads in batches without branches: past the end they repeat the last one
      constexpr int B = 8;
      for (int q0 = part; q0 < P.chunks; q0 += B * parts) {
        int h[B];
#pragma unroll
        for (int i = 0; i < B; ++i) h[i] = P.hist[min(q0 + i * parts, P.chunks - 1) * El + e];
#pragma unroll
        for (int i = 0; i < B; ++i) {
          const int q = q0 + i * parts;
          tot += q < P.chunks ? h[i] : 0;
          before += q < c ? h[i] : 0;
        }
      }
      atomicAdd(&s_tot[e], tot);
      atomicAdd(&s_before[e], before);
    }
  }
  __syncthreads();
  if (P.chunks == 1) {
    for (int e = tid; e < El; e += kSortThreads) {
      int tot = 0;
#pragma unroll
      for (int v = 0; v < kSortWaves; ++v) tot += s_cnt[v * El + e];
      s_tot[e] = tot;
    }
    __syncthreads();
  }
  block_exclusive_scan<kSortThreads>(s_off, s_tmp, El, [&](int e) { return s_tot[e]; });
  if (c == 0)
    for (int e = tid; e <= El; e += kSortThreads) P.offsets[e] = s_off[e];
  for (int e = tid; e < El; e += kSortThreads) {
    int row = s_off[e] + s_before[e];
#pragma unroll
    for (int v = 0; v < kSortWaves; ++v) {
      const int n = s_cnt[v * El + e];
      s_cnt[v * El + e] = row;
      row += n;
    }
  }
  __syncthreads();
  const uint64_t lt = (1ull << lane) - 1ull;
  int bits = 0;
  while ((1 << bits) < El) ++bits;
  for (int64_t i = i0; i < end; i += 64) {
    const int e = local_expert<WIDE>(P, i + lane, end);
    uint64_t match = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const bool my = (e >> b) & 1;
      const uint64_t m = __ballot(my);
      match &= my ? m : ~m;
    }
    int row = -1;
    if (e >= 0) row = cnt[e] + __popcll(match & lt);
    // the wave's next rows: written after every lane has read them
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (e >= 0 && (match & lt) == 0) cnt[e] = row + __popcll(match);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (i + lane < end) P.slot_row[i + lane] = row;
    if (P.row_src && e >= 0) P.row_src[row] = (int32_t)(i + lane);
  }
}

hipError_t launch_sort(const SortParams& P, hipStream_t st) {
  if (P.chunks > 1) {
    if (P.wide)
      sort_count_kernel<true><<<P.chunks, kSortThreads, 0, st>>>(P);
    else
      sort_count_kernel<false><<<P.chunks, kSortThreads, 0, st>>>(P);
  }
  if (P.wide)
    sort_place_kernel<true><<<P.chunks, kSortThreads, 0, st>>>(P);
  else
    sort_place_kernel<false><<<P.chunks, kSortThreads, 0, st>>>(P);
  return hipGetLastError();
}

}  // namespace moedet
