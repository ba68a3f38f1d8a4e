// Rows copied for their experts and summed back, forward and backward.
//
//  permute        rows[slot_row[t, j]] = x[t]
//  unpermute      y[t] = sum over j ascending of p[t, j] rows[slot_row[t, j]],
//                 float32 from 0, then add[t], rounded once.  Without p it is
//                 permute's backward.
//  unpermute_bwd  drows[slot_row[t, j]] = p[t, j] dy[t], rounded once;
//                 dprob[t, j] = <dy[t], rows[slot_row[t, j]]> in float32, each
//                 lane over its columns ascending, then a fixed tree over the lanes.
//
// All three go by token, not by row: a token's row is read once and stays in
// registers or the L1 for its k slots, and no row -> slot table is read.  All are
// bound by HBM.  Each output element is written by one thread: no atomics.
// A slot whose row is outside [0, nrows) has none: it is not read or written.
#include "rows.h"

namespace moedet {

namespace {

typedef uint32_t u32x4_b_t __attribute__((ext_vector_type(4), aligned(1)));

// A workgroup of 256 threads takes 256 / L tokens, L threads each (a power of two
// up to 256, the row's 16-byte vectors where they are fewer).
inline int row_threads(int64_t vecs) {
  int L = 8;
  while (L < 256 && L < vecs) L <<= 1;
  return L;
}

struct Place {
  int64_t t;      // token
  int v;          // first vector of this thread
  int j0, j1;     // slots
};
// L, the threads of a token, and S, the parts that its slots are split into
DEV bool place(const RowsParams& P, int L, int S, Place& p) {
  const int per = 256 / L;
  const int64_t groups = (P.tokens + per - 1) / per;
  const int64_t u = map_unit(blockIdx.x, groups * S, P.seed);
  if (u < 0) return false;
  // several parts only where they are few (launch_permute)
  const int64_t g = S == 1 ? u : (int64_t)((uint32_t)u / (uint32_t)S);
  const int s = (int)(u - g * S);
  p.t = g * per + threadIdx.x / L;
  p.v = threadIdx.x & (L - 1);
  p.j0 = (int)((int64_t)s * P.k / S);
  p.j1 = (int)((int64_t)(s + 1) * P.k / S);
  return p.t < P.tokens;
}

}  // namespace

// WHOLE: L >= 64, so a wave has one token and its slots' rows are scalars.
template <bool WHOLE>
__global__ __launch_bounds__(256) void permute_kernel(RowsParams P, int es, int L, int S) {
  Place p;
  if (!place(P, L, S, p)) return;
  const int64_t t = WHOLE ? (int64_t)__builtin_amdgcn_readfirstlane((int)p.t) : p.t;
  const int64_t len = (int64_t)P.cols * es;
  const int vecs = (int)((len + 15) / 16);
  const char* src = (const char*)P.x + t * P.ldx * es;
  const int32_t* sr = P.slot_row + t * P.k;
  for (int v = p.v; v < vecs; v += L) {
    const int64_t at = (int64_t)v * 16;
    const int n = (int)(len - at < 16 ? len - at : 16);
    u32x4_t x = {0u, 0u, 0u, 0u};
    if (n == 16) x = *(const u32x4_b_t*)(src + at);
    for (int j = p.j0; j < p.j1; ++j) {
      const int32_t r = sr[j];
      if (r < 0 || r >= P.nrows) continue;
      char* dst = (char*)P.out + (int64_t)r * len + at;
      if (n == 16) {
        *(u32x4_b_t*)dst = x;
      } else {
        for (int b = 0; b < n; ++b) dst[b] = src[at + b];
      }
    }
  }
}

template <typename T, bool WHOLE>
__global__ __launch_bounds__(256) void unpermute_kernel(RowsParams P, int L) {
  constexpr int V = Vec<T>::N;
  Place p;
  if (!place(P, L, 1, p)) return;
  const int64_t t = WHOLE ? (int64_t)__builtin_amdgcn_readfirstlane((int)p.t) : p.t;
  const int vecs = (P.cols + V - 1) / V;
  const int32_t* sr = P.slot_row + t * P.k;
  const float* pr = P.prob ? P.prob + t * P.k : nullptr;
  const T* rows = (const T*)P.rows;
  for (int v = p.v; v < vecs; v += L) {
    const int col = v * V, n = P.cols - col;
    float acc[V];
#pragma unroll
    for (int q = 0; q < V; ++q) acc[q] = 0.f;
    // slots in groups whose loads are in flight together; added in slot order
    constexpr int G = 8;
    for (int j0 = 0; j0 < P.k; j0 += G) {
      int32_t r[G];
      typename Vec<T>::raw x[G];
#pragma unroll
      for (int i = 0; i < G; ++i) {
        r[i] = j0 + i < P.k ? sr[j0 + i] : -1;
        if (r[i] >= P.nrows) r[i] = -1;
      }
#pragma unroll
      for (int i = 0; i < G; ++i)
        if (r[i] >= 0) x[i] = Vec<T>::load(rows + (int64_t)r[i] * P.cols + col, n);
#pragma unroll
      for (int i = 0; i < G; ++i) {
        if (r[i] < 0) continue;
        float f[V];
        Vec<T>::get(x[i], f);
        const float w = pr ? pr[j0 + i] : 1.f;
#pragma unroll
        for (int q = 0; q < V; ++q) acc[q] = pr ? __builtin_fmaf(w, f[q], acc[q]) : acc[q] + f[q];
      }
    }
    if (P.add) {
      float a[V];
      Vec<T>::get(Vec<T>::load((const T*)P.add + t * P.ldadd + col, n), a);
#pragma unroll
      for (int q = 0; q < V; ++q) acc[q] = acc[q] + a[q];
    }
    Vec<T>::store((T*)P.out + t * P.cols + col, acc, n);
  }
}

// A wave a slot; the four waves of a workgroup have neighbouring slots, mostly
// of one token.
template <typename T>
__global__ __launch_bounds__(256) void unpermute_bwd_kernel(RowsParams P) {
  constexpr int V = Vec<T>::N;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n = P.tokens * P.k;
  const int64_t u = map_unit(blockIdx.x, (n + 3) / 4, P.seed);
  if (u < 0) return;
  const int64_t i = u * 4 + w;
  if (i >= n) return;
  const int32_t r = P.slot_row[i];
  if (r < 0 || r >= P.nrows) {
    if (P.dprob && lane == 0) P.dprob[i] = 0.f;
    return;
  }
  const T* dy = (const T*)P.x + i / P.k * P.ldx;
  const T* row = (const T*)P.rows + (int64_t)r * P.cols;
  T* out = (T*)P.out + (int64_t)r * P.cols;
  const float p = P.prob[i];
  float dot = 0.f;
  const int vecs = (P.cols + V - 1) / V;
#pragma unroll 4
  for (int v = lane; v < vecs; v += 64) {
    const int col = v * V, m = P.cols - col;
    float g[V];
    Vec<T>::get(Vec<T>::load(dy + col, m), g);
    if (P.dprob) {
      float f[V];
      Vec<T>::get(Vec<T>::load(row + col, m), f);
#pragma unroll
      for (int q = 0; q < V; ++q) dot = __builtin_fmaf(g[q], f[q], dot);
    }
#pragma unroll
    for (int q = 0; q < V; ++q) g[q] = p * g[q];
    Vec<T>::store(out + col, g, m);
  }
  if (!P.dprob) return;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) dot = dot + __shfl_xor(dot, d, 64);
  if (lane == 0) P.dprob[i] = dot;
}

hipError_t launch_permute(const RowsParams& P, int es, hipStream_t st) {
  const int L = row_threads(((int64_t)P.cols * es + 15) / 16);
  const int64_t groups = (P.tokens + 256 / L - 1) / (256 / L);
  // too few tokens for the device: their slots are split too
  int64_t S = groups >= 512 ? 1 : (512 + groups - 1) / groups;
  if (S > P.k) S = P.k;
  const int64_t grid = grid_for_units(groups * S);
  if (L >= 64)
    permute_kernel<true><<<grid, 256, 0, st>>>(P, es, L, (int)S);
  else
    permute_kernel<false><<<grid, 256, 0, st>>>(P, es, L, (int)S);
  return hipGetLastError();
}

hipError_t launch_unpermute(const RowsParams& P, bool bf16, hipStream_t st) {
  const int V = bf16 ? 8 : 4;
  const int L = row_threads((P.cols + V - 1) / V);
  const int64_t grid = grid_for_units((P.tokens + 256 / L - 1) / (256 / L));
  if (bf16) {
    if (L >= 64)
      unpermute_kernel<uint16_t, true><<<grid, 256, 0, st>>>(P, L);
    else
      unpermute_kernel<uint16_t, false><<<grid, 256, 0, st>>>(P, L);
  } else {
    if (L >= 64)
      unpermute_kernel<float, true><<<grid, 256, 0, st>>>(P, L);
    else
      unpermute_kernel<float, false><<<grid, 256, 0, st>>>(P, L);
  }
  return hipGetLastError();
}

hipError_t launch_unpermute_bwd(const RowsParams& P, bool bf16, hipStream_t st) {
  const int64_t grid = grid_for_units((P.tokens * P.k + 3) / 4);
  if (bf16)
    unpermute_bwd_kernel<uint16_t><<<grid, 256, 0, st>>>(P);
  else
    unpermute_bwd_kernel<float><<<grid, 256, 0, st>>>(P);
  return hipGetLastError();
}

}  // namespace moedet
