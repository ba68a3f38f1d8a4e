// Layer norm, forward and backward.
//
//   mean = sum(x) / C,  rstd = 1 / sqrt(sum((x - mean)^2) / C + eps)
//   y  = h w + b,       h = (x - mean) rstd
//   dx = rstd (dh - sum(dh) / C - h sum(dh h) / C) (+ add),  dh = dy w
//   dw = sum over rows of dy h,   db = sum over rows of dy
//
// Both directions read each row once and keep it in registers, so the
// variance is the sum of the squared distances from the mean that the first
// sum gave (no cancellation of E[x^2] - mean^2).  A row belongs to TPR threads (one wave up
// to 2048 columns, so that a row needs no barrier; more waves for wider rows),
// each holding EPT of its elements as 16-byte vectors.  Vectors may start at
// any element, so odd widths and strides take the same path; the last vector
// of a row that is no multiple of the vector is read element by element.
//
// The rows of the backward are cut into at most 512 blocks with bounds made
// from the sizes alone.  A thread adds its columns' dy h and dy over the
// block's rows in registers, the block's row groups are added in order
// through LDS, and a second launch adds the blocks in order: no atomics.
//
// Both are bound by HBM.
#include "dense.h"
#include "kernels.h"

namespace moedet {

// Sum over the wave, the same bits in every lane (a + b == b + a).
DEV float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v = v + __shfl_xor(v, d, kWave);
  return v;
}

// Sum over the TPR threads of a row; s: one float per wave, free to use (two
// calls in a row take different arrays).
template <int TPR>
DEV float row_sum(float v, float* s) {
  v = wave_sum(v);
  if constexpr (TPR > kWave) {
    const int w = threadIdx.x / kWave, first = w / (TPR / kWave) * (TPR / kWave);
    if ((threadIdx.x & (kWave - 1)) == 0) s[w] = v;
    __syncthreads();
    v = s[first];
#pragma unroll
    for (int i = 1; i < TPR / kWave; ++i) v = v + s[first + i];
  }
  return v;
}

template <int TPR>
constexpr int norm_threads = TPR > 256 ? TPR : 256;

// Vector j of a row's `cols` elements, held by thread t of the row: loads give
// zeros past the row (GUARD; without it the row fills every thread's
// registers exactly, and no load or store is conditional).
template <typename T, int TPR, bool GUARD>
DEV typename Vec<T>::raw row_load(const T* p, int j, int t, int C) {
  const int c = (j * TPR + t) * Vec<T>::N;
  if constexpr (!GUARD) return Vec<T>::load(p + c, Vec<T>::N);
  typename Vec<T>::raw r{};
  if (c < C) r = Vec<T>::load(p + c, C - c);
  return r;
}
template <typename T, int TPR, bool GUARD>
DEV void row_store(T* p, int j, int t, int C, const float* v) {
  const int c = (j * TPR + t) * Vec<T>::N;
  if constexpr (!GUARD)
    Vec<T>::store(p + c, v, Vec<T>::N);
  else if (c < C)
    Vec<T>::store(p + c, v, C - c);
}
// A weight that is not given is 1.
template <typename T, int TPR, bool GUARD>
DEV typename Vec<T>::raw weight_load(const void* w, int j, int t, int C) {
  if (w) return row_load<T, TPR, GUARD>((const T*)w, j, t, C);
  typename Vec<T>::raw r;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (sizeof(T) == 2)
      r[q] = 0x3f803f80u;
    else
      r[q] = 1.f;
  }
  return r;
}

template <typename T, int TPR, int EPT, bool GUARD>
__global__ __launch_bounds__(norm_threads<TPR>) void norm_fwd_kernel(NormParams P) {
  constexpr int NT = norm_threads<TPR>, V = Vec<T>::N, NV = EPT / V, RPB = NT / TPR;
  __shared__ float s_a[2][NT / kWave], s_b[2][NT / kWave];
  const int64_t units = (P.rows + RPB - 1) / RPB;
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int C = GUARD ? P.cols : TPR * EPT;
  const float Cf = (float)C;
  typename Vec<T>::raw w[NV], b[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    w[j] = weight_load<T, TPR, GUARD>(P.weight, j, t, C);
    b[j] = typename Vec<T>::raw{};
    if (P.bias) b[j] = row_load<T, TPR, GUARD>((const T*)P.bias, j, t, C);
  }
  int odd = 0;
  for (int64_t i = blockIdx.x; i < units; i += gridDim.x, odd ^= 1) {
    // the shuffle permutes the units; it keeps every unit on one block
    const int64_t u = P.seed ? shuffle_unit(i, units, P.seed) : i;
    const int64_t row = u * RPB + grp;
    const bool live = row < P.rows;
    const T* xr = (const T*)P.x + (live ? row : 0) * P.ldx;
    typename Vec<T>::raw raw[NV];
    float v[EPT];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) raw[j] = row_load<T, TPR, GUARD>(xr, j, t, C);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      Vec<T>::get(raw[j], v + j * V);
#pragma unroll
      for (int q = 0; q < V; ++q) sum = sum + v[j * V + q];   // past the row: zeros
    }
    // a division: a row of one value then has exactly that mean
    const float mean = row_sum<TPR>(sum, s_a[odd]) / Cf;
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + t) * V;
#pragma unroll
      for (int q = 0; q < V; ++q) {
        v[j * V + q] = v[j * V + q] - mean;
        const float d = GUARD && c + q >= C ? 0.f : v[j * V + q];
        sq = __builtin_fmaf(d, d, sq);
      }
    }
    const float rstd = 1.f / sqrtf(row_sum<TPR>(sq, s_b[odd]) / Cf + P.eps);
    if (!live) continue;
    T* yr = (T*)P.y + row * C;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float o[V], fw[V], fb[V];
      Vec<T>::get(w[j], fw);
      Vec<T>::get(b[j], fb);
#pragma unroll
      for (int q = 0; q < V; ++q) o[q] = __builtin_fmaf(v[j * V + q] * rstd, fw[q], fb[q]);
      row_store<T, TPR, GUARD>(yr, j, t, C, o);
    }
    if (P.mean && t == 0) {
      P.mean[row] = mean;
      P.rstd[row] = rstd;
    }
  }
}

// Block u of P.blocks takes the rows [u rows / blocks, (u + 1) rows / blocks);
// its row groups take them in turn.
template <typename T, int TPR, int EPT, bool GUARD>
__global__ __launch_bounds__(norm_threads<TPR>) void norm_bwd_kernel(NormParams P) {
  constexpr int NT = norm_threads<TPR>, V = Vec<T>::N, NV = EPT / V, RPB = NT / TPR;
  // the widest rows load the weight and the added gradient where they are
  // used: held over the row they do not fit in 128 registers
  constexpr bool kHold = TPR * EPT < kNormMaxCols;
  __shared__ float s_a[2][NT / kWave], s_b[2][NT / kWave];
  __shared__ float s_col[RPB > 1 ? TPR * EPT : 1];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int C = GUARD ? P.cols : TPR * EPT;
  const float Cf = (float)C;
  int64_t u = blockIdx.x;
  if (P.seed) {
    shuffle_delay(P.seed, u);
    u = shuffle_unit(u, P.blocks, P.seed);
  }
  const int64_t r0 = u * P.rows / P.blocks, r1 = (u + 1) * P.rows / P.blocks;
  typename Vec<T>::raw w[NV];
  if constexpr (kHold) {
#pragma unroll
    for (int j = 0; j < NV; ++j) w[j] = weight_load<T, TPR, GUARD>(P.weight, j, t, C);
  }
  float dw[EPT], db[EPT];
#pragma unroll
  for (int q = 0; q < EPT; ++q) dw[q] = db[q] = 0.f;
  int odd = 0;
  // every group runs the same number of rounds: row_sum has barriers
  for (int64_t base = r0; base < r1; base += RPB, odd ^= 1) {
    const int64_t row = base + grp;
    const bool live = row < r1;
    const int64_t rr = live ? row : r0;
    const T* xr = (const T*)P.x + rr * P.ldx;
    const T* gr = (const T*)P.dy + rr * P.lddy;
    const T* ar = P.add ? (const T*)P.add + rr * P.ldadd : nullptr;
    typename Vec<T>::raw rx[NV], rg[NV], ra[NV];
    const float mean = P.mean[rr], rstd = P.rstd[rr];
    if constexpr (kHold) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        rx[j] = row_load<T, TPR, GUARD>(xr, j, t, C);
        rg[j] = row_load<T, TPR, GUARD>(gr, j, t, C);
      }
    }
    if (kHold && ar) {
#pragma unroll
      for (int j = 0; j < NV; ++j) ra[j] = row_load<T, TPR, GUARD>(ar, j, t, C);
    }
    // past the row dy = 0 and the weight are 0, which adds nothing
    float h[EPT], dh[EPT], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float x[V], g[V], f[V];
      Vec<T>::get(kHold ? rx[j] : row_load<T, TPR, GUARD>(xr, j, t, C), x);
      Vec<T>::get(kHold ? rg[j] : row_load<T, TPR, GUARD>(gr, j, t, C), g);
      Vec<T>::get(kHold ? w[j] : weight_load<T, TPR, GUARD>(P.weight, j, t, C), f);
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const int e = j * V + q;
        h[e] = (x[q] - mean) * rstd;
        dh[e] = g[q] * f[q];
        s1 = s1 + dh[e];
        s2 = __builtin_fmaf(dh[e], h[e], s2);
        if (RPB == 1 || live) {
          dw[e] = __builtin_fmaf(g[q], h[e], dw[e]);
          db[e] = db[e] + g[q];
        }
      }
    }
    const float m1 = row_sum<TPR>(s1, s_a[odd]) / Cf;
    const float m2 = row_sum<TPR>(s2, s_b[odd]) / Cf;
    if (!live) continue;
    T* dr = (T*)P.y + row * C;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float o[V];
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const int e = j * V + q;
        o[q] = (dh[e] - m1 - h[e] * m2) * rstd;
      }
      if (ar) {
        float f[V];
        Vec<T>::get(kHold ? ra[j] : row_load<T, TPR, GUARD>(ar, j, t, C), f);
#pragma unroll
        for (int q = 0; q < V; ++q) o[q] = o[q] + f[q];
      }
      row_store<T, TPR, GUARD>(dr, j, t, C, o);
    }
  }
  if (!P.part) return;
  float* pw = P.part + u * 2 * C;
  // the groups' sums in group order, dw then db
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* acc = which ? db : dw;
    if constexpr (RPB > 1) {
      for (int g = 1; g < RPB; ++g) {
        __syncthreads();
        if (grp == g)
#pragma unroll
          for (int q = 0; q < EPT; ++q) s_col[q * TPR + t] = acc[q];
        __syncthreads();
        if (grp == 0)
#pragma unroll
          for (int q = 0; q < EPT; ++q) acc[q] = acc[q] + s_col[q * TPR + t];
      }
    }
    if (grp == 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int q = 0; q < V; ++q) {
          const int c = (j * TPR + t) * V + q;
          if (c < C) pw[which * C + c] = acc[j * V + q];
        }
    }
  }
}

// One launch for dweight and dbias: the second half of the grid sums the
// columns after the first `cols`.
__global__ __launch_bounds__(256) void block_sums_kernel(const float* part, int blocks, int64_t stride, int cols,
                                                         void* out, void* out2) {
  const uint32_t per = (uint32_t)(cols + 15) / 16;
  const bool second = blockIdx.x >= per;
  block_sum16(second ? part + cols : part, blocks, stride, cols, second ? blockIdx.x - per : blockIdx.x,
              second ? out2 : out, false);
}

int norm_bwd_blocks(int64_t rows, int64_t cols, bool bf16) {
  const int rpb = cols <= (bf16 ? 2048 : 1024) ? 4 : 1;   // rows a block holds at a time
  const int64_t b = (rows + rpb - 1) / rpb;
  return (int)(b < 1 ? 1 : b > kNormBlocks ? kNormBlocks : b);
}

template <typename T, int TPR, int EPT, bool GUARD>
static void norm_launch_as(const NormParams& P, bool bwd, unsigned blocks, hipStream_t st) {
  if (bwd)
    norm_bwd_kernel<T, TPR, EPT, GUARD><<<blocks, norm_threads<TPR>, 0, st>>>(P);
  else
    norm_fwd_kernel<T, TPR, EPT, GUARD><<<blocks, norm_threads<TPR>, 0, st>>>(P);
}

template <typename T, int TPR, int EPT>
static hipError_t norm_launch(const NormParams& P, bool bwd, hipStream_t st) {
  constexpr int NT = norm_threads<TPR>, RPB = NT / TPR;
  // a forward block takes several rows only when every CU already holds 8
  // waves a SIMD: then the weight stays in registers
  const int64_t units = (P.rows + RPB - 1) / RPB, most = 2048 * 256 / NT;
  const unsigned blocks = bwd ? P.blocks : (unsigned)(units < most ? units : most);
  if (P.cols == TPR * EPT)
    norm_launch_as<T, TPR, EPT, false>(P, bwd, blocks, st);
  else
    norm_launch_as<T, TPR, EPT, true>(P, bwd, blocks, st);
  return hipGetLastError();
}

template <typename T>
static hipError_t norm_dispatch(const NormParams& P, bool bwd, hipStream_t st) {
  // One wave per row up to 2048 bf16 or 1024 float32 columns (what its
  // registers hold twice over), four waves up to 4096, sixteen beyond.
  if (P.cols <= 512) return norm_launch<T, 64, 8>(P, bwd, st);
  if (P.cols <= 1024) return norm_launch<T, 64, 16>(P, bwd, st);
  if (P.cols <= 2048) return norm_launch<T, sizeof(T) == 2 ? 64 : 256, sizeof(T) == 2 ? 32 : 8>(P, bwd, st);
  if (P.cols <= 4096) return norm_launch<T, 256, 16>(P, bwd, st);
  if (P.cols <= 8192) return norm_launch<T, 1024, 8>(P, bwd, st);
  return norm_launch<T, 1024, 16>(P, bwd, st);
}

hipError_t launch_norm_fwd(const NormParams& P, bool bf16, hipStream_t st) {
  if (P.rows == 0) return hipSuccess;
  return bf16 ? norm_dispatch<uint16_t>(P, false, st) : norm_dispatch<float>(P, false, st);
}

hipError_t launch_norm_bwd(const NormParams& P, bool bf16, hipStream_t st) {
  return bf16 ? norm_dispatch<uint16_t>(P, true, st) : norm_dispatch<float>(P, true, st);
}

hipError_t launch_block_sums(const float* part, int blocks, int64_t stride, int cols, void* out, void* out2,
                             hipStream_t st) {
  block_sums_kernel<<<(cols + 15) / 16 * (out2 ? 2 : 1), 256, 0, st>>>(part, blocks, stride, cols, out, out2);
  return hipGetLastError();
}

}  // namespace moedet
