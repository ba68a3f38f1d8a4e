// Dropout with numbers from a counter, so that no mask is stored and the
// backward, a rerun or a resumed run finds the same one.
//
// Element i (counted over the logical tensor, row by row) takes word i % 4 of
// Philox 4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011) at counter first + i / 4 under the key;
// it is dropped where the word is below round(p 2^32).  y = x scale + add for
// a kept element, add (or 0) for a dropped one: one fused multiply-add in float32 (where x scale
// and add cancel, their difference keeps what a rounded product would lose), rounded to the type.
//
// Bound by HBM (16384 x 2048 bf16 with a residual and its gradient, 335 MB: 64 to 74 us, 4.5 to 5.3
// TB/s): the 19 products of 64 bits behind four elements, quarter-rate instructions,
// run beside the loads.
#include "rows.h"

namespace moedet {

namespace {

struct Words {
  uint32_t w[4];
};
DEV uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) { return (uint32_t)__builtin_amdgcn_bitop3_b32((int)a, (int)b, (int)c, 0x96); }
DEV Words philox(uint64_t counter, uint64_t key) {
  uint32_t c0 = (uint32_t)counter, c1 = (uint32_t)(counter >> 32), c2 = 0u, c3 = 0u;
  uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = xor3((uint32_t)(b >> 32), c1, k0);
    c1 = (uint32_t)b;
    c2 = xor3((uint32_t)(a >> 32), c3, k1);
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Words{{c0, c1, c2, c3}};
}

DEV float load1(const uint16_t* p) { return bf16_to_f32(*p); }
DEV float load1(const float* p) { return *p; }
DEV void store1(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16(v); }
DEV void store1(float* p, float v) { *p = v; }

}  // namespace

enum { kFlat = 0, kRowVecs = 1, kElements = 2 };

// kFlat      every matrix contiguous: one long row
// kRowVecs   whole 16-byte vectors in a row, rows apart
// kElements  any columns, rows apart: four elements of one counter a thread
template <typename T, int FORM>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutParams P, int64_t n) {
  constexpr int V = FORM == kElements ? 4 : Vec<T>::N;
  const int64_t units = (n + 256 * V - 1) / (256 * V);
  const int64_t u = stream_unit(blockIdx.x, units, P.seed);
  if (u < 0) return;
  const int64_t i0 = (u * 256 + threadIdx.x) * V;
  if (i0 >= n) return;
  const uint64_t key = P.rng[0], first = P.rng[1];
  const T* x = (const T*)P.x;
  const T* add = (const T*)P.add;
  T* y = (T*)P.y;
  if constexpr (FORM == kElements) {
    const Words w = philox(first + (uint64_t)(i0 >> 2), key);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t i = i0 + q;
      if (i >= n) break;
      const int64_t row = i / P.cols, col = i - row * P.cols;
      const float a = add ? load1(add + row * P.ldadd + col) : 0.f;
      const float v = load1(x + row * P.ldx + col);
      store1(y + i, w.w[q] < P.limit || P.all ? a : __builtin_fmaf(v, P.scale, a));
    }
  } else {
    int64_t at = i0, at_add = i0;
    if constexpr (FORM == kRowVecs) {
      const int64_t vec = i0 / V, per = P.cols / V;
      const int64_t row = n < ((int64_t)1 << 32) ? (int64_t)((uint32_t)vec / (uint32_t)per) : vec / per;
      const int64_t col = i0 - row * P.cols;
      at = row * P.ldx + col;
      at_add = row * P.ldadd + col;
    }
    const int m = (int)(n - i0 < V ? n - i0 : V);
    const typename Vec<T>::raw rx = Vec<T>::load(x + at, m);
    float f[V], a[V];
    if (add) {
      Vec<T>::get(Vec<T>::load(add + at_add, m), a);
    } else {
#pragma unroll
      for (int q = 0; q < V; ++q) a[q] = 0.f;
    }
    Vec<T>::get(rx, f);
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
      const Words w = philox(first + (uint64_t)((i0 >> 2) + h), key);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        f[4 * h + q] = w.w[q] < P.limit || P.all ? a[4 * h + q] : __builtin_fmaf(f[4 * h + q], P.scale, a[4 * h + q]);
    }
    Vec<T>::store(y + i0, f, m);
  }
}

static int dropout_form(const DropoutParams& P, int vec) {
  const bool flat = P.rows == 1 || (P.ldx == P.cols && (!P.add || P.ldadd == P.cols));
  return flat ? kFlat : P.cols % vec == 0 ? kRowVecs : kElements;
}
static int64_t form_grid(const DropoutParams& P, int form, int vec) {
  const int64_t per = 256 * (form == kElements ? 4 : vec);
  return (P.rows * P.cols + per - 1) / per;
}
int64_t dropout_grid(const DropoutParams& P, bool bf16) {
  const int vec = bf16 ? Vec<uint16_t>::N : Vec<float>::N;
  return form_grid(P, dropout_form(P, vec), vec);
}

template <typename T>
static hipError_t launch_form(const DropoutParams& P, hipStream_t st) {
  const int64_t n = P.rows * P.cols;
  const int form = dropout_form(P, Vec<T>::N);
  const int64_t grid = form_grid(P, form, Vec<T>::N);
  if (form == kFlat)
    dropout_kernel<T, kFlat><<<grid, 256, 0, st>>>(P, n);
  else if (form == kRowVecs)
    dropout_kernel<T, kRowVecs><<<grid, 256, 0, st>>>(P, n);
  else
    dropout_kernel<T, kElements><<<grid, 256, 0, st>>>(P, n);
  return hipGetLastError();
}

hipError_t launch_dropout(const DropoutParams& P, bool bf16, hipStream_t st) {
  return bf16 ? launch_form<uint16_t>(P, st) : launch_form<float>(P, st);
}

}  // namespace moedet
