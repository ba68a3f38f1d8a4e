// Epilogues of the dense matrix operators on four consecutive columns of a
// row, shared by the tile kernels, the few-row kernels and the join of
// split contractions.
#pragma once

#include "dense.h"

namespace moedet {

// Activation and derivative in float32.  SiLU takes the hardware reciprocal
// and exponential (about 2^-22 relative); for z below about -88 the exponential
// overflows to infinity and the product is -0, the limit.  GELU's
// distribution function is Abramowitz and Stegun 7.1.26 for erfc, within
// 0.75e-7 of Phi and without the cancellation of 1 + erf for negative z:
//   Phi(-|z|) = 0.5 t (a1 + t (a2 + t (a3 + t (a4 + t a5)))) exp(-z^2 / 2),
//   t = 1 / (1 + 0.3275911 |z| / sqrt 2).
// (The library's erff, with its branch, took 40 us of the epilogues of a 4096 x
// 2048 x 8192 product, this form about 11.)
DEV float sigmoid_f(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }
// Phi(z), and exp(-z^2 / 2) in e
DEV float normal_cdf(float z, float& e) {
  const float x = __builtin_fabsf(z) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, x, 1.f));
  float p = __builtin_fmaf(t, 1.061405429f, -1.453152027f);
  p = __builtin_fmaf(t, p, 1.421413741f);
  p = __builtin_fmaf(t, p, -0.284496736f);
  p = __builtin_fmaf(t, p, 0.254829592f);
  e = __expf(-x * x);
  const float q = 0.5f * t * p * e;
  return z > 0.f ? 1.f - q : q;
}
DEV float act_f(int act, float z) {
  switch (act) {
    case kActRelu: return z < 0.f ? 0.f : z;
    case kActRelu2: {
      const float r = z < 0.f ? 0.f : z;
      return r * r;
    }
    case kActSilu: return z * sigmoid_f(z);
    case kActGelu: {
      float e;
      return z * normal_cdf(z, e);
    }
    default: return z;
  }
}
// value and derivative
DEV void act_df(int act, float z, float& v, float& d) {
  switch (act) {
    case kActRelu:
      v = z < 0.f ? 0.f : z;
      d = z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
      break;
    case kActRelu2: {
      const float r = z < 0.f ? 0.f : z;
      v = r * r;
      d = 2.f * r;
      break;
    }
    case kActSilu: {
      const float p = sigmoid_f(z);
      v = z * p;
      d = __builtin_fmaf(v, 1.f - p, p);
      break;
    }
    case kActGelu: {
      float e;
      const float c = normal_cdf(z, e);
      v = z * c;
      d = __builtin_fmaf(z * 0.39894228040143268f, e, c);
      break;
    }
    default:
      v = z;
      d = 1.f;
  }
}

// N values and derivatives, with the switch outside as in act_n.
template <int N>
DEV void act_df_n(int act, const float (&z)[N], float (&v)[N], float (&d)[N]) {
  switch (act) {
    case kActNone:
#pragma unroll
      for (int i = 0; i < N; ++i) act_df(kActNone, z[i], v[i], d[i]);
      return;
    case kActRelu:
#pragma unroll
      for (int i = 0; i < N; ++i) act_df(kActRelu, z[i], v[i], d[i]);
      return;
    case kActRelu2:
#pragma unroll
      for (int i = 0; i < N; ++i) act_df(kActRelu2, z[i], v[i], d[i]);
      return;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < N; ++i) act_df(kActSilu, z[i], v[i], d[i]);
      return;
    default:
#pragma unroll
      for (int i = 0; i < N; ++i) act_df(kActGelu, z[i], v[i], d[i]);
  }
}

// Elements [0, n) of four, n >= 1 (more count as four); any address.
DEV void get4(const uint16_t* p, int n, float (&v)[4]) {
  if (n >= 4) {
    const u32x2_t r = *(const u32x2_any_t*)p;
    v[0] = __uint_as_float(r[0] << 16);
    v[1] = __uint_as_float(r[0] & 0xffff0000u);
    v[2] = __uint_as_float(r[1] << 16);
    v[3] = __uint_as_float(r[1] & 0xffff0000u);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = i < n ? bf16_to_f32(p[i]) : 0.f;
}
DEV void get4(const float* p, int n, float (&v)[4]) {
  const f32x4_t r = Vec<float>::load(p, n);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = r[i];
}
// STREAM: non-temporal, for the outputs of the tile kernels, which are written
// once and in bulk: the L2 keeps the operand tiles instead (4096 x 2048 x 8192
// gated product with saved pre-activations 264 -> 248 us, 8192^3 792 -> 779 us).
template <bool STREAM>
DEV void put4(uint16_t* p, int n, const float (&v)[4]) {
  const u32x2_t r = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  if (n >= 4) {
    if constexpr (STREAM)
      __builtin_nontemporal_store(r, (u32x2_any_t*)p);
    else
      *(u32x2_any_t*)p = r;
    return;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < n) p[i] = (uint16_t)(r[i >> 1] >> (16 * (i & 1)));
}
template <bool STREAM>
DEV void put4(float* p, int n, const float (&v)[4]) {
  if (STREAM && n >= 4)
    __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, (f32x4_any_t*)p);
  else
    Vec<float>::store(p, v, n);
}

// Saved pre-activations of matrix m, in the storage type or float32.
template <typename T, bool STREAM>
DEV void put_z(const DenseParams& P, int m, int64_t row, int col, int n, const float (&v)[4]) {
  if (sizeof(T) == 2 && P.z_f32)
    put4<STREAM>((float*)P.z[m] + row * P.ldz + col, n, v);
  else
    put4<STREAM>((T*)P.z[m] + row * P.ldz + col, n, v);
}

// Activation of N values: the switch is outside, so that the values' chains of
// dependent operations overlap (a wave is alone on its SIMD in the tile kernels).
template <int N>
DEV void act_n(int act, float (&v)[N]) {
  switch (act) {
    case kActNone: return;
    case kActRelu:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_f(kActRelu, v[i]);
      return;
    case kActRelu2:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_f(kActRelu2, v[i]);
      return;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_f(kActSilu, v[i]);
      return;
    default:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_f(kActGelu, v[i]);
  }
}

// Where the R groups of four columns of an epilogue step lie.
struct AtRows {   // rows row, row + step, ... below `end`, columns col..col+3
  int64_t row0, end;
  int step, col0;
  DEV int64_t row(int i) const { return row0 + i * step; }
  DEV int col(int) const { return col0; }
  DEV bool ok(int i, int) const { return row0 + i * step < end; }
};
struct AtCols {   // one row, columns col, col + step, ...
  int64_t row0;
  int step, col0;
  DEV int64_t row(int) const { return row0; }
  DEV int col(int i) const { return col0 + i * step; }
  DEV bool ok(int i, int N) const { return col0 + i * step < N; }
};

// C at R groups (matrix `seg` in kFormDw); v holds them one after the other.
// BIASED: the caller has added the bias.
template <typename T, int FORM, int R, bool STREAM, bool BIASED, class At>
DEV void emit(const DenseParams& P, int seg, const At& at, float (&v)[4 * R]) {
  float t[4], o[4 * R];
  if (FORM != kFormDw && P.add) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (at.ok(i, P.N)) {
        get4((const T*)P.add + at.row(i) * P.ldadd + at.col(i), P.N - at.col(i), t);
#pragma unroll
        for (int q = 0; q < 4; ++q) o[4 * i + q] = t[q];
      }
  }
  if constexpr (FORM == kFormLinear) {
    if (!BIASED && P.bias) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (at.ok(i, P.N)) {
          get4((const T*)P.bias + at.col(i), P.N - at.col(i), t);
#pragma unroll
          for (int q = 0; q < 4; ++q) v[4 * i + q] = v[4 * i + q] + t[q];
        }
    }
    if (P.z[0]) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (at.ok(i, P.N))
          put_z<T, STREAM>(P, 0, at.row(i), at.col(i), P.N - at.col(i), {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]});
    }
    act_n<4 * R>(P.act, v);
  }
  if (FORM != kFormDw && P.add) {
#pragma unroll
    for (int i = 0; i < 4 * R; ++i) v[i] = v[i] + o[i];
  }
  void* c = FORM == kFormDw && seg ? P.c[1] : P.c[0];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (!at.ok(i, P.N)) continue;
    const int64_t pos = at.row(i) * P.ldc + at.col(i);
    const float w[4] = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    if (FORM == kFormDw && P.c_f32)
      put4<STREAM>((float*)c + pos, P.N - at.col(i), w);
    else
      put4<STREAM>((T*)c + pos, P.N - at.col(i), w);
  }
}

// The same for the gated product: g and u.
template <typename T, int R, bool STREAM, class At>
DEV void emit_glu(const DenseParams& P, const At& at, float (&g)[4 * R], const float (&u)[4 * R]) {
  if (P.z[0]) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (at.ok(i, P.N)) {
        const int n = P.N - at.col(i);
        put_z<T, STREAM>(P, 0, at.row(i), at.col(i), n, {g[4 * i], g[4 * i + 1], g[4 * i + 2], g[4 * i + 3]});
        put_z<T, STREAM>(P, 1, at.row(i), at.col(i), n, {u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]});
      }
  }
  act_n<4 * R>(P.act, g);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (!at.ok(i, P.N)) continue;
    const float w[4] = {g[4 * i] * u[4 * i], g[4 * i + 1] * u[4 * i + 1], g[4 * i + 2] * u[4 * i + 2],
                        g[4 * i + 3] * u[4 * i + 3]};
    put4<STREAM>((T*)P.c[0] + at.row(i) * P.ldc + at.col(i), P.N - at.col(i), w);
  }
}

template <typename T, int FORM>
DEV void emit4(const DenseParams& P, int seg, int64_t row, int col, float (&v)[4]) {
  emit<T, FORM, 1, false, false>(P, seg, AtRows{row, row + 1, 1, col}, v);
}
template <typename T>
DEV void emit4_glu(const DenseParams& P, int64_t row, int col, float (&g)[4], const float (&u)[4]) {
  emit_glu<T, 1, false>(P, AtRows{row, row + 1, 1, col}, g, u);
}

// A chunk's partial of matrix seg; partial rows hold whole groups of four.
DEV void part4(const DenseParams& P, int chunk, int seg, int64_t row, int col, const float (&v)[4]) {
  *(f32x4_t*)(P.part + ((int64_t)chunk * P.M + row) * P.part_ld + seg * P.part_seg + col) =
      f32x4_t{v[0], v[1], v[2], v[3]};
}
template <int R, class At>
DEV void part(const DenseParams& P, int chunk, int seg, const At& at, const float (&v)[4 * R]) {
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (at.ok(i, P.N)) part4(P, chunk, seg, at.row(i), at.col(i), {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]});
}

}  // namespace moedet
