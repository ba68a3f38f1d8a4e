// Epilogues of the dense matrix operators on four consecutive columns of a
// row, shared by the tile kernels, the few-row kernels and the join of
// split contractions.
#pragma once

#include "dense.h"

namespace moedet {

// Activations and derivatives in float32, accurate for a result in float32 (FINE) or
// rounded to bf16.  Errors are relative, in the tails too, down to results of about
// 2^-120, where the exponential's underflow ends them.  E = 2^-24.
//
// SiLU is z s(z), s(z) = 1 / (1 + exp(-z)), s' = s (1 - s).  The hardware's
// exponential (of base 2) and reciprocal are within 2 E.
//   FINE  from e = exp(-|z|), which cannot overflow: s(|z|) = 1 / (1 + e) and s(-|z|) =
//         e / (1 + e), so neither s nor 1 - s cancels, and the error stays below 12 E.
//   else  s directly: the rounding of the exponential's argument grows with |z|, and
//         the error with it to about (2 |z| + 8) E.
//
// GELU is z Phi(z) with Phi(-|z|) = erfc(|z| / sqrt 2) / 2 = t P(t) exp(-z^2 / 2),
// t = 1 / (1 + p |z|), and Phi(|z|) = 1 - Phi(-|z|), which does not cancel either.
// P is a polynomial fitted to erfcx(|z| / sqrt 2) / (2 t) for the least relative error
// over 0 <= |z| <= 13.3, beyond which the exponential is 0.
//   FINE  9 coefficients, within 1.9e-8, and z^2 / 2 in two parts: below 24 E altogether.
//   else  7 coefficients, within 1.2e-6, below (3 z^2 + 64) E altogether.
// (The library's erff, with its branch, took 40 us of the epilogues of a 4096 x
// 2048 x 8192 product, this form and the bias about 15.)
//
// exp(-(h + l)) for h >= 0 and a small l, the product with log2 e in two parts
DEV float exp_neg(float h, float l) {
  const float c = 1.44269502f, c2 = 1.92596299e-8f, ln2 = 0.693147182f;
  const float y = h * c;
  const float r = __builtin_fmaf(l, c, __builtin_fmaf(h, c2, __builtin_fmaf(h, c, -y)));
  const float e = __builtin_amdgcn_exp2f(-y);
  return __builtin_fmaf(e, -ln2 * r, e);
}
// s(z) and s(-z)
template <bool FINE>
DEV void sigmoid_f(float z, float& s, float& c) {
  if constexpr (FINE) {
    const float e = exp_neg(__builtin_fminf(__builtin_fabsf(z), 128.f), 0.f), r = __builtin_amdgcn_rcpf(1.f + e);
    s = z >= 0.f ? r : e * r;
    c = z >= 0.f ? e * r : r;
  } else {
    s = __builtin_amdgcn_rcpf(1.f + __expf(-z));
    c = 1.f - s;
  }
}
// Phi(z), and exp(-z^2 / 2) in e
template <bool FINE>
DEV float normal_cdf(float z, float& e) {
  float q;
  if constexpr (FINE) {
    const float x = __builtin_fminf(__builtin_fabsf(z), 16.f), h = x * x;
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.344f, x, 1.f));
    q = __builtin_fmaf(t, -2.826836167e-2f, 1.457166378e-1f);
    q = __builtin_fmaf(t, q, -2.746732555e-1f);
    q = __builtin_fmaf(t, q, 1.934512497e-1f);
    q = __builtin_fmaf(t, q, -4.106735419e-2f);
    q = __builtin_fmaf(t, q, 1.133146049e-1f);
    q = __builtin_fmaf(t, q, 1.166451889e-1f);
    q = __builtin_fmaf(t, q, 1.376630181e-1f);
    q = __builtin_fmaf(t, q, 1.372182633e-1f);
    e = exp_neg(0.5f * h, 0.5f * __builtin_fmaf(x, x, -h));
    q = q * t * e;
  } else {
    const float x = __builtin_fabsf(z);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.199f, x, 1.f));
    q = __builtin_fmaf(t, 3.008919769e-1f, -4.435143378e-1f);
    q = __builtin_fmaf(t, q, 5.122382957e-1f);
    q = __builtin_fmaf(t, q, -1.644029879e-1f);
    q = __builtin_fmaf(t, q, 1.466305782e-1f);
    q = __builtin_fmaf(t, q, 6.799873163e-2f);
    q = __builtin_fmaf(t, q, 8.015767340e-2f);
    // exp(-z^2 / 2) as a power of 2: one product less than through the base e
    e = __builtin_amdgcn_exp2f(-0.721347520f * x * x);
    q = q * t * e;
  }
  return z > 0.f ? 1.f - q : q;
}
template <bool FINE>
DEV float act_f(int act, float z) {
  switch (act) {
    case kActRelu: return z < 0.f ? 0.f : z;
    case kActRelu2: {
      const float r = z < 0.f ? 0.f : z;
      return r * r;
    }
    case kActSilu: {
      float s, c;
      sigmoid_f<FINE>(z, s, c);
      return z * s;
    }
    case kActGelu: {
      float e;
      return z * normal_cdf<FINE>(z, e);
    }
    default: return z;
  }
}
// value and derivative
template <bool FINE>
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
      float s, c;
      sigmoid_f<FINE>(z, s, c);
      v = z * s;
      d = __builtin_fmaf(v, c, s);
      break;
    }
    case kActGelu: {
      float e;
      const float c = normal_cdf<FINE>(z, e);
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
template <bool FINE, int N>
DEV void act_df_n(int act, const float (&z)[N], float (&v)[N], float (&d)[N]) {
  switch (act) {
    case kActNone:
#pragma unroll
      for (int i = 0; i < N; ++i) act_df<FINE>(kActNone, z[i], v[i], d[i]);
      return;
    case kActRelu:
#pragma unroll
      for (int i = 0; i < N; ++i) act_df<FINE>(kActRelu, z[i], v[i], d[i]);
      return;
    case kActRelu2:
#pragma unroll
      for (int i = 0; i < N; ++i) act_df<FINE>(kActRelu2, z[i], v[i], d[i]);
      return;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < N; ++i) act_df<FINE>(kActSilu, z[i], v[i], d[i]);
      return;
    default:
#pragma unroll
      for (int i = 0; i < N; ++i) act_df<FINE>(kActGelu, z[i], v[i], d[i]);
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
template <bool FINE, int N>
DEV void act_n(int act, float (&v)[N]) {
  switch (act) {
    case kActNone: return;
    case kActRelu:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_f<FINE>(kActRelu, v[i]);
      return;
    case kActRelu2:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_f<FINE>(kActRelu2, v[i]);
      return;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_f<FINE>(kActSilu, v[i]);
      return;
    default:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_f<FINE>(kActGelu, v[i]);
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
    act_n<sizeof(T) == 4, 4 * R>(P.act, v);
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
  act_n<sizeof(T) == 4, 4 * R>(P.act, g);
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
