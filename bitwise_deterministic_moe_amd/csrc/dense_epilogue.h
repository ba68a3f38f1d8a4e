// Epilogues of the dense matrix operators on four consecutive columns of a
// row, shared by the tile kernels, the few-row kernels and the join of
// split contractions.
#pragma once

#include "dense.h"

namespace moedet {

// Activation and derivative in float32.  SiLU takes the hardware reciprocal
// and exponential (about 2^-22 relative); for z below about -88 the exponential
// overflows to infinity and the product is -0, the limit.  GELU's
// distribution function is 0.5 + 0.5 erf(z / sqrt 2).
DEV float sigmoid_f(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }
DEV float act_f(int act, float z) {
  switch (act) {
    case kActRelu: return z < 0.f ? 0.f : z;
    case kActRelu2: {
      const float r = z < 0.f ? 0.f : z;
      return r * r;
    }
    case kActSilu: return z * sigmoid_f(z);
    case kActGelu: return z * __builtin_fmaf(0.5f, erff(z * 0.70710678118654752f), 0.5f);
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
      const float c = __builtin_fmaf(0.5f, erff(z * 0.70710678118654752f), 0.5f);
      v = z * c;
      d = __builtin_fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z), c);
      break;
    }
    default:
      v = z;
      d = 1.f;
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
DEV void put4(uint16_t* p, int n, const float (&v)[4]) {
  const u32x2_t r = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  if (n >= 4) {
    *(u32x2_any_t*)p = r;
    return;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < n) p[i] = (uint16_t)(r[i >> 1] >> (16 * (i & 1)));
}
DEV void put4(float* p, int n, const float (&v)[4]) { Vec<float>::store(p, v, n); }

// Saved pre-activations of matrix m, in the storage type or float32.
template <typename T>
DEV void put_z(const DenseParams& P, int m, int64_t row, int col, int n, const float (&v)[4]) {
  if (sizeof(T) == 2 && P.z_f32)
    put4((float*)P.z[m] + row * P.ldz + col, n, v);
  else
    put4((T*)P.z[m] + row * P.ldz + col, n, v);
}

// v = C[row, col..col+3] of matrix `seg` (kFormDw), n = columns that exist
template <typename T, int FORM>
DEV void emit4(const DenseParams& P, int seg, int64_t row, int col, float (&v)[4]) {
  const int n = P.N - col;
  if constexpr (FORM == kFormLinear) {
    float t[4];
    if (P.bias) {
      get4((const T*)P.bias + col, n, t);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = v[q] + t[q];
    }
    if (P.z[0]) put_z<T>(P, 0, row, col, n, v);
    if (P.act != kActNone) {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = act_f(P.act, v[q]);
    }
    if (P.add) {
      get4((const T*)P.add + row * P.ldadd + col, n, t);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = v[q] + t[q];
    }
    put4((T*)P.c[0] + row * P.ldc + col, n, v);
  } else if constexpr (FORM == kFormDx) {
    if (P.add) {
      float t[4];
      get4((const T*)P.add + row * P.ldadd + col, n, t);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = v[q] + t[q];
    }
    put4((T*)P.c[0] + row * P.ldc + col, n, v);
  } else {
    static_assert(FORM == kFormDw, "one matrix per call");
    void* c = seg ? P.c[1] : P.c[0];
    if (P.c_f32)
      put4((float*)c + row * P.ldc + col, n, v);
    else
      put4((T*)c + row * P.ldc + col, n, v);
  }
}

// g, u: columns col..col+3 of the two products
template <typename T>
DEV void emit4_glu(const DenseParams& P, int64_t row, int col, float (&g)[4], const float (&u)[4]) {
  const int n = P.N - col;
  if (P.z[0]) {
    put_z<T>(P, 0, row, col, n, g);
    put_z<T>(P, 1, row, col, n, u);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) g[q] = act_f(P.act, g[q]) * u[q];
  put4((T*)P.c[0] + row * P.ldc + col, n, g);
}

// chunk's partial of matrix seg; partial rows hold whole groups of four
DEV void part4(const DenseParams& P, int chunk, int seg, int64_t row, int col, const float (&v)[4]) {
  *(f32x4_t*)(P.part + ((int64_t)chunk * P.M + row) * P.part_ld + seg * P.part_seg + col) =
      f32x4_t{v[0], v[1], v[2], v[3]};
}

}  // namespace moedet
