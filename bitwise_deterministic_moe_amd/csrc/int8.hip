// Products in 8-bit integers with a scale for each row of x (token) and each row of
// the weights (output channel), for serving.
//
//   quantise   s = max |x| / 127 of the row (rounded to float32); code = the
//              whole number nearest to 127 x / max |x|, ties to even, decided exactly
//   product    y[m, n] = act(s_x[m] s_w[n] sum_k cx[m, k] cw[n, k] + bias[n]) + residual
//
// The sum is exact in int32, so its order and its split have no effect on the
// bits.  It is rounded to float32 once, and its products with the two scales once each.
//
// Tiles for many rows use the main loops of the bf16 operators (dense_bf16.h): a K
// slice of 64 bytes a row is 64 codes, the fragments are the same 16 bytes a
// lane, and v_mfma_i32_32x32x32_i8 takes the place of the bf16 instruction.
// Few rows stream the weights into registers.
#include "dense_bf16.h"
#include "dense_epilogue.h"
#include "int8.h"

namespace moedet {

// ------------------------------------------------------------------ quantising
namespace {

// The code of x, r about 127 / top.  With m = floor(|x| r), off by at most one where
// |x| r is next to a whole number, the code is m or m + 1 as 127 |x| - (m + 1/2) top is
// negative or positive, and the even one where it is 0 (x = top / 2 is such a
// tie: an ordinary value).  That difference is exact: 15 + 8 bits in float32 for
// bf16, 31 + 32 bits in float64 for float32.
template <typename T>
DEV int code_of(float x, float top, float r) {
  const float a = __builtin_fabsf(x), m = __builtin_floorf(a * r), h = m + 0.5f;
  int up, tie;
  if constexpr (sizeof(T) == 2) {
    const float d = __builtin_fmaf(-h, top, 127.f * a);
    up = d > 0.f;
    tie = d == 0.f;
  } else {
    const double d = __builtin_fma(-(double)h, (double)top, 127.0 * (double)a);
    up = d > 0.0;
    tie = d == 0.0;
  }
  const int i = (int)m, c = i + (up | (tie & i));
  return x < 0.f ? -c : c;
}
template <typename T>
DEV uint32_t pack4(const float* v, float top, float r) {
  uint32_t p = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) p |= ((uint32_t)code_of<T>(v[i], top, r) & 0xffu) << (8 * i);
  return p;
}
DEV uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Scale and reciprocal of a row whose largest magnitude has the bits `top`:
// a row with a number that is not finite gets a NaN scale and codes 0.
struct RowScale {
  float top, r, scale;
};
DEV RowScale row_scale(uint32_t bits) {
  const float t = __uint_as_float(bits);
  RowScale s{1.f, 0.f, 0.f};
  if (bits >= 0x7f800000u) {
    s.scale = __uint_as_float(0x7fc00000u);
  } else if (t >= kInt8Tiny) {
    s.top = t;
    s.r = 127.f / t;
    s.scale = t / 127.f;
  }
  return s;
}

}  // namespace

// L threads a row (64: four rows a workgroup; 256: one).  The first kQuantKeep
// vectors of a thread stay in registers between the two passes, the others are read again.
constexpr int kQuantKeep = 8;
template <typename T, int L>
__global__ __launch_bounds__(256) void int8_quantize_kernel(Int8QuantParams P) {
  constexpr int V = Vec<T>::N;
  __shared__ uint32_t s_top[4];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int R = 256 / L;
  const int64_t rows = P.limit ? min((int64_t)*P.limit, P.rows) : P.rows;
  const int64_t u = map_unit(blockIdx.x, (rows + R - 1) / R, P.seed);
  if (u < 0) return;
  const int64_t row = L == 64 ? u * 4 + w : u;
  if (row >= rows) return;               // L = 256: the whole workgroup
  const int v0 = L == 64 ? lane : (int)threadIdx.x;
  const T* x = (const T*)P.x + row * P.ldx;
  const int vecs = P.cols16 / V;
  typename Vec<T>::raw keep[kQuantKeep];
  uint32_t top = 0u;
  auto load = [&](int v) __attribute__((always_inline)) {
    const int n = P.cols - v * V;
    return n > 0 ? Vec<T>::load(x + (int64_t)v * V, n) : typename Vec<T>::raw{};
  };
  auto most = [&](const typename Vec<T>::raw& r) __attribute__((always_inline)) {
    float f[V];
    Vec<T>::get(r, f);
#pragma unroll
    for (int q = 0; q < V; ++q) top = max(top, magnitude(f[q]));
  };
#pragma unroll
  for (int i = 0; i < kQuantKeep; ++i)
    if (v0 + i * L < vecs) keep[i] = load(v0 + i * L);
#pragma unroll
  for (int i = 0; i < kQuantKeep; ++i)
    if (v0 + i * L < vecs) most(keep[i]);
  for (int v = v0 + kQuantKeep * L; v < vecs; v += L) most(load(v));
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
  if constexpr (L == 256) {
    if (lane == 0) s_top[w] = top;
    __syncthreads();
    top = max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3]));
  }
  const RowScale s = row_scale(top);
  int8_t* out = P.codes + row * P.cols16;
  auto put = [&](int v, const typename Vec<T>::raw& r) __attribute__((always_inline)) {
    float f[V];
    Vec<T>::get(r, f);
    if (s.r == 0.f) {
#pragma unroll
      for (int q = 0; q < V; ++q) f[q] = 0.f;
    }
    if constexpr (V == 8)
      *(u32x2_t*)(out + (int64_t)v * 8) = u32x2_t{pack4<T>(f, s.top, s.r), pack4<T>(f + 4, s.top, s.r)};
    else
      *(uint32_t*)(out + (int64_t)v * 4) = pack4<T>(f, s.top, s.r);
  };
#pragma unroll
  for (int i = 0; i < kQuantKeep; ++i) {
    if (v0 + i * L < vecs) put(v0 + i * L, keep[i]);
    __builtin_amdgcn_sched_barrier(0);   // one vector's registers at a time
  }
  for (int v = v0 + kQuantKeep * L; v < vecs; v += L) put(v, load(v));
  if (v0 == 0) P.scales[row] = s.scale;
}

hipError_t launch_int8_quantize(const Int8QuantParams& P, bool bf16, hipStream_t st) {
  const int V = bf16 ? 8 : 4;
  // a wave a row while it keeps the row in registers
  if (P.cols16 / V <= 64 * kQuantKeep) {
    const int64_t grid = grid_for_units((P.rows + 3) / 4);
    if (bf16)
      int8_quantize_kernel<uint16_t, 64><<<grid, 256, 0, st>>>(P);
    else
      int8_quantize_kernel<float, 64><<<grid, 256, 0, st>>>(P);
  } else {
    const int64_t grid = grid_for_units(P.rows);
    if (bf16)
      int8_quantize_kernel<uint16_t, 256><<<grid, 256, 0, st>>>(P);
    else
      int8_quantize_kernel<float, 256><<<grid, 256, 0, st>>>(P);
  }
  return hipGetLastError();
}

// Weights [rows][cols] along their rows, codes transposed: a workgroup takes 64
// columns of a matrix, once for their largest magnitudes and once more (from the
// caches) for the codes, which go through LDS so that a wave writes whole 64-byte runs.
// Weights are laid out once, so their two reads are left as they are.
template <typename T>
__global__ __launch_bounds__(512) void int8_quantize_t_kernel(Int8QuantTParams P) {
  constexpr int V = Vec<T>::N, C = 64, TPR = C / V, RPI = 512 / TPR;   // threads a row, rows a step
  __shared__ uint32_t s_top[C];
  __shared__ __attribute__((aligned(16))) int8_t s_codes[C][64 + 16];
  const int tid = threadIdx.x;
  const int64_t strips = (P.cols + C - 1) / C;
  const int64_t u = map_unit(blockIdx.x, P.batch * strips, P.seed);
  if (u < 0) return;
  const int64_t b = u / strips;
  const int c0 = (int)(u - b * strips) * C;
  const T* w = (const T*)P.w + b * P.rows * (int64_t)P.cols + c0;
  const int vc = (tid % TPR) * V, r0 = tid / TPR, n = P.cols - c0 - vc;   // columns that exist from this thread's first
  if (tid < C) s_top[tid] = 0u;
  __syncthreads();
  uint32_t top[V];
#pragma unroll
  for (int q = 0; q < V; ++q) top[q] = 0u;
  if (n > 0) {
#pragma unroll 4
    for (int r = r0; r < P.rows; r += RPI) {
      float f[V];
      Vec<T>::get(Vec<T>::load(w + (int64_t)r * P.cols + vc, n), f);
#pragma unroll
      for (int q = 0; q < V; ++q) top[q] = max(top[q], magnitude(f[q]));
    }
  }
#pragma unroll
  for (int q = 0; q < V; ++q) atomicMax(&s_top[vc + q], top[q]);
  __syncthreads();
  RowScale s[V];
#pragma unroll
  for (int q = 0; q < V; ++q) s[q] = row_scale(s_top[vc + q]);
  if (r0 == 0) {
#pragma unroll
    for (int q = 0; q < V; ++q)
      if (q < n) P.scales[b * P.cols + c0 + vc + q] = s[q].scale;
  }
  for (int rt = 0; rt < P.rows16; rt += 64) {
#pragma unroll
    for (int i = 0; i < 64; i += RPI) {
      const int r = r0 + i;
      if (RPI > 64 && r >= 64) continue;
      float f[V];
#pragma unroll
      for (int q = 0; q < V; ++q) f[q] = 0.f;
      if (n > 0 && rt + r < P.rows) Vec<T>::get(Vec<T>::load(w + (int64_t)(rt + r) * P.cols + vc, n), f);
#pragma unroll
      for (int q = 0; q < V; ++q) s_codes[vc + q][r] = (int8_t)code_of<T>(s[q].r == 0.f ? 0.f : f[q], s[q].top, s[q].r);
    }
    __syncthreads();
    const int c = tid >> 2, k = (tid & 3) * 16;
    if (tid < C * 4 && c0 + c < P.cols && rt + k < P.rows16)
      *(u32x4_t*)(P.codes + (b * P.cols + c0 + c) * (int64_t)P.rows16 + rt + k) = *(const u32x4_t*)&s_codes[c][k];
    __syncthreads();
  }
}

hipError_t launch_int8_quantize_t(const Int8QuantTParams& P, bool bf16, hipStream_t st) {
  const int64_t grid = grid_for_units(P.batch * ((P.cols + 63) / 64));
  if (bf16)
    int8_quantize_t_kernel<uint16_t><<<grid, 512, 0, st>>>(P);
  else
    int8_quantize_t_kernel<float><<<grid, 512, 0, st>>>(P);
  return hipGetLastError();
}

// ----------------------------------------------------------------------- units
namespace {

struct Int8Tile {
  int g;            // group
  int64_t m0;       // first row
  int rows;         // rows of the tile that exist
  int n0;
};

// The tile of this workgroup, BM x bn.  One group: bands of four tile rows, down the
// band before across, so that the consecutive units of an XCD share both operands.
// Groups: one after the other, down the group's tile rows before across, so that the
// units that read one strip of weights follow each other; each workgroup
// counts the groups' tiles itself from the offsets, which costs less than a launch.
// Offsets are clamped to 0..M, and a launch that they would make larger than ascending
// ones can does nothing, so that no row outside the matrices is touched whatever
// they hold.  NT threads; s: 8 + NT / 64 words of LDS.
template <bool GROUPS, int NT>
DEV bool int8_tile(const Int8Params& P, int bm, int bn, int* s, Int8Tile& t) {
  const uint32_t nT = (uint32_t)((P.d.N + bn - 1) / bn);
  if constexpr (!GROUPS) {
    constexpr uint32_t kBand = 4;
    const uint32_t mT = (uint32_t)((P.d.M + bm - 1) / bm);
    const int64_t unit = map_unit(blockIdx.x, (int64_t)mT * nT, P.d.seed);
    if (unit < 0) return false;
    const uint32_t L = (uint32_t)unit;
    const uint32_t band = L / (kBand * nT), in = L - band * kBand * nT;
    const uint32_t left = mT - band * kBand, h = left < kBand ? left : kBand;
    t.g = 0;
    t.m0 = (int64_t)(band * kBand + in % h) * bm;
    t.n0 = (int)(in / h) * bn;
    t.rows = (int)(P.d.M - t.m0 < bm ? P.d.M - t.m0 : bm);
    return true;
  } else {
    constexpr int PER = (kInt8MaxGroups + NT - 1) / NT;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int g0 = tid * PER;
    const int64_t M = P.d.M;
    int at[PER + 1], n[PER];
    uint32_t own = 0;
#pragma unroll
    for (int i = 0; i <= PER; ++i) at[i] = P.offsets[min(g0 + i, P.groups)];
#pragma unroll
    for (int i = 0; i <= PER; ++i) at[i] = (int)min((int64_t)max(at[i], 0), M);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int rows = g0 + i < P.groups ? max(at[i + 1] - at[i], 0) : 0;
      n[i] = min((int)(((uint32_t)rows + bm - 1) / bm), (1 << 24) - 1);   // sums over a wave stay below 2^32
      own += n[i];
    }
    uint32_t incl = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = __shfl_up(incl, d, 64);
      if (lane >= d) incl += o;
    }
    if (lane == 63) s[8 + w] = (int)incl;
    __syncthreads();
    uint64_t base = 0, total = 0;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) {
      const uint32_t v = (uint32_t)s[8 + i];
      base += i < w ? v : 0u;
      total += v;
    }
    if (total * nT > gridDim.x) return false;
    const int64_t unit = map_unit(blockIdx.x, (int64_t)(total * nT), P.d.seed);
    if (unit < 0) return false;            // uniform
    const int L = (int)((uint32_t)unit / nT);
    int pre = (int)((uint32_t)base + incl - own);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (L >= pre && L < pre + n[i]) {
        s[0] = g0 + i;
        s[1] = at[i];
        s[2] = at[i + 1] - at[i];
        s[3] = pre;
        s[4] = n[i];
      }
      pre += n[i];
    }
    __syncthreads();
    t.g = __builtin_amdgcn_readfirstlane(s[0]);
    const int first = __builtin_amdgcn_readfirstlane(s[1]), rows = __builtin_amdgcn_readfirstlane(s[2]);
    const uint32_t in = (uint32_t)unit - (uint32_t)__builtin_amdgcn_readfirstlane(s[3]) * nT;
    const uint32_t h = (uint32_t)__builtin_amdgcn_readfirstlane(s[4]);
    const int m = (int)(in % h) * bm;
    t.m0 = first + m;
    t.n0 = (int)(in / h) * bn;
    t.rows = min(rows - m, bm);
    __syncthreads();                       // s may be the main loop's LDS
    return true;
  }
}

// Scales (and bias, added) of four columns: v = v sb + bias.
template <typename T>
struct Cols4 {
  float sb[4], bias[4];
  DEV void load(const Int8Params& P, int g, int col) {
    const int n = P.d.N - col;
#pragma unroll
    for (int q = 0; q < 4; ++q) sb[q] = bias[q] = 0.f;
    if (n <= 0) return;
    get4(P.sb + (int64_t)g * P.d.N + col, n, sb);
    if (P.d.bias) get4((const T*)P.d.bias + (int64_t)g * P.d.N + col, n, bias);
  }
};

}  // namespace

// ----------------------------------------------------------------------- tiles
constexpr int kInt8StageRow = 260;

template <typename T, int WTM, bool GROUPS>
__global__ __launch_bounds__(256) void int8_tile_kernel(Int8Params P) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[dn::kRingBytes<WTM> / 2];
  constexpr int BM = 2 * WTM;
  static_assert(64 * kInt8StageRow * 4 <= dn::kRingBytes<WTM>, "epilogue stage must fit in the ring");
  Int8Tile t;
  if (!int8_tile<GROUPS, 256>(P, BM, 256, (int*)lds, t)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, r32 = lane & 31, half = lane >> 5;
  const uint32_t ring = bf::lds_base(lds);
  constexpr int LA = dn::kALoads<WTM>;
  constexpr uint32_t AB = dn::kAOper<WTM> * 2;
  const int nvalid = P.d.N - t.n0 < 256 ? P.d.N - t.n0 : 256;
  // pairs of codes as 16-bit elements
  const int64_t K2 = P.d.K / 2, lda = P.lda / 2;
  const int nsteps = (int)((K2 + dn::BK - 1) / dn::BK);
  const int kc = dn::KcOp<LA>::chunk(lane) * 8;
  dn::KcOp<LA> oa;
  dn::KcOp<4> ob;
  oa.init(P.a + t.m0 * P.lda, ((t.rows - 1) * lda + K2) * 2, wave, lane, t.rows, lda);
  ob.init(P.b + ((int64_t)t.g * P.d.N + t.n0) * P.d.K, ((nvalid - 1) * K2 + K2) * 2, wave, lane, nvalid, K2);
  i32x16_t acc[4][4];
  dn::mainloop<dn::KC, dn::KC, WTM>(ring, nsteps, [&](int s, uint32_t st, int i) {
    const bool live = s < nsteps;
    const int ks = live ? s : 0;
    const bool ok = live && ks * dn::BK + kc < K2;
    if (i < LA)
      oa.issue(st, wave, i, ok, (uint32_t)ks * 64u);
    else
      ob.issue(st + AB, wave, i - LA, ok, (uint32_t)ks * 64u);
  }, acc, wm, wn, lane);
  Cols4<T> c4;
  const int col = t.n0 + lane * 4;
  c4.load(P, t.g, col);
  // The sums go through LDS in passes of 64 rows, so that a wave writes whole rows
  // (and a row's scale is a scalar).  They are converted behind it: in front, the
  // compiler converts all of them at once and spills.
  int* stage = (int*)lds;
  const int64_t end = t.m0 + t.rows;
#pragma unroll 1
  for (int p = 0; 64 * p < t.rows; ++p) {
#pragma unroll
    for (int q = 0; q < 2 * WTM / 64; ++q) {
      if (p != q) continue;
#pragma unroll
      for (int mb = 0; mb < WTM / 32; ++mb) {
        const int r0 = wm * WTM + mb * 32 - 64 * q;
        if (r0 < 0 || r0 >= 64) continue;
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const i32x16_t& a = acc[mb][nb];
            *(i32x4_t*)(stage + (r0 + r32) * kInt8StageRow + wn * 128 + nb * 32 + 8 * i + 4 * half) =
                i32x4_t{a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]};
          }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int st = 0; st < 16; st += 4) {
      float v[16];
      const int m = 4 * st + wave;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const i32x4_t sv = *(const i32x4_t*)(stage + (m + 4 * i) * kInt8StageRow + lane * 4);
        const float sa = P.sa[min(t.m0 + 64 * p + m + 4 * i, end - 1)];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[4 * i + q] = __builtin_fmaf((float)sv[q] * sa, c4.sb[q], c4.bias[q]);
      }
      if (col >= P.d.N) continue;
      emit<T, kFormLinear, 4, true, true>(P.d, 0, AtRows{t.m0 + 64 * p + m, end, 4, col}, v);
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
}

template <typename T, int MB, int NB, bool GROUPS>
__global__ __launch_bounds__(256) void int8_small_kernel(Int8Params P) {
  using S = dn::Small<MB, NB, false>;
  constexpr int BM = 64 * MB, BN = 64 * NB, ROW = 64 * NB + 4;
  static_assert(BM * ROW * 4 <= S::RING, "epilogue stage must fit in the ring");
  __shared__ __attribute__((aligned(16))) uint16_t lds[S::RING / 2];
  Int8Tile t;
  if (!int8_tile<GROUPS, 256>(P, BM, BN, (int*)lds, t)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const uint32_t ring = bf::lds_base(lds), own = (uint32_t)wave * 1024u;
  const int nvalid = P.d.N - t.n0 < BN ? P.d.N - t.n0 : BN;
  const int64_t K2 = P.d.K / 2, lda = P.lda / 2;
  const int nsteps = (int)((K2 + dn::SBK - 1) / dn::SBK);
  const int kc = dn::KcOp<1>::chunk(lane) * 8;
  dn::KcPart<MB> oa;
  dn::KcPart<NB> ob;
  oa.init(P.a + t.m0 * P.lda, ((t.rows - 1) * lda + K2) * 2, wave, lane, t.rows, lda);
  ob.init(P.b + ((int64_t)t.g * P.d.N + t.n0) * P.d.K, nvalid * K2 * 2, wave, lane, nvalid, K2);
  i32x16_t acc[MB][NB];
  dn::small_mainloop<dn::KC, dn::KC, MB, NB, false>(ring, nsteps, [&](int h, uint32_t at, int i) {
    const bool live = h < 2 * nsteps;
    const int ks = live ? h : 0;
    const bool ok = live && ks * dn::BK + kc < K2;
    if (i < MB)
      bf::dma16(oa.rs, at + own, ok ? oa.voff[i < MB ? i : 0] : dn::kOOB, (uint32_t)ks * 64u);
    else
      bf::dma16(ob.rs, at + own, ok ? ob.voff[i < MB ? 0 : i - MB] : dn::kOOB, (uint32_t)ks * 64u);
  }, acc, wm, wn, lane);
  // through LDS, so that 16 lanes write 64 columns of a row
  float* stage = (float*)lds;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int m = mb * 64 + wm * 32 + (lane & 31);
    const float sa = P.sa[t.m0 + min(m, t.rows - 1)];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const i32x16_t& a = acc[mb][n];
        *(f32x4_t*)(stage + m * ROW + 64 * n + wn * 32 + 8 * i + 4 * (lane >> 5)) =
            f32x4_t{(float)a[4 * i] * sa, (float)a[4 * i + 1] * sa, (float)a[4 * i + 2] * sa, (float)a[4 * i + 3] * sa};
      }
  }
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  const int c = (lane & 15) * 4, m = 4 * wave + (lane >> 4);
#pragma unroll 1
  for (int n = 0; n < NB; ++n) {
    const int col = t.n0 + 64 * n + c;
    if (col >= P.d.N) continue;
    Cols4<T> c4;
    c4.load(P, t.g, col);
#pragma unroll 1
    for (int mb = 0; mb < MB; ++mb) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4_t sv = *(const f32x4_t*)(stage + (mb * 64 + m + 16 * i) * ROW + 64 * n + c);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[4 * i + q] = __builtin_fmaf(sv[q], c4.sb[q], c4.bias[q]);
      }
      emit<T, kFormLinear, 4, false, true>(P.d, 0, AtRows{t.m0 + mb * 64 + m, t.m0 + t.rows, 16, col}, v);
    }
  }
}

// -------------------------------------------------------------------- few rows
// A workgroup streams 16 weight rows: its 8 waves take steps of 64 codes in turn,
// so that together they read 512 bytes of a row, and multiply each with MT
// blocks of 16 rows of x (v_mfma_i32_16x16x64_i8; a lane's 16 bytes of both operands
// come straight from memory, those of x from the caches).  The waves' sums meet in
// LDS.  A lane ends with four neighbouring columns of one row.
constexpr int kFewWaves = 8, kFewDepth = 4;
template <typename T, int MT, bool GROUPS>
__global__ __launch_bounds__(64 * kFewWaves) void int8_few_kernel(Int8Params P) {
  __shared__ __attribute__((aligned(16))) i32x4_t s_acc[kFewWaves * MT * 64];
  Int8Tile t;
  if (!int8_tile<GROUPS, 64 * kFewWaves>(P, 16 * MT, 16, (int*)s_acc, t)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int K = (int)P.d.K, steps = (K + 63) / 64;
  const int8_t* w = P.b + ((int64_t)t.g * P.d.N + min(t.n0 + i16, P.d.N - 1)) * P.d.K;
  const int8_t* x[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) x[m] = P.a + (t.m0 + min(16 * m + i16, t.rows - 1)) * P.lda;
  i32x4_t acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = i32x4_t{0, 0, 0, 0};
  struct Step {
    i32x4_t w, x[MT];
  };
  // past the end of the rows: their last 16 codes again, and zeros for x
  auto load = [&](Step& f, int s) __attribute__((always_inline)) {
    const int k = 64 * s + 16 * g, kk = min(k, K - 16);
    f.w = *(const i32x4_t*)(w + kk);
#pragma unroll
    for (int m = 0; m < MT; ++m) f.x[m] = *(const i32x4_t*)(x[m] + kk);
  };
  auto mul = [&](const Step& f, int s) __attribute__((always_inline)) {
    const bool in = 64 * s + 16 * g < K;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      i32x4_t v = f.x[m];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = in ? v[q] : 0;
      acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.w, v, acc[m], 0, 0, 0);
    }
  };
  // rounds of kFewDepth steps, the next round's loads in flight
  Step st[kFewDepth];
#pragma unroll
  for (int d = 0; d < kFewDepth; ++d) load(st[d], wave + d * kFewWaves);
#pragma unroll 1
  for (int s = wave; s < steps; s += kFewDepth * kFewWaves) {
#pragma unroll
    for (int d = 0; d < kFewDepth; ++d) {
      mul(st[d], s + d * kFewWaves);
      load(st[d], s + (kFewDepth + d) * kFewWaves);
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) s_acc[(wave * MT + m) * 64 + lane] = acc[m];
  __syncthreads();
  if (tid >= 64 * MT) return;
  i32x4_t a = s_acc[tid];
#pragma unroll
  for (int v = 1; v < kFewWaves; ++v) a = a + s_acc[v * MT * 64 + tid];
  const int row = (tid >> 6) * 16 + i16, col = t.n0 + 4 * g;
  if (row >= t.rows || col >= P.d.N) return;
  const float sa = P.sa[t.m0 + row];
  Cols4<T> c4;
  c4.load(P, t.g, col);
  float v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = __builtin_fmaf((float)a[q] * sa, c4.sb[q], c4.bias[q]);
  emit<T, kFormLinear, 1, false, true>(P.d, 0, AtRows{t.m0 + row, t.m0 + row + 1, 1, col}, v);
}

// --------------------------------------------------------------------- launches
namespace {

// Workgroups of a launch: with groups, as many as any offsets can need.
int64_t int8_grid(const Int8Params& P, int bm, int bn) {
  const int64_t nT = (P.d.N + bn - 1) / bn;
  int64_t mT = (P.d.M + bm - 1) / bm;
  if (P.offsets) {
    mT = P.d.M / bm + P.groups;
    if (mT > P.d.M) mT = P.d.M;
  }
  return grid_for_units(mT * nT);
}

template <typename T, bool GROUPS>
void tiles(const Int8Params& P, int tile, hipStream_t st) {
  const DenseShape sh = dense_shape(kFormLinear, true, tile);
  const dim3 grid((uint32_t)int8_grid(P, sh.bm, sh.bn));
  switch (tile) {
    case 0: int8_tile_kernel<T, 128, GROUPS><<<grid, 256, 0, st>>>(P); break;
    case 1: int8_tile_kernel<T, 64, GROUPS><<<grid, 256, 0, st>>>(P); break;
    case 2: int8_small_kernel<T, 2, 2, GROUPS><<<grid, 256, 0, st>>>(P); break;
    default: int8_small_kernel<T, 1, 1, GROUPS><<<grid, 256, 0, st>>>(P);
  }
}
template <typename T, bool GROUPS>
void few(const Int8Params& P, int mt, hipStream_t st) {
  const dim3 grid((uint32_t)int8_grid(P, 16 * mt, 16));
  if (mt == 1)
    int8_few_kernel<T, 1, GROUPS><<<grid, 64 * kFewWaves, 0, st>>>(P);
  else
    int8_few_kernel<T, 2, GROUPS><<<grid, 64 * kFewWaves, 0, st>>>(P);
}

}  // namespace

hipError_t launch_int8_tiles(const Int8Params& P, bool bf16, int tile, hipStream_t st) {
  if (bf16)
    P.offsets ? tiles<uint16_t, true>(P, tile, st) : tiles<uint16_t, false>(P, tile, st);
  else
    P.offsets ? tiles<float, true>(P, tile, st) : tiles<float, false>(P, tile, st);
  return hipGetLastError();
}

hipError_t launch_int8_few(const Int8Params& P, bool bf16, int mt, hipStream_t st) {
  if (bf16)
    P.offsets ? few<uint16_t, true>(P, mt, st) : few<uint16_t, false>(P, mt, st);
  else
    P.offsets ? few<float, true>(P, mt, st) : few<float, false>(P, mt, st);
  return hipGetLastError();
}

}  // namespace moedet
