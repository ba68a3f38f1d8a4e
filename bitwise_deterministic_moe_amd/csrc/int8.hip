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
// Tiles for many rows copy both operands by DMA into a ring of LDS slots and feed
// v_mfma_i32_32x32x32_i8; few rows stream the weights into registers.
#include <type_traits>

#include "dense_epilogue.h"
#include "gemm_bf16.h"
#include "int8.h"

namespace moedet {

// ------------------------------------------------------------------ quantising
namespace {

// Codes of bf16 numbers: fma(x, r, 1.5 2^23) is the whole number nearest to x r, ties to
// even, in its low bits, and for r = 127 / top rounded up it is the nearest to
// 127 x / top, as x = X u and top = A 2^d u with X, A of 8 bits show:
//   a quotient that is no tie is at least 1 / (254 X) > 2^-16 of its value away from
//   one, and x r is off by at most 2^-23 of it;
//   a tie is 254 X = (2 m + 1) A 2^d, and 127 divides 2 m + 1 or A.  In the first case
//   x = top / 2, whose code is 64: x r >= 63.5 gives that.  In the second A = 254, r
//   is a power of two, and x r is exact.
//
// Codes of float32 numbers: with m = floor(|x| r), off by at most one where
// |x| r is next to a whole number, the code is m or m + 1 as 127 |x| - (m + 1/2) top is
// negative or positive, and the even one where it is 0; the difference is exact in
// float64 (31 + 32 bits).
DEV int code_f32(float x, float top, float r) {
  const float a = __builtin_fabsf(x), m = __builtin_floorf(a * r), h = m + 0.5f;
  const double d = __builtin_fma(-(double)h, (double)top, 127.0 * (double)a);
  const int up = d > 0.0, tie = d == 0.0, i = (int)m, c = i + (up | (tie & i));
  return x < 0.f ? -c : c;
}
template <typename T>
DEV uint32_t code_bits(float x, float top, float r) {   // the code in the low byte
  if constexpr (sizeof(T) == 2) return __float_as_uint(__builtin_fmaf(x, r, 0x1.8p23f));
  return (uint32_t)code_f32(x, top, r);
}
template <typename T>
DEV uint32_t pack4(const float* v, float top, float r) {
  const uint32_t lo = __builtin_amdgcn_perm(code_bits<T>(v[1], top, r), code_bits<T>(v[0], top, r), 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(code_bits<T>(v[3], top, r), code_bits<T>(v[2], top, r), 0x04000c0cu);
  return lo | hi;
}
DEV uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Largest magnitude of a vector, as float32 bits.
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
DEV uint32_t magnitude(const u32x4_t& v) {
  u16x2_t m = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, v[i] & 0x7fff7fffu));
  return (uint32_t)max(m[0], m[1]) << 16;
}
DEV uint32_t magnitude(const f32x4_t& v) {
  return max(max(magnitude(v[0]), magnitude(v[1])), max(magnitude(v[2]), magnitude(v[3])));
}

// Scale and reciprocal (rounded up) of a row whose largest magnitude has the bits
// `top`.  A row of zeros, of numbers below kInt8Tiny, or with one that is not finite
// has r = 0, which makes every code 0 if its numbers are taken as 0 (clean).
struct RowScale {
  float top, r, scale;
  DEV float clean(float v) const { return r == 0.f ? 0.f : v; }
};
DEV RowScale row_scale(uint32_t bits) {
  const float t = __uint_as_float(bits);
  RowScale s{1.f, 0.f, 0.f};
  if (bits >= 0x7f800000u) {
    s.scale = __uint_as_float(0x7fc00000u);
  } else if (t >= kInt8Tiny) {
    s.top = t;
    s.r = 127.f / t;
    if (__builtin_fmaf(s.r, t, -127.f) < 0.f) s.r = __uint_as_float(__float_as_uint(s.r) + 1u);
    s.scale = t / 127.f;
  }
  return s;
}

// The codes of a vector.
template <typename T>
DEV void put_codes(int8_t* out, const typename Vec<T>::raw& v, const RowScale& s) {
  float f[Vec<T>::N];
  Vec<T>::get(v, f);
#pragma unroll
  for (int q = 0; q < Vec<T>::N; ++q) f[q] = s.clean(f[q]);
  if constexpr (sizeof(T) == 2)
    *(u32x2_t*)out = u32x2_t{pack4<T>(f, s.top, s.r), pack4<T>(f + 4, s.top, s.r)};
  else
    *(uint32_t*)out = pack4<T>(f, s.top, s.r);
}

}  // namespace

// L threads a row (64: four rows a workgroup; 256: one).  The first kQuantKeep
// vectors of a thread stay in registers between the two passes, the others are read again.
// Bound by HBM where rows are many: 16384 x 2048 bf16 21.6 to 24.7 us (4.1 to 4.7 TB/s), 4096 x
// 2048 7.3, of it 2 the launch.
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
#pragma unroll
  for (int i = 0; i < kQuantKeep; ++i)
    if (v0 + i * L < vecs) keep[i] = load(v0 + i * L);
#pragma unroll
  for (int i = 0; i < kQuantKeep; ++i)
    if (v0 + i * L < vecs) top = max(top, magnitude(keep[i]));
  for (int v = v0 + kQuantKeep * L; v < vecs; v += L) top = max(top, magnitude(load(v)));
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
  if constexpr (L == 256) {
    if (lane == 0) s_top[w] = top;
    __syncthreads();
    top = max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3]));
  }
  const RowScale s = row_scale(top);
  int8_t* out = P.codes + row * P.cols16;
#pragma unroll
  for (int i = 0; i < kQuantKeep; ++i) {
    if (v0 + i * L < vecs) put_codes<T>(out + (int64_t)(v0 + i * L) * V, keep[i], s);
    __builtin_amdgcn_sched_barrier(0);   // one vector's registers at a time
  }
  for (int v = v0 + kQuantKeep * L; v < vecs; v += L) put_codes<T>(out + (int64_t)v * V, load(v), s);
  if (v0 == 0) P.scales[row] = s.scale;
}

// A wave a row while it keeps the row in registers (several rows a wave are no faster: 4096 x
// 2048 bf16 7.3 us, 8.0 with four).
static bool wave_a_row(int cols16, bool bf16) { return cols16 / (bf16 ? 8 : 4) <= 64 * kQuantKeep; }
int64_t int8_quantize_grid(int64_t rows, int cols16, bool bf16) { return grid_for_units(wave_a_row(cols16, bf16) ? (rows + 3) / 4 : rows); }

hipError_t launch_int8_quantize(const Int8QuantParams& P, bool bf16, hipStream_t st) {
  const bool wave = wave_a_row(P.cols16, bf16);
  const int64_t grid = int8_quantize_grid(P.rows, P.cols16, bf16);
  if (wave) {
    if (bf16)
      int8_quantize_kernel<uint16_t, 64><<<grid, 256, 0, st>>>(P);
    else
      int8_quantize_kernel<float, 64><<<grid, 256, 0, st>>>(P);
  } else {
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
// Weights are laid out once, so their two reads are left as they are (64 matrices of 2048 x
// 2048 bf16 301 us, 2.7 TB/s counted once; one of 2048 x 8192 39, by 128 workgroups).
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
      for (int q = 0; q < V; ++q) s_codes[vc + q][r] = (int8_t)code_bits<T>(s[q].clean(f[q]), s[q].top, s[q].r);
    }
    __syncthreads();
    const int c = tid >> 2, k = (tid & 3) * 16;
    if (tid < C * 4 && c0 + c < P.cols && rt + k < P.rows16)
      *(u32x4_t*)(P.codes + (b * P.cols + c0 + c) * (int64_t)P.rows16 + rt + k) = *(const u32x4_t*)&s_codes[c][k];
    __syncthreads();
  }
}

int64_t int8_quantize_t_grid(int64_t batch, int cols) { return grid_for_units(batch * ((cols + 63) / 64)); }

hipError_t launch_int8_quantize_t(const Int8QuantTParams& P, bool bf16, hipStream_t st) {
  const int64_t grid = int8_quantize_t_grid(P.batch, P.cols);
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
  int chunk;        // one group: the chunk of the contraction
};

// The group and tile row of unit L of a launch, by one wave for itself: lane l counts
// the tile rows of groups PER l .. PER l + PER - 1.
// Offsets are clamped to 0..M, and a launch that they would make larger than ascending
// ones can does nothing, so that no row outside the matrices is touched whatever
// they hold.
template <int PER>
DEV bool group_tile(const Int8Params& P, int bm, int bn, uint32_t nT, Int8Tile& t) {
  const int lane = threadIdx.x & 63, g0 = lane * PER;
  int at[PER + 1];
  uint32_t n[PER], own = 0;
#pragma unroll
  for (int i = 0; i <= PER; ++i) at[i] = P.offsets[min(g0 + i, P.groups)];
#pragma unroll
  for (int i = 0; i <= PER; ++i) at[i] = (int)min((int64_t)max(at[i], 0), P.d.M);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t rows = g0 + i < P.groups ? (uint32_t)max(at[i + 1] - at[i], 0) : 0u;
    n[i] = min((rows + bm - 1) / bm, 1u << 24);
    own += n[i];
  }
  own = min(own, 1u << 25);   // 64 lanes stay below 2^32; ascending offsets below 2^24
  uint32_t incl = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(incl, d, 64);
    if (lane >= d) incl += o;
  }
  const uint32_t total = (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
  if ((uint64_t)total * nT > gridDim.x) return false;
  const int64_t unit = map_unit(blockIdx.x, (int64_t)total * nT, P.d.seed);
  if (unit < 0) return false;
  const uint32_t L = (uint32_t)unit / nT;
  // the lane whose groups hold tile row L, and the group among its own
  const int who = __popcll(__ballot(incl <= L));
  uint32_t pre = incl - own, h = 0;
  int g = 0, first = 0, rows = 0;
  bool found = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (!found && L < pre + n[i]) {
      found = true;
      g = g0 + i;
      first = at[i];
      rows = at[i + 1] - at[i];
      h = n[i];
    }
    if (!found) pre += n[i];
  }
  t.g = __builtin_amdgcn_readlane(g, who);
  const uint32_t hh = (uint32_t)__builtin_amdgcn_readlane((int)h, who);
  const uint32_t in = (uint32_t)unit - (uint32_t)__builtin_amdgcn_readlane((int)pre, who) * nT;
  const int m = (int)(in % hh) * bm;
  t.m0 = __builtin_amdgcn_readlane(first, who) + m;
  t.n0 = (int)(in / hh) * bn;
  t.rows = min(__builtin_amdgcn_readlane(rows, who) - m, bm);
  t.chunk = 0;
  return true;
}

// The tile of this workgroup, BM x bn.  One group: bands of four tile rows, down the
// band before across, so that the consecutive units of an XCD share both operands,
// and all chunks of a tile one after the other.  Groups: one after the other, down the
// group's tile rows before across, so that the units that read one strip of
// weights follow each other; every wave finds its group from the offsets itself, which
// costs less than a launch, and without a barrier less than once a workgroup.
template <bool GROUPS>
DEV bool int8_tile(const Int8Params& P, int bm, int bn, Int8Tile& t) {
  const uint32_t nT = (uint32_t)((P.d.N + bn - 1) / bn);
  if constexpr (!GROUPS) {
    constexpr uint32_t kBand = 4;
    const uint32_t mT = (uint32_t)((P.d.M + bm - 1) / bm), S = (uint32_t)P.d.S;
    const int64_t unit = map_unit(blockIdx.x, (int64_t)mT * nT * S, P.d.seed);
    if (unit < 0) return false;
    const uint32_t L = (uint32_t)unit / S;
    t.chunk = (int)((uint32_t)unit - L * S);
    const uint32_t band = L / (kBand * nT), in = L - band * kBand * nT;
    const uint32_t left = mT - band * kBand, h = left < kBand ? left : kBand;
    t.g = 0;
    t.m0 = (int64_t)(band * kBand + in % h) * bm;
    t.n0 = (int)(in / h) * bn;
    t.rows = (int)(P.d.M - t.m0 < bm ? P.d.M - t.m0 : bm);
    return true;
  } else {
    if (P.groups <= 64) return group_tile<1>(P, bm, bn, nT, t);
    if (P.groups <= 256) return group_tile<4>(P, bm, bn, nT, t);
    return group_tile<kInt8MaxGroups / 64>(P, bm, bn, nT, t);
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
// Tiles of 64 MB x 64 NB: 4 waves in a 2 x 2 grid, each 32 MB x 32 NB as blocks of
// v_mfma_i32_32x32x32_i8.
//
// K slices are 128 codes, so that a row's slice is one whole 128-byte line: the L2s serve
// requests, and lines asked for in halves cost two.  (Copies alone, every CU reading
// panels of 128 and 256 rows of 2 to 8 KB: 17.6 TB/s in pieces of 64 bytes, 25 in lines.
// 4096 x 2048 x 8192 in tiles of 128 x 128: 75 and 70 us.)
// In LDS a row is 128 bytes, and its 16-byte chunk c sits at c ^ ((row >> 1) & 7): the 16
// lanes that one cycle of a ds_read_b128 serves then cover all 64 banks (no bank
// conflicts counted in the loop).
//
// A ring of NS slots.  A slice is multiplied in four quarters of 32 codes, the fragments
// of the next quarter being read meanwhile; before the last one the wave waits for its own loads
// of slice s + 1 and for its reads of slice s and meets the other waves, then reads the first
// quarter of slice s + 1 and loads slice s + NS into the slot of slice s.
namespace line {
constexpr int BK = 128;
template <int MB, int NB>
constexpr uint32_t kSlot = (uint32_t)(MB + NB) * 8192u;   // bytes: A, then B

DEV int swz(int row) { return (row >> 1) & 7; }

// An operand's loads: load i of wave w covers tile rows 8 (w NL + i) .. + 7.
template <int NL>
struct Op {
  bf::i32x4_t rs;
  uint32_t voff[NL];
  DEV void init(const void* base, int64_t extent, int wave, int lane, int valid, int64_t ld) {
    rs = bf::make_rsrc(base, (uint32_t)extent);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int row = 8 * (wave * NL + i) + (lane >> 3);
      voff[i] = row < valid ? (uint32_t)(row * ld) + (uint32_t)((lane & 7) ^ swz(row)) * 16u : bf::kOOB;
    }
  }
};
// First code of a slice that this lane loads in even and in odd loads (NL is even).
DEV int first_code(int lane, int odd) { return ((lane & 7) ^ swz(8 * odd + (lane >> 3))) * 16; }

// issue(s, addr, i): load i (those of A, then of B) of slice s into the slot at addr; slices
// at or past nsteps must read zeros (their loads keep the count of outstanding ones).
template <int MB, int NB, int NS, class Issue>
DEV void mainloop(uint32_t ring, int nsteps, Issue issue, i32x16_t (&acc)[MB][NB], int wm, int wn, int lane) {
  constexpr int L = 2 * (MB + NB), R = MB + NB, M = MB * NB;
  constexpr uint32_t SB = kSlot<MB, NB>;
  // Loads issued in the last quarter; the others in the first one of the next slice.  All of
  // them at once are as good where a quarter is short (8192^3 in tiles of 128 x 128 552 us,
  // 568 spread; of 256 x 256 6 us more at once).
  constexpr int LAST = M >= 16 ? L / 2 : L;
  uint32_t aa[4], ba[4];
  {
    const int ra = wm * 32 * MB + (lane & 31), rb = wn * 32 * NB + (lane & 31), half = lane >> 5;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      aa[q] = ring + (uint32_t)(ra * 128 + (((2 * q + half) ^ swz(ra)) << 4));
      ba[q] = ring + (uint32_t)MB * 8192u + (uint32_t)(rb * 128 + (((2 * q + half) ^ swz(rb)) << 4));
    }
  }
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int i = 0; i < L; ++i) issue(s, ring + s * SB, i);
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[m][n][r] = 0;
  struct Frag {
    i32x4_t a[MB], b[NB];
  } f[2];
  // fragment j (those of A, then of B) of quarter q in slot sl
  auto read = [&](Frag& g, int q, int sl, int j) __attribute__((always_inline)) {
    const bool isa = j < MB;
    const LDS_AS char* p = (const LDS_AS char*)(uintptr_t)((isa ? aa[q] : ba[q]) + (uint32_t)sl * SB);
    const i32x4_t v = *(const LDS_AS i32x4_t*)(p + (isa ? j : j - MB) * 4096);
    if (isa)
      g.a[isa ? j : 0] = v;
    else
      g.b[isa ? 0 : j - MB] = v;
  };
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((NS - 1) * L) : "memory");
#pragma unroll
  for (int j = 0; j < R; ++j) read(f[0], 0, 0, j);
  auto step = [&](int s, int sl) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q == 3) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NS - 2) * L) : "memory");
#pragma unroll
      for (int j = 0; j < M; ++j) {
#pragma unroll
        for (int k = j * R / M; k < (j + 1) * R / M; ++k) {
          if (q < 3)
            read(f[(q + 1) & 1], q + 1, sl, k);
          else
            read(f[0], 0, (sl + 1) % NS, k);
        }
        __builtin_amdgcn_sched_barrier(0);
        acc[j / NB][j % NB] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f[q & 1].b[j % NB], f[q & 1].a[j / NB], acc[j / NB][j % NB], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        if (q == 3) {
#pragma unroll
          for (int k = j * LAST / M; k < (j + 1) * LAST / M; ++k) issue(s + NS, ring + sl * SB, k);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (LAST < L && q == 0 && s > 0) {
#pragma unroll
          for (int k = j * (L - LAST) / M; k < (j + 1) * (L - LAST) / M; ++k)
            issue(s - 1 + NS, ring + (sl + NS - 1) % NS * SB, LAST + k);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  };
  int s = 0;
#pragma unroll 1
  for (; s + NS <= nsteps; s += NS) {
#pragma unroll
    for (int j = 0; j < NS; ++j) step(s + j, j);
  }
#pragma unroll
  for (int j = 0; j < NS - 1; ++j)
    if (s + j < nsteps) step(s + j, j);
  bf::block_barrier();
}
}  // namespace line

// Row scales, column scales and bias of a tile of up to 256 x 256: thread i holds
// those of row i and column i from before the main loop, and puts them into LDS
// behind it.  (Loaded where they are used, they cost a 256 x 256 tile 3.5 us.)
struct TileScales {
  float sa, sb, bias;
  template <typename T>
  DEV void load(const Int8Params& P, const Int8Tile& t, int tid) {
    sa = P.sa[t.m0 + min(tid, t.rows - 1)];
    const int64_t col = (int64_t)t.g * P.d.N + min(t.n0 + tid, P.d.N - 1);
    sb = P.sb[col];
    bias = 0.f;
    if (P.d.bias) bias = sizeof(T) == 2 ? bf16_to_f32(((const uint16_t*)P.d.bias)[col]) : ((const float*)P.d.bias)[col];
  }
  DEV void put(float* s, int tid) const {
    s[tid] = sa;
    s[256 + tid] = sb;
    s[512 + tid] = bias;
  }
};

DEV void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The end of a tile: four columns, and CG of them COLS apart, of rows row, row + STEP, ... (four of
// them, those below end): activation, residual, store.  FULL: all rows and columns are there,
// so nothing is tested (a wave is alone on its SIMD, and branches around every store are
// not hidden: 4096 x 8192 x 2048 in tiles of 256 x 256 82 us, 72 so).
template <typename T, bool FULL, int CG, int COLS, int STEP>
DEV void emit_rows(const DenseParams& P, int64_t row, int64_t end, int col, float (&v)[16 * CG]) {
  float o[16 * CG];
  if (P.add) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int g = 0; g < CG; ++g) {
        const int n = P.N - (col + g * COLS);
        if (!FULL && (row + i * STEP >= end || n <= 0)) continue;
        float t[4];
        get4((const T*)P.add + (row + i * STEP) * P.ldadd + col + g * COLS, FULL ? 4 : n, t);
#pragma unroll
        for (int q = 0; q < 4; ++q) o[16 * g + 4 * i + q] = t[q];
      }
  }
  act_n<sizeof(T) == 4, 16 * CG>(P.act, v);
  if (P.add) {
#pragma unroll
    for (int i = 0; i < 16 * CG; ++i) v[i] = v[i] + o[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int g = 0; g < CG; ++g) {
      const int n = P.N - (col + g * COLS);
      if (!FULL && (row + i * STEP >= end || n <= 0)) continue;
      const float* w = v + 16 * g + 4 * i;
      put4<true>((T*)P.c[0] + (row + i * STEP) * P.ldc + col + g * COLS, FULL ? 4 : n, {w[0], w[1], w[2], w[3]});
    }
}

// WGS: workgroups that share a CU (its registers and LDS), so that one's first loads and
// epilogue run beside another's slices.
// 8192^3 432 to 450 us, 2.4 to 2.5 POP/s: matrix units busy 62 to 68% of the cycles, at the 1.5 to 1.8 GHz
// that the power leaves.  4096 x 8192 x 2048 69 to 72 us: of each of its two rounds (256 x 256) 5 the launch and
// first slice, 23 the slices, 8 the 33 MB stored; GELU adds 5 to 7, which nothing hides.
// A contraction split into S chunks (one group only): each workgroup leaves its sums in
// the workspace, and int8_join_kernel adds them and runs the epilogue.  (The last workgroup
// of a tile doing that, by a ticket, needs a fence across the XCDs in each: 37 x 8192 x
// 2048 73 us, against 8 unsplit.)
template <typename T, int MB, int NB, int NS, int WGS, bool GROUPS>
__global__ __launch_bounds__(256, WGS) void int8_tile_kernel(Int8Params P) {
  constexpr int BM = 64 * MB, BN = 64 * NB, LA = 2 * MB, LB = 2 * NB;
  // The sums go through LDS, so that a wave writes whole pieces of rows: each wave for itself,
  // 32 rows at a time, the next ones stored before these are read.  They are converted behind it:
  // in front, the compiler converts all of them at once and spills.
  constexpr int ROW = 32 * NB + 4, STAGE = 32 * ROW, STAGES = MB > 1 ? 2 : 1;   // in words
  constexpr int LR = NB > 1 ? 16 : 8;             // lanes on a row, four columns each
  constexpr int CG = 32 * NB / (4 * LR), STEPS = NB > 1 ? 2 : 1;   // groups of columns; 16 or 32 rows a step
  constexpr int RING = NS * line::kSlot<MB, NB>, BEHIND = (4 * STAGES * STAGE + 768) * 4;
  __shared__ __attribute__((aligned(16))) int8_t lds[RING > BEHIND ? RING : BEHIND];
  Int8Tile t;
  if (!int8_tile<GROUPS>(P, BM, BN, t)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int nvalid = P.d.N - t.n0 < BN ? P.d.N - t.n0 : BN;
  const int K = (int)P.d.K;
  int s0 = 0, nsteps = (K + line::BK - 1) / line::BK;
  if constexpr (!GROUPS) {
    const int all = nsteps, chunks = P.d.S;
    s0 = (int)((int64_t)t.chunk * all / chunks);
    nsteps = (int)((int64_t)(t.chunk + 1) * all / chunks) - s0;
  }
  line::Op<LA> oa;
  line::Op<LB> ob;
  oa.init(P.a + t.m0 * P.lda, (t.rows - 1) * P.lda + K, wave, lane, t.rows, P.lda);
  ob.init(P.b + ((int64_t)t.g * P.d.N + t.n0) * K, (int64_t)nvalid * K, wave, lane, nvalid, K);
  const int k0 = line::first_code(lane, 0), k1 = line::first_code(lane, 1);
  TileScales ts;
  ts.load<T>(P, t, tid);
  i32x16_t acc[MB][NB];
  line::mainloop<MB, NB, NS>(bf::lds_base(lds), nsteps, [&](int s, uint32_t st, int i) {
    const bool live = s < nsteps, isa = i < LA;
    const int ks = live ? (s0 + s) * line::BK : 0, j = isa ? i : i - LA;
    const bool ok = live && ks + ((i & 1) ? k1 : k0) < K;
    bf::dma16(isa ? oa.rs : ob.rs, st + (isa ? 0u : (uint32_t)MB * 8192u) + (uint32_t)(wave * (isa ? LA : LB) + j) * 1024u,
              ok ? (isa ? oa.voff[isa ? j : 0] : ob.voff[isa ? 0 : j]) : bf::kOOB, (uint32_t)ks);
  }, acc, wm, wn, lane);
  float* scales = (float*)(lds + 4 * STAGES * STAGE * 4);
  ts.put(scales, tid);
  lds_barrier();
  int* stage = (int*)lds + wave * STAGES * STAGE;
  auto put = [&](int buf, const i32x16_t (&a)[NB]) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *(i32x4_t*)(stage + buf * STAGE + (lane & 31) * ROW + n * 32 + 8 * i + 4 * (lane >> 5)) =
            i32x4_t{a[n][4 * i], a[n][4 * i + 1], a[n][4 * i + 2], a[n][4 * i + 3]};
    asm volatile("" ::: "memory");
  };
  put(0, acc[0]);
  const int lr = lane / LR, c0 = wn * 32 * NB + lane % LR * 4;
  float sb[CG][4], bias[CG][4];
#pragma unroll
  for (int g = 0; g < CG; ++g)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      sb[g][q] = scales[256 + c0 + g * 4 * LR + q];
      bias[g][q] = scales[512 + c0 + g * 4 * LR + q];
    }
  auto rows = [&](auto full) __attribute__((always_inline)) {
#pragma unroll 1
    for (int s = 0; s < MB * STEPS; ++s) {
      const int mb = s / STEPS;
      if (s % STEPS == 0) {
        if ((wm * MB + mb) * 32 >= t.rows) return;
#pragma unroll
        for (int q = 1; q < MB; ++q)
          if (mb + 1 == q) put(q % STAGES, acc[q]);
      }
      const int r0 = s % STEPS * 16 + lr, row0 = (wm * MB + mb) * 32 + r0;
      const int* src = stage + mb % STAGES * STAGE + r0 * ROW + lane % LR * 4;
      if constexpr (!GROUPS) {
        if (P.d.S > 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int g = 0; g < CG; ++g)
              if (row0 + i * (64 / LR) < t.rows && c0 + g * 4 * LR < nvalid)
                *(i32x4_t*)(P.part + ((int64_t)t.chunk * P.d.M + t.m0 + row0 + i * (64 / LR)) * P.part_ld + t.n0 + c0 + g * 4 * LR) =
                    *(const i32x4_t*)(src + i * (64 / LR) * ROW + g * 4 * LR);
          continue;
        }
      }
      float v[16 * CG];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float sa = scales[row0 + i * (64 / LR)];
#pragma unroll
        for (int g = 0; g < CG; ++g) {
          const i32x4_t sv = *(const i32x4_t*)(src + i * (64 / LR) * ROW + g * 4 * LR);
#pragma unroll
          for (int q = 0; q < 4; ++q) v[16 * g + 4 * i + q] = __builtin_fmaf((float)sv[q] * sa, sb[g][q], bias[g][q]);
        }
      }
      emit_rows<T, full.value, CG, 4 * LR, 64 / LR>(P.d, t.m0 + row0, t.m0 + t.rows, t.n0 + c0, v);
    }
  };
  if (t.rows == BM && nvalid == BN)
    rows(std::true_type{});
  else
    rows(std::false_type{});
}

// The chunks' sums of four columns a thread, then the epilogue.
template <typename T>
__global__ __launch_bounds__(256) void int8_join_kernel(Int8Params P) {
  const uint32_t quads = ((uint32_t)P.d.N + 3) / 4;
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;   // a split product has few elements
  if (i >= (uint32_t)P.d.M * quads) return;
  const int64_t row = i / quads;
  const int col = (int)(i - (uint32_t)row * quads) * 4;
  const int32_t* p = P.part + row * P.part_ld + col;
  i32x4_t a = *(const i32x4_t*)p;
#pragma unroll 4
  for (int s = 1; s < P.d.S; ++s) a = a + *(const i32x4_t*)(p + (int64_t)s * P.d.M * P.part_ld);
  const float sa = P.sa[row];
  Cols4<T> c4;
  c4.load(P, 0, col);
  float v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = __builtin_fmaf((float)a[q] * sa, c4.sb[q], c4.bias[q]);
  emit<T, kFormLinear, 1, false, true>(P.d, 0, AtRows{row, row + 1, 1, col}, v);
}

// -------------------------------------------------------------------- few rows
// A wave streams 16 weight rows in steps of 64 codes, and multiplies each with 16 rows
// of x (v_mfma_i32_16x16x64_i8; a lane's 16 bytes of the weights come straight from
// memory).  A workgroup's four waves are 4 / ks neighbouring blocks of weight rows, each
// streamed by ks waves that take its steps in turn and whose sums meet in LDS.  A
// lane ends with four neighbouring columns of one row.
// FUSED: x is not yet quantised; every workgroup does that itself for its rows, into LDS,
// while its first weights are on the way: a launch of 4 to 5 us saved (1 x 2048 x 2048 5.8
// us, 3.9 and 4.4 in two launches).
// Bound by the weights' stream where experts are many (a token's 22 experts of 2048 x 2048, 92
// MB: 18.8 to 19.8 us, 4.6 to 4.9 TB/s), by latency below (4.2 MB: 4.9 to 6.0).
constexpr int kFewWaves = 4, kFewDepth = 8;
template <typename T, bool GROUPS, bool FUSED>
__global__ __launch_bounds__(64 * kFewWaves) void int8_few_kernel(Int8Params P, int ks) {
  constexpr int NT = 64 * kFewWaves;
  __shared__ __attribute__((aligned(16))) i32x4_t s_acc[NT];
  __shared__ __attribute__((aligned(16))) int8_t s_x[FUSED ? kInt8FusedBytes : 16];
  __shared__ uint32_t s_top[16];
  Int8Tile t;
  if (!int8_tile<GROUPS>(P, 16, 16 * kFewWaves / ks, t)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int part = wave & (ks - 1), n0 = t.n0 + 16 * (wave / ks);   // ks is a power of two
  const int K = (int)P.d.K, steps = (K + 63) / 64;
  const int8_t* w = P.b + ((int64_t)t.g * P.d.N + min(n0 + i16, P.d.N - 1)) * P.d.K;
  const int xrow = min(i16, t.rows - 1);
  const int8_t* x = FUSED ? s_x + xrow * K : P.a + (t.m0 + xrow) * P.lda;
  i32x4_t acc = {0, 0, 0, 0};
  // past the end of the rows: their last 16 codes again, and zeros for x
  auto at = [&](int s) { return min(64 * s + 16 * g, K - 16); };
  auto load_x = [&](int s) __attribute__((always_inline)) { return *(const i32x4_t*)(x + at(s)); };
  struct Step {
    i32x4_t w, x;
  };
  auto load = [&](Step& f, int s) __attribute__((always_inline)) {
    f.w = *(const i32x4_t*)(w + at(s));
    if constexpr (!FUSED) f.x = load_x(s);
  };
  auto mul = [&](const Step& f, int s) __attribute__((always_inline)) {
    const bool in = 64 * s + 16 * g < K;
    i32x4_t v = FUSED ? load_x(s) : f.x;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = in ? v[q] : 0;
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.w, v, acc, 0, 0, 0);
  };
  // the steps part, part + ks, ... in rounds of kFewDepth, the next round's loads in
  // flight; the last round loads nothing
  const int n = steps > part ? (steps - part + ks - 1) / ks : 0;
  Step st[kFewDepth];
#pragma unroll
  for (int d = 0; d < kFewDepth; ++d) load(st[d], part + min(d, max(n - 1, 0)) * ks);
  // the epilogue's numbers, loaded beside the stream
  const int col = n0 + 4 * g;
  Cols4<T> c4;
  c4.load(P, t.g, col);
  float sa = 0.f;
  if constexpr (FUSED) {
    constexpr int V = Vec<T>::N;
    const int per = K / V, vecs = t.rows * per;
    if (tid < 16) s_top[tid] = 0u;
    __syncthreads();
    auto get = [&](int v, int row) __attribute__((always_inline)) {
      const int c = (v - row * per) * V, left = P.xcols - c;
      return left > 0 ? Vec<T>::load((const T*)P.x + (t.m0 + row) * P.ldx + c, left) : typename Vec<T>::raw{};
    };
    for (int v = tid; v < vecs; v += NT) {
      const int row = v / per;
      atomicMax(&s_top[row], magnitude(get(v, row)));
    }
    __syncthreads();
    for (int v = tid; v < vecs; v += NT) {
      const int row = v / per;
      put_codes<T>(s_x + v * V, get(v, row), row_scale(s_top[row]));
    }
    sa = row_scale(s_top[xrow]).scale;
    __syncthreads();
  } else {
    sa = P.sa[t.m0 + xrow];
  }
  int i = 0;
#pragma unroll 1
  for (; i + kFewDepth < n; i += kFewDepth) {
#pragma unroll
    for (int d = 0; d < kFewDepth; ++d) {
      mul(st[d], part + (i + d) * ks);
      load(st[d], part + min(i + kFewDepth + d, n - 1) * ks);
    }
  }
#pragma unroll
  for (int d = 0; d < kFewDepth; ++d)
    if (i + d < n) mul(st[d], part + (i + d) * ks);
  if (ks > 1) {
    s_acc[tid] = acc;
    __syncthreads();
    if (part != 0) return;
    for (int v = 1; v < ks; ++v) acc = acc + s_acc[tid + 64 * v];
  }
  if (col >= P.d.N || i16 >= t.rows) return;
  float v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = __builtin_fmaf((float)acc[q] * sa, c4.sb[q], c4.bias[q]);
  emit<T, kFormLinear, 1, false, true>(P.d, 0, AtRows{t.m0 + i16, t.m0 + i16 + 1, 1, col}, v);
}

// --------------------------------------------------------------------- launches
namespace {

// Workgroups of a launch: with groups, as many as ascending offsets can need.
dim3 int8_grid(const Int8Params& P, int bm, int bn) {
  const int64_t nT = (P.d.N + bn - 1) / bn;
  int64_t mT = (P.d.M + bm - 1) / bm;
  if (P.offsets) {
    mT = P.d.M / bm + P.groups;
    if (mT > P.d.M) mT = P.d.M;
  }
  return dim3((uint32_t)grid_for_units(mT * nT * P.d.S));
}

template <typename T, bool GROUPS>
void tiles(const Int8Params& P, int tile, hipStream_t st) {
  const Int8Shape sh = kInt8Shapes[tile];
  const dim3 grid = int8_grid(P, sh.bm, sh.bn);
  switch (tile) {   // kInt8Shapes
    case 0: int8_tile_kernel<T, 4, 4, 2, 1, GROUPS><<<grid, 256, 0, st>>>(P); break;
    case 1: int8_tile_kernel<T, 2, 2, 2, 2, GROUPS><<<grid, 256, 0, st>>>(P); break;
    case 2: int8_tile_kernel<T, 2, 1, 3, 2, GROUPS><<<grid, 256, 0, st>>>(P); break;
    case 3: int8_tile_kernel<T, 2, 1, 2, 3, GROUPS><<<grid, 256, 0, st>>>(P); break;
    case 4: int8_tile_kernel<T, 1, 1, 2, 4, GROUPS><<<grid, 256, 0, st>>>(P); break;
    default: int8_tile_kernel<T, 1, 1, 4, 2, GROUPS><<<grid, 256, 0, st>>>(P);
  }
  if (!GROUPS && P.d.S > 1) int8_join_kernel<T><<<(uint32_t)((P.d.M * ((P.d.N + 3) / 4) + 255) / 256), 256, 0, st>>>(P);
}

template <typename T, bool FUSED>
void few(const Int8Params& P, dim3 grid, int ks, hipStream_t st) {
  if (P.offsets)
    int8_few_kernel<T, true, FUSED><<<grid, 64 * kFewWaves, 0, st>>>(P, ks);
  else
    int8_few_kernel<T, false, FUSED><<<grid, 64 * kFewWaves, 0, st>>>(P, ks);
}

}  // namespace

hipError_t launch_int8_tiles(const Int8Params& P, bool bf16, int tile, hipStream_t st) {
  if (bf16)
    P.offsets ? tiles<uint16_t, true>(P, tile, st) : tiles<uint16_t, false>(P, tile, st);
  else
    P.offsets ? tiles<float, true>(P, tile, st) : tiles<float, false>(P, tile, st);
  return hipGetLastError();
}

hipError_t launch_int8_few(const Int8Params& P, bool bf16, int ks, hipStream_t st) {
  const dim3 grid = int8_grid(P, 16, 16 * kFewWaves / ks);
  if (bf16)
    P.x ? few<uint16_t, true>(P, grid, ks, st) : few<uint16_t, false>(P, grid, ks, st);
  else
    P.x ? few<float, true>(P, grid, ks, st) : few<float, false>(P, grid, ks, st);
  return hipGetLastError();
}

}  // namespace moedet
