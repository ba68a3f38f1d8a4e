// Rows copied for their experts and summed back, forward and backward.
//
//  permute        rows[slot_row[t, j]] = x[t]
//  unpermute      y[t] = sum over j ascending of p[t, j] rows[slot_row[t, j]],
//                 float32 from 0, then add[t], rounded once.  Without p it is
//                 permute's backward.
//  unpermute_bwd  drows[slot_row[t, j]] = p[t, j] dy[t] in float32, rounded to the type;
//                 dprob[t, j] = <dy[t], rows[slot_row[t, j]]> in float32, each
//                 lane over its columns ascending, then a fixed tree over the lanes.
//
// All three go by token, not by row: a token's row is read once and stays in
// registers or the L1 for its k slots, and no row -> slot table is read.  All are
// bound by HBM.  Each output element is written by one thread: no atomics.
// A slot whose row is outside [0, nrows) has none: it is not read or written.
#include <type_traits>

#include "rows.h"

namespace moedet {

namespace {

typedef uint32_t u32x4_b_t __attribute__((ext_vector_type(4), aligned(1)));

// Rows that the last-level cache cannot hold are stored past it: otherwise the next
// kernel's reads wait for their write-back.  4096 tokens of 22 slots, 2048 bf16 (369 MB of
// rows): copied and summed back 177 us through the caches, 150 past them, gradients
// 161 and 167 us alone but 246 and 218 behind the forward.  180 MB copied and summed back:
// 37 and 42 us.  How many slots have a row is known on the GPU alone, so the size of the matrix
// decides, here and below: one that is larger than its rows need may be taken for one that the
// cache cannot hold (16384 tokens of 22 slots with 4 of 512 experts here, 2048 bf16, about 2050 rows
// summed back: 20.5 us in a matrix of 65536 rows, 25.6 past the cache in one of 360448).
constexpr int64_t kLastLevelBytes = (int64_t)256 << 20;
bool past_cache(const RowsParams& P, int es) {
  const int64_t slots = P.tokens * P.k;
  return (P.nrows < slots ? P.nrows : slots) * P.cols * es > kLastLevelBytes;
}

// Such rows are loaded past it as well (the 369 MB summed back: 72.6 us through the
// caches, 67.8 past them; 6 MB of rows that the backward reads again: 4.3 and 5.2 us).
DEV u32x4_t load_past(const uint16_t* p) { return __builtin_nontemporal_load((const u32x4_any_t*)p); }
DEV f32x4_t load_past(const float* p) { return __builtin_nontemporal_load((const f32x4_any_t*)p); }

DEV void store_past(uint16_t* p, const float* v) {
  __builtin_nontemporal_store(u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])},
                              (u32x4_any_t*)p);
}
DEV void store_past(float* p, const float* v) {
  __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, (f32x4_any_t*)p);
}

// A workgroup of 256 threads takes 256 / L tokens, L threads each (a power of two
// up to 256, the row's 16-byte vectors where they are fewer).
int row_threads(int64_t vecs, int most) {
  int L = 8;
  while (L < most && L < vecs) L <<= 1;
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

// The row of slot j of a token, -1 if it has none.
DEV int32_t slot_at(const RowsParams& P, const int32_t* sr, int j, int end) {
  const int32_t r = j < end ? sr[j] : -1;
  return r < P.nrows ? r : -1;
}

// The slots that have a row, ascending, up to 64 at a time: the lanes read them
// together and a ballot finds the ones with a row, so a rank with few of the
// experts passes over the other slots at once.  f(lane of the slot, row) for each
// in turn, where the wave has one token (WHOLE).
template <class F>
DEV void each_slot(uint64_t mask, int32_t r, F f) {
  while (mask) {
    const int b = (int)__builtin_ctzll(mask);
    mask &= mask - 1;
    f(b, __builtin_amdgcn_readlane(r, b));
  }
}

// WHOLE: L >= 64, so a wave has one token.
// 4096 tokens of 22 slots, 2048 bf16 (386 MB): 75 to 78 us, 5.0 to 5.2 TB/s.  16384 tokens of
// which 2816 slots have a row: 42 us where every token's row was read and every
// slot looked at in turn by four waves a token, 21 with the ballot, 10 with one wave.
template <bool WHOLE, bool PAST>
__global__ __launch_bounds__(256) void permute_kernel(RowsParams P, int es, int L, int S) {
  Place p;
  if (!place(P, L, S, p)) return;
  const int64_t t = WHOLE ? (int64_t)__builtin_amdgcn_readfirstlane((int)p.t) : p.t;
  const int64_t len = (int64_t)P.cols * es;
  const int vecs = (int)((len + 15) / 16);
  const char* src = (const char*)P.x + t * P.ldx * es;
  const int32_t* sr = P.slot_row + t * P.k;
  const int lane = threadIdx.x & 63;
  auto put = [&](int32_t r, int64_t at, int n, const u32x4_t& x) __attribute__((always_inline)) {
    char* dst = (char*)P.out + (int64_t)r * len + at;
    if (n == 16) {
      if constexpr (PAST)
        __builtin_nontemporal_store(x, (u32x4_b_t*)dst);
      else
        *(u32x4_b_t*)dst = x;
    } else {
      for (int b = 0; b < n; ++b) dst[b] = src[at + b];
    }
  };
  if constexpr (WHOLE) {
    for (int j0 = p.j0; j0 < p.j1; j0 += 64) {
      const int32_t r = slot_at(P, sr, j0 + lane, p.j1);
      const uint64_t mask = __ballot(r >= 0);
      if (!mask) continue;
      // 4 KB of the row at a time, stored whole for one slot after the other (4096 tokens of
      // 22 slots, 2048 bf16, again and again: 85 us in pieces of 1 KB, 77 so)
      constexpr int C = 4;
      // The loop is the same for all lanes: each_slot reads r of lanes that have no vector left.
      for (int v0 = 0; v0 < vecs; v0 += C * 64) {
        const int v = v0 + lane;
        u32x4_t x[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int64_t at = ((int64_t)v + c * 64) * 16;
          if (at + 16 <= len) x[c] = *(const u32x4_b_t*)(src + at);
        }
        each_slot(mask, r, [&](int, int32_t row) __attribute__((always_inline)) {
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const int64_t at = ((int64_t)v + c * 64) * 16;
            if (at < len) put(row, at, (int)(len - at < 16 ? len - at : 16), x[c]);
          }
        });
      }
    }
  } else {
    for (int v = p.v; v < vecs; v += L) {
      const int64_t at = (int64_t)v * 16;
      const int n = (int)(len - at < 16 ? len - at : 16);
      u32x4_t x = {0u, 0u, 0u, 0u};
      if (n == 16) x = *(const u32x4_b_t*)(src + at);
      for (int j = p.j0; j < p.j1; ++j) {
        const int32_t r = slot_at(P, sr, j, p.j1);
        if (r >= 0) put(r, at, n, x);
      }
    }
  }
}

// acc += w * the row's vector (or the vector itself without weights)
template <typename T>
DEV void add_row(float (&acc)[Vec<T>::N], const typename Vec<T>::raw& x, bool weighted, float w) {
  float f[Vec<T>::N];
  Vec<T>::get(x, f);
#pragma unroll
  for (int q = 0; q < Vec<T>::N; ++q) acc[q] = weighted ? __builtin_fmaf(w, f[q], acc[q]) : acc[q] + f[q];
}

DEV float get1(const uint16_t* p) { return bf16_to_f32(*p); }
DEV float get1(const float* p) { return *p; }
DEV void put1(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16(v); }
DEV void put1(float* p, float v) { *p = v; }

// Narrow rows, several tokens a wave.
template <typename T>
__global__ __launch_bounds__(256) void unpermute_narrow_kernel(RowsParams P, int L) {
  constexpr int V = Vec<T>::N;
  Place p;
  if (!place(P, L, 1, p)) return;
  const int64_t t = p.t;
  const int32_t* sr = P.slot_row + t * P.k;
  const float* pr = P.prob ? P.prob + t * P.k : nullptr;
  const int col = p.v * V, n = P.cols - col;   // L threads hold the whole row
  if (n <= 0) return;
  float acc[V];
#pragma unroll
  for (int q = 0; q < V; ++q) acc[q] = 0.f;
  // slots in groups whose numbers, then rows, are loaded together
  constexpr int G = 4;
  for (int j0 = 0; j0 < P.k; j0 += G) {
    int32_t r[G];
    typename Vec<T>::raw x[G];
#pragma unroll
    for (int i = 0; i < G; ++i) r[i] = slot_at(P, sr, j0 + i, P.k);
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (r[i] >= 0) x[i] = Vec<T>::load((const T*)P.rows + (int64_t)r[i] * P.cols + col, n);
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (r[i] >= 0) add_row<T>(acc, x[i], pr != nullptr, pr ? pr[j0 + i] : 1.f);
  }
  if (P.add) {
    float a[V];
    Vec<T>::get(Vec<T>::load((const T*)P.add + t * P.ldadd + col, n), a);
#pragma unroll
    for (int q = 0; q < V; ++q) acc[q] = acc[q] + a[q];
  }
  Vec<T>::store((T*)P.out + t * P.cols + col, acc, n);
}

// A wave has one token, and every loop and branch on the way to a load is the
// same for its lanes: lanes past the row's last whole vector repeat it and
// store nothing, and the columns behind it are summed one a lane by the token's
// first wave.
// 4096 tokens of 22 slots, 2048 bf16 (386 MB): 68 us, 5.7 TB/s; groups of 4 or 16
// loads are no faster.
template <typename T, bool PAST>
__global__ __launch_bounds__(256) void unpermute_kernel(RowsParams P, int L) {
  constexpr int V = Vec<T>::N;
  Place p;
  if (!place(P, L, 1, p)) return;
  const int64_t t = __builtin_amdgcn_readfirstlane((int)p.t);
  const int lane = threadIdx.x & 63, whole = P.cols / V;
  const int32_t* sr = P.slot_row + t * P.k;
  const bool weighted = P.prob != nullptr;
  const float* pr = weighted ? P.prob + t * P.k : nullptr;
  const T* rows = (const T*)P.rows;
  // add(weight, element offset of the row) for the slots with a row, ascending, in
  // groups of G whose loads go out together
  constexpr int G = 8;
  auto sum = [&](auto load, auto add) __attribute__((always_inline)) {
    for (int j0 = 0; j0 < P.k; j0 += 64) {
      const int32_t r = slot_at(P, sr, j0 + lane, P.k);
      const float wl = weighted && j0 + lane < P.k ? pr[j0 + lane] : 0.f;
      uint64_t mask = __ballot(r >= 0);
      auto group = [&](int left, auto N) __attribute__((always_inline)) {
        decltype(load((int64_t)0)) x[N.value];
        float w[N.value];
#pragma unroll
        for (int i = 0; i < N.value; ++i) {
          const int b = (int)__builtin_ctzll(mask);
          if (i + 1 < left || left == N.value) mask &= mask - 1;   // past `left`: the last one again, not added
          w[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wl), b));
          x[i] = load((int64_t)__builtin_amdgcn_readlane(r, b) * P.cols);
        }
#pragma unroll
        for (int i = 0; i < N.value; ++i)
          if (i < left) add(x[i], w[i]);
      };
      int n = __popcll(mask);
      for (; n >= G; n -= G) group(G, std::integral_constant<int, G>{});
      if (n > G / 2)
        group(n, std::integral_constant<int, G - 1>{});
      else if (n > 0)
        group(n, std::integral_constant<int, G / 2>{});
    }
  };
  for (int v0 = __builtin_amdgcn_readfirstlane(p.v); v0 < whole; v0 += L) {
    const int v = v0 + lane, col = min(v, whole - 1) * V;
    float acc[V];
#pragma unroll
    for (int q = 0; q < V; ++q) acc[q] = 0.f;
    sum([&](int64_t at) __attribute__((always_inline)) {
          if constexpr (PAST)
            return load_past(rows + at + col);
          else
            return Vec<T>::load(rows + at + col, V);
        },
        [&](const typename Vec<T>::raw& x, float w) __attribute__((always_inline)) { add_row<T>(acc, x, weighted, w); });
    if (P.add) {
      float a[V];
      Vec<T>::get(Vec<T>::load((const T*)P.add + t * P.ldadd + col, V), a);
#pragma unroll
      for (int q = 0; q < V; ++q) acc[q] = acc[q] + a[q];
    }
    if (v < whole) Vec<T>::store((T*)P.out + t * P.cols + col, acc, V);
  }
  if (__builtin_amdgcn_readfirstlane(p.v) == 0 && whole * V < P.cols) {
    const int c = whole * V + lane, col = min(c, P.cols - 1);
    float acc = 0.f;
    sum([&](int64_t at) __attribute__((always_inline)) { return get1(rows + at + col); },
        [&](float x, float w) __attribute__((always_inline)) { acc = weighted ? __builtin_fmaf(w, x, acc) : acc + x; });
    if (P.add) acc = acc + get1((const T*)P.add + t * P.ldadd + col);
    if (c < P.cols) put1((T*)P.out + t * P.cols + c, acc);
  }
}

// A wave G slots: four where less than a third of many can have a row, by the rows of the matrix (a
// rank with few of the experts; those that have one are found by a ballot), or a row is one load of
// a wave, one otherwise.  By one and by four, 16384 tokens of 22 slots, 2048 bf16, with 4, 64, 128
// and 256 of 512 experts in a matrix of as many rows as slots have one: 46
// and 21 us, 144 and 104, 206 and 178, 336 and 328; 4096 tokens, 256 of 512: 92 and 95; all
// slots with a row: 131072 of 512 columns 71 and 57, 65536 of 1024 63 and 76.  The 4 of 512 in a
// matrix of 65536 rows 19.3, of 360448, which could hold a row of every slot, 41.
// Rows that the caches cannot hold are taken in the order of the
// slots, not in runs an XCD: rows of one expert that lie side by side are then
// read and written at about the same time (369 MB of rows behind the forward:
// 243 us in runs, 218 so; 6 MB of them 6.6 and 8.4 us).  4096 tokens of 22 slots, 2048 bf16:
// 755 MB in 158 to 169 us, 4.5 to 4.8 TB/s; 5.7 were the rows in the slots' order.
template <typename T, bool PAST, int G>
__global__ __launch_bounds__(256) void unpermute_bwd_kernel(RowsParams P) {
  constexpr int V = Vec<T>::N;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n = P.tokens * P.k;
  const int64_t units = (n + 4 * G - 1) / (4 * G);
  int64_t u = blockIdx.x;
  if (!PAST || P.seed) u = map_unit(u, units, P.seed);
  if (u < 0 || u >= units) return;
  const int64_t i0 = (u * 4 + w) * G;
  if (i0 >= n) return;
  auto slot = [&](int64_t i, int32_t r) __attribute__((always_inline)) {
    const T* dy = (const T*)P.x + (int64_t)((uint32_t)i / (uint32_t)P.k) * P.ldx;
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
      if (PAST && m >= V)
        store_past(out + col, g);
      else
        Vec<T>::store(out + col, g, m);
    }
    if (!P.dprob) return;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) dot = dot + __shfl_xor(dot, d, 64);
    if (lane == 0) P.dprob[i] = dot;
  };
  if constexpr (G == 1) {
    const int32_t r = P.slot_row[i0];
    if (r >= 0 && r < P.nrows)
      slot(i0, r);
    else if (P.dprob && lane == 0)
      P.dprob[i0] = 0.f;
  } else {
    const int64_t i = i0 + lane;
    const bool mine = lane < G && i < n;
    const int32_t r = mine ? P.slot_row[i] : -1;
    const bool has = r >= 0 && r < P.nrows;
    if (mine && !has && P.dprob) P.dprob[i] = 0.f;
    each_slot(__ballot(has), r, [&](int b, int32_t row) __attribute__((always_inline)) { slot(i0 + b, row); });
  }
}

namespace {

struct RowsPlan {
  int L, S;        // threads of a token, parts of its slots
  int64_t grid;
};
RowsPlan permute_plan(const RowsParams& P, int es) {
  const int L = row_threads(((int64_t)P.cols * es + 15) / 16, 64);
  const int64_t groups = (P.tokens + 256 / L - 1) / (256 / L);
  // too few tokens for the device: their slots are split too
  int64_t S = groups >= 512 ? 1 : (512 + groups - 1) / groups;
  if (S > P.k) S = P.k;
  return {L, (int)S, grid_for_units(groups * S)};
}

}  // namespace

int64_t permute_grid(const RowsParams& P, int es) { return permute_plan(P, es).grid; }
hipError_t launch_permute(const RowsParams& P, int es, hipStream_t st) {
  const RowsPlan p = permute_plan(P, es);
  if (p.L < 64)
    permute_kernel<false, false><<<p.grid, 256, 0, st>>>(P, es, p.L, p.S);
  else if (past_cache(P, es))
    permute_kernel<true, true><<<p.grid, 256, 0, st>>>(P, es, p.L, p.S);
  else
    permute_kernel<true, false><<<p.grid, 256, 0, st>>>(P, es, p.L, p.S);
  return hipGetLastError();
}

static RowsPlan sum_plan(const RowsParams& P, int vec) {
  // four waves a token, one where few tokens can have any row, by the rows of the matrix (16384 tokens of
  // 22 slots, 2048 bf16, as many rows as slots have one: 4 of 512 experts 23 and 17.5 us, 64 of them 35
  // and 39; 4096 tokens, all 74 and 96).  The 4 of 512 in a matrix of tokens x 4 rows take four waves, 20.5.
  const bool few = P.tokens >= 4096 && 16 * P.nrows < P.tokens * P.k;
  const int L = row_threads((P.cols + vec - 1) / vec, few ? 64 : 256);
  return {L, 1, grid_for_units((P.tokens + 256 / L - 1) / (256 / L))};
}
template <typename T>
static hipError_t launch_sum(const RowsParams& P, hipStream_t st) {
  const RowsPlan p = sum_plan(P, Vec<T>::N);
  if (p.L < 64)
    unpermute_narrow_kernel<T><<<p.grid, 256, 0, st>>>(P, p.L);
  else if (past_cache(P, sizeof(T)))
    unpermute_kernel<T, true><<<p.grid, 256, 0, st>>>(P, p.L);
  else
    unpermute_kernel<T, false><<<p.grid, 256, 0, st>>>(P, p.L);
  return hipGetLastError();
}
int64_t unpermute_grid(const RowsParams& P, bool bf16) { return sum_plan(P, bf16 ? Vec<uint16_t>::N : Vec<float>::N).grid; }
hipError_t launch_unpermute(const RowsParams& P, bool bf16, hipStream_t st) {
  return bf16 ? launch_sum<uint16_t>(P, st) : launch_sum<float>(P, st);
}

// Slots from which a wave may take four of them (below, waves are too few: 32768 slots of which
// 2048 have a row 10.5 us by one, 11.8 by four).
constexpr int64_t kManySlots = 65536;
static bool many_slots(const RowsParams& P, int vec) {
  const int64_t n = P.tokens * P.k;
  return n >= kManySlots && (3 * P.nrows < n || P.cols <= 64 * vec);
}
static int64_t bwd_grid(const RowsParams& P, bool many) {
  const int64_t n = P.tokens * P.k;
  return grid_for_units(many ? (n + 15) / 16 : (n + 3) / 4);
}
int64_t unpermute_bwd_grid(const RowsParams& P, bool bf16) { return bwd_grid(P, many_slots(P, bf16 ? Vec<uint16_t>::N : Vec<float>::N)); }
template <typename T>
static hipError_t launch_bwd(const RowsParams& P, hipStream_t st) {
  const bool many = many_slots(P, Vec<T>::N), past = past_cache(P, sizeof(T));
  const int64_t grid = bwd_grid(P, many);
  if (many && past)
    unpermute_bwd_kernel<T, true, 4><<<grid, 256, 0, st>>>(P);
  else if (many)
    unpermute_bwd_kernel<T, false, 4><<<grid, 256, 0, st>>>(P);
  else if (past)
    unpermute_bwd_kernel<T, true, 1><<<grid, 256, 0, st>>>(P);
  else
    unpermute_bwd_kernel<T, false, 1><<<grid, 256, 0, st>>>(P);
  return hipGetLastError();
}
hipError_t launch_unpermute_bwd(const RowsParams& P, bool bf16, hipStream_t st) {
  return bf16 ? launch_bwd<uint16_t>(P, st) : launch_bwd<float>(P, st);
}

}  // namespace moedet
