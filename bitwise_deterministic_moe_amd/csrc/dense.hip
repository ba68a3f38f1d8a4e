// Matrix products of the dense operators (linear map, gated product), for
// bf16 and float32 storage: tiles for many rows, a weight-streaming kernel for
// few rows, the join of split contractions, and the elementwise passes.
//
//   linear  z = x w + bias, y = act(z) + residual
//   glu     g = x wg, u = x wu, a = act(g) u
//   dx      dz w^T (or dg wg^T + du wu^T as one contraction over both) + dx_add
//   dw      x^T dz (x^T dg and x^T du as one launch)
//
// Every output element is accumulated in float32 by one workgroup in
// ascending k, or, where the launch would leave compute units idle, by S
// workgroups over chunks of k whose float32 partials a second launch adds in
// chunk order.  S and every chunk bound depend on sizes only, and no atomics
// are used, so the bits do not depend on scheduling.
#include <type_traits>

#include "dense_bf16.h"
#include "dense_epilogue.h"
#include "kernels.h"

namespace moedet {

// ------------------------------------------------------------------- units
// Tile order: bands of kBand tile rows, down the band before across, so the
// consecutive units that map_unit gives to an XCD share operand tiles in its
// L2 both ways.
constexpr uint32_t kBand = 4;
struct DenseTile {
  int64_t m0;
  int n0, seg, chunk;
  int s0, s1;       // slices of the contraction (over all K segments)
};

template <int FORM>
DEV bool dense_tile(const DenseParams& P, int bm, int bn, int bk, DenseTile& t) {
  // 32 bits: the launch has one workgroup per unit, fewer than 2^24
  const uint32_t mT = (uint32_t)((P.M + bm - 1) / bm), nTs = (uint32_t)((P.N + bn - 1) / bn);
  const uint32_t nT = FORM == kFormDw ? nTs * P.nseg : nTs;
  const uint32_t tiles = mT * nT;
  const int64_t unit = map_unit(blockIdx.x, (int64_t)tiles * P.S, P.seed);
  if (unit < 0) return false;
  const uint32_t L = (uint32_t)unit;
  t.chunk = (int)(L / tiles);
  const uint32_t tile = L - t.chunk * tiles;
  const uint32_t band = tile / (kBand * nT), in = tile - band * kBand * nT;
  const uint32_t left = mT - band * kBand, h = left < kBand ? left : kBand;
  t.m0 = (int64_t)(band * kBand + in % h) * bm;
  const uint32_t nt = in / h;
  t.seg = FORM == kFormDw && nt >= nTs ? 1 : 0;
  t.n0 = (int)(nt - t.seg * nTs) * bn;
  // chunks of steps / S slices, the first steps % S of one more
  const uint32_t steps = (uint32_t)((P.K + bk - 1) / bk * (FORM == kFormDx ? P.nseg : 1));
  const uint32_t q = steps / P.S, r = steps - q * P.S;
  t.s0 = (int)(t.chunk * q + min((uint32_t)t.chunk, r));
  t.s1 = t.s0 + (int)(q + ((uint32_t)t.chunk < r ? 1 : 0));
  return true;
}

// ---------------------------------------------------------------- bf16 tiles
// The accumulator tile goes through LDS in passes of 64 rows (row stride
// 260 floats), so that a wave reads and writes whole rows in global memory.
constexpr int kDenseStageRow = 260;
static_assert(64 * kDenseStageRow * 4 <= dn::kRingBytes<64>, "epilogue stage must fit in the ring");

// Operands are read in chunks of 8 columns: their rows hold whole chunks
// (sizes and row distances are multiples of 8, or the operand was copied into such rows).
DEV int64_t up8(int64_t n) { return (n + 7) & ~(int64_t)7; }

DEV void dense_lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Only the copy into LDS is written out per pass (its registers are fixed);
// the rest is one loop body: unrolled, the kernels took 50 to 67 KB of code, about the
// whole instruction cache, run through once.
template <int FORM, int WTM>
DEV void dense_store_tile(const DenseParams& P, const DenseTile& t, float* stage, f32x16_t (&acc)[4][4], int wm, int wn,
                          int lane, int wave) {
  const int r32 = lane & 31, half = lane >> 5;
  const int rows = (int)(P.M - t.m0 < 2 * WTM ? P.M - t.m0 : 2 * WTM);
  const int64_t end = t.m0 + rows;
  // a thread's four columns, and so its bias, are the same in every row
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if (FORM == kFormLinear && P.bias && P.S == 1 && t.n0 + lane * 4 < P.N)
    get4((const uint16_t*)P.bias + t.n0 + lane * 4, P.N - t.n0 - lane * 4, bias);
#pragma unroll 1
  for (int p = 0; 64 * p < rows; ++p) {
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
            // GLU: g in columns 0..127, u in 128..255
            const int col = (FORM == kFormGlu ? (nb >> 1) * 128 + wn * 64 + (nb & 1) * 32 : wn * 128 + nb * 32) + 8 * i +
                            4 * half;
            const f32x16_t& a = acc[mb][nb];
            *(f32x4_t*)(stage + (r0 + r32) * kDenseStageRow + col) =
                f32x4_t{a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]};
          }
      }
    }
    dense_lds_barrier();
    if constexpr (FORM == kFormGlu) {
      // two rows per wave and step: lanes 0..31 one, lanes 32..63 the next
      const int c = (lane & 31) * 4, col = t.n0 + c;
#pragma unroll
      for (int st = 0; st < 8; st += 4) {
        float g[16], u[16];
        const int m = 8 * st + 2 * wave + half;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4_t sg = *(const f32x4_t*)(stage + (m + 8 * i) * kDenseStageRow + c);
          const f32x4_t su = *(const f32x4_t*)(stage + (m + 8 * i) * kDenseStageRow + 128 + c);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            g[4 * i + q] = sg[q];
            u[4 * i + q] = su[q];
          }
        }
        if (col >= P.N) continue;
        const AtRows at{t.m0 + 64 * p + m, end, 8, col};
        if (P.S > 1) {
          part<4>(P, t.chunk, 0, at, g);
          part<4>(P, t.chunk, 1, at, u);
        } else {
          emit_glu<uint16_t, 4, true>(P, at, g, u);
        }
      }
    } else {
      const int c = lane * 4, col = t.n0 + c;
#pragma unroll
      for (int st = 0; st < 16; st += 4) {
        float v[16];
        const int m = 4 * st + wave;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4_t sv = *(const f32x4_t*)(stage + (m + 4 * i) * kDenseStageRow + c);
#pragma unroll
          for (int q = 0; q < 4; ++q) v[4 * i + q] = FORM == kFormLinear ? sv[q] + bias[q] : sv[q];
        }
        if (col >= P.N) continue;
        const AtRows at{t.m0 + 64 * p + m, end, 4, col};
        if (P.S > 1)
          part<4>(P, t.chunk, t.seg, at, v);
        else
          emit<uint16_t, FORM, 4, true, true>(P, t.seg, at, v);
      }
    }
    dense_lds_barrier();
  }
}

template <int FORM, int WTM>
__global__ __launch_bounds__(256) void dense_bf16_kernel(DenseParams P) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[dn::kRingBytes<WTM> / 2];
  constexpr int BMv = 2 * WTM, BNv = FORM == kFormGlu ? 128 : 256;
  DenseTile t;
  if (!dense_tile<FORM>(P, BMv, BNv, dn::BK, t)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const uint32_t ring = bf::lds_base(lds);
  constexpr int LA = dn::kALoads<WTM>;
  constexpr uint32_t AB = dn::kAOper<WTM> * 2;   // bytes of an A slot
  const int nsteps = t.s1 - t.s0;
  const int mvalid = (int)(P.M - t.m0 < BMv ? P.M - t.m0 : BMv);
  const int nvalid = P.N - t.n0;
  f32x16_t acc[4][4];
  if constexpr (FORM == kFormDw) {
    // both operands row k = contraction; the chunk starts at row 32 s0
    const int64_t k0 = (int64_t)t.s0 * dn::BK;
    const int64_t kn = P.K - k0 < (int64_t)nsteps * dn::BK ? P.K - k0 : (int64_t)nsteps * dn::BK;
    dn::MncOp<BMv, LA> oa;
    dn::MncOp<256, 4> ob;
    oa.init((const uint16_t*)P.a + k0 * P.lda + t.m0, ((kn - 1) * P.lda + up8(mvalid)) * 2, wave, lane, mvalid, P.lda);
    ob.init((const uint16_t*)P.b[0] + k0 * P.ldb + t.seg * P.seg + t.n0, ((kn - 1) * P.ldb + up8(nvalid)) * 2, wave,
            lane, nvalid, P.ldb);
    const uint32_t sa = (uint32_t)(dn::BK * P.lda * 2), sb = (uint32_t)(dn::BK * P.ldb * 2);
    dn::mainloop<dn::MNC, dn::MNC, WTM>(ring, nsteps, [&](int s, uint32_t st, int i) {
      if (i < LA)
        oa.issue(st, wave, i, (uint32_t)s * sa);
      else
        ob.issue(st + AB, wave, i - LA, (uint32_t)s * sb);
    }, acc, wm, wn, lane);
  } else {
    const int steps_seg = (int)((P.K + dn::BK - 1) / dn::BK);
    dn::KcOp<LA> oa;
    const int64_t a_cols = (FORM == kFormDx && P.nseg > 1 ? P.seg : 0) + up8(P.K);
    oa.init((const uint16_t*)P.a + t.m0 * P.lda, ((mvalid - 1) * P.lda + a_cols) * 2, wave, lane, mvalid, P.lda);
    const int kc = dn::KcOp<LA>::chunk(lane) * 8;   // first k of this lane's chunk in a slice
    if constexpr (FORM == kFormDx) {
      dn::KcOp<4> ob, ob1;
      const int64_t eb = ((int64_t)(nvalid < 256 ? nvalid - 1 : 255) * P.ldb + up8(P.K)) * 2;
      ob.init((const uint16_t*)P.b[0] + (int64_t)t.n0 * P.ldb, eb, wave, lane, nvalid, P.ldb);
      ob1.rs = bf::make_rsrc((const uint16_t*)P.b[P.nseg - 1] + (int64_t)t.n0 * P.ldb, (uint32_t)eb);
      dn::mainloop<dn::KC, dn::KC, WTM>(ring, nsteps, [&](int s, uint32_t st, int i) {
        const bool live = s < nsteps;
        int ks = live ? t.s0 + s : 0;
        const bool second = ks >= steps_seg;
        if (second) ks -= steps_seg;
        const bool ok = live && ks * dn::BK + kc < P.K;
        if (i < LA) {
          oa.issue(st, wave, i, ok, (uint32_t)ks * 64u + (second ? (uint32_t)P.seg * 2u : 0u));
        } else {
          const bf::i32x4_t rs = second ? ob1.rs : ob.rs;
          bf::dma16(rs, st + AB + (uint32_t)(wave * 4 + i - LA) * 1024u, ok ? ob.voff[i - LA] : dn::kOOB, (uint32_t)ks * 64u);
        }
      }, acc, wm, wn, lane);
    } else {
      const int64_t k0 = (int64_t)t.s0 * dn::BK;
      const uint32_t sb = (uint32_t)(dn::BK * P.ldb * 2);
      auto issue_a = [&](int s, uint32_t st, int i) {
        const bool live = s < nsteps;
        const int ks = live ? t.s0 + s : 0;
        oa.issue(st, wave, i, live && ks * dn::BK + kc < P.K, (uint32_t)ks * 64u);
      };
      // rows of w from the chunk's first to the matrix' last: rows past a
      // chunk that is not the last one are read and never multiplied
      const int64_t kn = P.K - k0;
      if constexpr (FORM == kFormLinear) {
        dn::MncOp<256, 4> ob;
        ob.init((const uint16_t*)P.b[0] + k0 * P.ldb + t.n0, ((kn - 1) * P.ldb + up8(nvalid)) * 2, wave, lane, nvalid, P.ldb);
        dn::mainloop<dn::KC, dn::MNC, WTM>(ring, nsteps, [&](int s, uint32_t st, int i) {
          if (i < LA)
            issue_a(s, st, i);
          else
            ob.issue(st + AB, wave, i - LA, (uint32_t)s * sb);
        }, acc, wm, wn, lane);
      } else {
        dn::MncOp<128, 2> og, ou;
        const int64_t e = ((kn - 1) * P.ldb + up8(nvalid)) * 2;
        og.init((const uint16_t*)P.b[0] + k0 * P.ldb + t.n0, e, wave, lane, nvalid, P.ldb);
        ou.init((const uint16_t*)P.b[1] + k0 * P.ldb + t.n0, e, wave, lane, nvalid, P.ldb);
        dn::mainloop<dn::KC, dn::GLU, WTM>(ring, nsteps, [&](int s, uint32_t st, int i) {
          if (i < LA)
            issue_a(s, st, i);
          else if (i < LA + 2)
            og.issue(st + AB, wave, i - LA, (uint32_t)s * sb);
          else
            ou.issue(st + AB + 8192u, wave, i - LA - 2, (uint32_t)s * sb);
        }, acc, wm, wn, lane);
      }
    }
  }
  dense_store_tile<FORM, WTM>(P, t, (float*)lds, acc, wm, wn, lane, wave);
}

// The small tiles: operands as above, two K slices of 32 a step.
template <int FORM, int MB, int NB, bool SHORT>
__global__ __launch_bounds__(256) void dense_bf16_small_kernel(DenseParams P) {
  using S = dn::Small<MB, NB, SHORT>;
  constexpr int BM = 64 * MB, BN = FORM == kFormGlu ? 64 : 64 * NB;
  constexpr int ROW = 64 * NB + 4;   // floats of a staged row
  static_assert(BM * ROW * 4 <= S::RING, "epilogue stage must fit in the ring");
  __shared__ __attribute__((aligned(16))) uint16_t lds[S::RING / 2];
  DenseTile t;
  if (!dense_tile<FORM>(P, BM, BN, dn::SBK, t)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const uint32_t ring = bf::lds_base(lds);
  const uint32_t own = (uint32_t)wave * 1024u;   // this wave's share of a 64 x 32 part
  const int nsteps = t.s1 - t.s0;
  const int mvalid = (int)(P.M - t.m0 < BM ? P.M - t.m0 : BM), nvalid = P.N - t.n0;
  f32x16_t acc[MB][NB];
  if constexpr (FORM == kFormDw) {
    const int64_t k0 = (int64_t)t.s0 * dn::SBK;
    const int64_t kn = P.K - k0 < (int64_t)nsteps * dn::SBK ? P.K - k0 : (int64_t)nsteps * dn::SBK;
    dn::MncOp<64, 1> oa[MB], ob[NB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
      oa[m].init((const uint16_t*)P.a + k0 * P.lda + t.m0, ((kn - 1) * P.lda + up8(mvalid)) * 2, wave, lane, 64 * m, mvalid,
                 P.lda);
#pragma unroll
    for (int n = 0; n < NB; ++n)
      ob[n].init((const uint16_t*)P.b[0] + k0 * P.ldb + t.seg * P.seg + t.n0, ((kn - 1) * P.ldb + up8(nvalid)) * 2, wave,
                 lane, 64 * n, nvalid, P.ldb);
    const uint32_t sa = (uint32_t)(dn::BK * P.lda * 2), sb = (uint32_t)(dn::BK * P.ldb * 2);
    dn::small_mainloop<dn::MNC, dn::MNC, MB, NB, SHORT>(ring, nsteps, [&](int h, uint32_t at, int i) {
      if (i < MB)
        oa[i < MB ? i : 0].issue(at, wave, 0, (uint32_t)h * sa);
      else
        ob[i < MB ? 0 : i - MB].issue(at, wave, 0, (uint32_t)h * sb);
    }, acc, wm, wn, lane);
  } else {
    const int64_t a_cols = (FORM == kFormDx && P.nseg > 1 ? P.seg : 0) + up8(P.K);
    dn::KcPart<MB> oa;
    oa.init((const uint16_t*)P.a + t.m0 * P.lda, ((mvalid - 1) * P.lda + a_cols) * 2, wave, lane, mvalid, P.lda);
    const int kc = dn::KcOp<1>::chunk(lane) * 8;
    // half slices of a K segment
    const int halves_seg = 2 * (int)((P.K + dn::SBK - 1) / dn::SBK);
    if constexpr (FORM == kFormDx) {
      const int rows = nvalid < BN ? nvalid : BN;
      const int64_t eb = ((int64_t)(rows - 1) * P.ldb + up8(P.K)) * 2;
      dn::KcPart<NB> ob;
      ob.init((const uint16_t*)P.b[0] + (int64_t)t.n0 * P.ldb, eb, wave, lane, rows, P.ldb);
      const bf::i32x4_t rs1 = bf::make_rsrc((const uint16_t*)P.b[P.nseg - 1] + (int64_t)t.n0 * P.ldb, (uint32_t)eb);
      dn::small_mainloop<dn::KC, dn::KC, MB, NB, SHORT>(ring, nsteps, [&](int h, uint32_t at, int i) {
        const bool live = h < 2 * nsteps;
        int ks = live ? 2 * t.s0 + h : 0;
        const bool second = ks >= halves_seg;
        if (second) ks -= halves_seg;
        const bool ok = live && ks * dn::BK + kc < P.K;
        if (i < MB)
          bf::dma16(oa.rs, at + own, ok ? oa.voff[i < MB ? i : 0] : dn::kOOB,
                    (uint32_t)ks * 64u + (second ? (uint32_t)P.seg * 2u : 0u));
        else
          bf::dma16(second ? rs1 : ob.rs, at + own, ok ? ob.voff[i < MB ? 0 : i - MB] : dn::kOOB, (uint32_t)ks * 64u);
      }, acc, wm, wn, lane);
    } else {
      const int64_t k0 = (int64_t)t.s0 * dn::SBK, kn = P.K - k0;
      const uint32_t sb = (uint32_t)(dn::BK * P.ldb * 2);
      dn::MncOp<64, 1> ob[NB];
#pragma unroll
      for (int n = 0; n < NB; ++n)
        ob[n].init((const uint16_t*)P.b[FORM == kFormGlu ? n : 0] + k0 * P.ldb + t.n0,
                   ((kn - 1) * P.ldb + up8(nvalid)) * 2, wave, lane, FORM == kFormGlu ? 0 : 64 * n, nvalid, P.ldb);
      dn::small_mainloop<dn::KC, dn::MNC, MB, NB, SHORT>(ring, nsteps, [&](int h, uint32_t at, int i) {
        const bool live = h < 2 * nsteps;
        const int ks = live ? 2 * t.s0 + h : 0;
        if (i < MB)
          bf::dma16(oa.rs, at + own, live && ks * dn::BK + kc < P.K ? oa.voff[i < MB ? i : 0] : dn::kOOB, (uint32_t)ks * 64u);
        else
          ob[i < MB ? 0 : i - MB].issue(at, wave, 0, (uint32_t)h * sb);
      }, acc, wm, wn, lane);
    }
  }
  // through LDS, so that 16 lanes write 64 columns of a row
  float* stage = (float*)lds;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *(f32x4_t*)(stage + (mb * 64 + wm * 32 + (lane & 31)) * ROW + 64 * n + wn * 32 + 8 * i + 4 * (lane >> 5)) =
            f32x4_t{acc[mb][n][4 * i], acc[mb][n][4 * i + 1], acc[mb][n][4 * i + 2], acc[mb][n][4 * i + 3]};
  dense_lds_barrier();
  const int c = (lane & 15) * 4, m = 4 * wave + (lane >> 4);
  auto get = [&](int mb, int n, float (&v)[16]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4_t sv = *(const f32x4_t*)(stage + (mb * 64 + m + 16 * i) * ROW + 64 * n + c);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[4 * i + q] = sv[q];
    }
  };
#pragma unroll 1
  for (int p = 0; p < (FORM == kFormGlu ? MB : MB * NB); ++p) {
    const int mb = FORM == kFormGlu ? p : p / NB, n = FORM == kFormGlu ? 0 : p % NB;
    const int col = t.n0 + 64 * n + c;
    if (col >= P.N) continue;
    const AtRows at{t.m0 + mb * 64 + m, t.m0 + mvalid, 16, col};
    float v[16];
    get(mb, n, v);
    if constexpr (FORM == kFormGlu) {
      float u[16];
      get(mb, 1, u);
      if (P.S > 1) {
        part<4>(P, t.chunk, 0, at, v);
        part<4>(P, t.chunk, 1, at, u);
      } else {
        emit_glu<uint16_t, 4, SHORT>(P, at, v, u);
      }
    } else if (P.S > 1) {
      part<4>(P, t.chunk, t.seg, at, v);
    } else {
      emit<uint16_t, FORM, 4, SHORT, false>(P, t.seg, at, v);
    }
  }
}

// ------------------------------------------------------------- float32 tiles
// Tile (64 MB) x (64 NB) x 16 (the gated product: 32 NB columns of both
// matrices, NB = 2), 4 waves of MB x NB blocks of v_mfma_f32_32x32x2f32.  A
// thread holds the next kAhead slices in registers (a slice of a lone 64 x 64
// tile is multiplied in about 0.3 us, a fraction of the load latency) and
// copies one to LDS per step (three buffers, one barrier a slice).  LDS keeps each
// operand's own order: K-contiguous rows [64 B][20], read four k at a time, or
// [16][64 B + 4].  In both, the MFMA e of group q takes k = 8 q + e from lanes
// 0..31 and k = 8 q + 4 + e from lanes 32..63.
// Loads are buffer loads without branches (an offset past the buffer reads
// zero), so that the compiler's waits can count them; V4 says that every group of
// four columns is whole, otherwise elements are loaded one by one.
namespace f32t {
constexpr int BK = 16, KROW = 20, kAhead = 3;
constexpr uint32_t kOut = 0x80000000u;
template <int B>
constexpr int MROW = 64 * B + 4;
template <int B>
constexpr int OPER = 64 * B * KROW;   // floats of an operand's LDS buffer (the larger layout)

DEV __amdgpu_buffer_rsrc_t rsrc(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, 0x7fffffff, 0x00020000);
}
// four elements at byte offset o, of which the first n exist (n <= 0: none)
template <bool V4>
DEV f32x4_t load4(__amdgpu_buffer_rsrc_t r, uint32_t o, int n) {
  if constexpr (V4) return __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, n > 0 ? o : kOut, 0, 0));
  f32x4_t v;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    v[e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, n > e ? o + 4 * e : kOut, 0, 0));
  return v;
}

// The thread's part of an operand's slice: K-contiguous, row tid / 4 + 64 i and
// k = 4 (tid % 4); M/N-contiguous, k = tid / (16 B) + i (16 / B) and columns 4 (tid % (16 B)).
template <bool KCL, int B, bool V4>
struct Op {
  int mn[B], k[B];
  uint32_t off[B];
  int n[B];     // M/N-contiguous: columns that exist from this thread's first; K-contiguous: 1 if the row exists
  DEV void init(int tid, int64_t ld, int valid) {
#pragma unroll
    for (int i = 0; i < B; ++i) {
      mn[i] = KCL ? (tid >> 2) + 64 * i : 4 * (tid & (16 * B - 1));
      k[i] = KCL ? 4 * (tid & 3) : tid / (16 * B) + i * (16 / B);
      off[i] = (uint32_t)((KCL ? mn[i] * ld + k[i] : k[i] * ld + mn[i]) * 4);
      n[i] = KCL ? (mn[i] < valid ? 1 : 0) : valid - mn[i];
    }
  }
  // base: the slice's first k; left: k that remain from there
  DEV void load(f32x4_t (&v)[B], __amdgpu_buffer_rsrc_t r, int left) const {
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if constexpr (KCL)
        v[i] = load4<V4>(r, off[i], n[i] ? left - k[i] : 0);
      else
        v[i] = load4<V4>(r, off[i], k[i] < left ? n[i] : 0);
    }
  }
  DEV void store(float* s, const f32x4_t (&v)[B]) const {
#pragma unroll
    for (int i = 0; i < B; ++i) *(f32x4_t*)(s + (KCL ? mn[i] * KROW + k[i] : k[i] * MROW<B> + mn[i])) = v[i];
  }
};
template <bool KCL, int B>
DEV f32x4_t frag(const float* s, int row, int q, int half) {
  if constexpr (KCL) return *(const f32x4_t*)(s + row * KROW + 8 * q + 4 * half);
  const float* p = s + (8 * q + 4 * half) * MROW<B> + row;
  return f32x4_t{p[0], p[MROW<B>], p[2 * MROW<B>], p[3 * MROW<B>]};
}
}  // namespace f32t

namespace f32s {
// The upper 16 bits of a float32 number, which are a bf16 number.
DEV float cut(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
// Not zero where x is not the sum of its three bf16 parts (the third one's lower half).
DEV uint32_t cut_off(float x) {
  const float r = x - cut(x);
  return __float_as_uint(r - cut(r)) & 0xffffu;
}
}  // namespace f32s

// The product of a tile over its slices, for the tile of SUB slices of 16.
// MARK: `marks`, zeros before the call, then tells of each row of the tile (words 0..64
// MB - 1) and each column (the next 64 NB; the gated product's in the order of its LDS
// tile) whether it holds a number that is not the sum of its three bf16 parts; the caller
// waits for the other waves before it reads them.
template <int FORM, int MB, int NB, bool V4, int SUB, bool MARK>
DEV void f32_loop(const DenseParams& P, const DenseTile& t, float (*sa)[f32t::OPER<MB>], float (*sb)[f32t::OPER<NB>],
                  f32x16_t (&acc)[MB][NB], uint32_t* marks) {
  using namespace f32t;
  static_assert(FORM != kFormGlu || NB == 2, "a wave holds g and u of the same columns");
  constexpr int BM = 64 * MB;
  constexpr bool AK = FORM != kFormDw, BKC = FORM == kFormDx;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
  const int r32 = lane & 31, half = lane >> 5;
  const int mvalid = (int)(P.M - t.m0 < BM ? P.M - t.m0 : BM), nvalid = P.N - t.n0;
  const int steps_seg = (int)((P.K + BK * SUB - 1) / (BK * SUB));
  const int s0 = t.s0 * SUB, s1 = t.s1 * SUB;
  // the gated product's B slice is one load a thread from each matrix,
  // columns 0..63 of the LDS tile from wg, 64..127 from wu
  constexpr int OB = FORM == kFormGlu ? 1 : NB;
  Op<AK, MB, V4> oa;
  Op<BKC, OB, V4> ob;
  oa.init(tid, P.lda, mvalid);
  ob.init(tid, P.ldb, nvalid);
  f32x4_t ra[kAhead][MB], rb[kAhead][NB];
  auto load = [&](f32x4_t (&va)[MB], f32x4_t (&vb)[NB], int s) __attribute__((always_inline)) {
    const int whole = s / SUB;
    const bool second = FORM == kFormDx && whole >= steps_seg;
    const int64_t k = (int64_t)(second ? whole - steps_seg : whole) * (BK * SUB) + s % SUB * BK;
    // past the last slice nothing is left to load
    const int left = s < s1 ? (int)(P.K - k < BK ? P.K - k : BK) : 0;
    const float* pa = (const float*)P.a + (AK ? t.m0 * P.lda + (second ? P.seg : 0) + k : k * P.lda + t.m0);
    oa.load(va, rsrc(pa), left);
    if constexpr (FORM == kFormDx) {
      ob.load(vb, rsrc((const float*)(second ? P.b[1] : P.b[0]) + t.n0 * P.ldb + k), left);
    } else if constexpr (FORM == kFormGlu) {
      f32x4_t v[1];
      ob.load(v, rsrc((const float*)P.b[0] + k * P.ldb + t.n0), left);
      vb[0] = v[0];
      ob.load(v, rsrc((const float*)P.b[1] + k * P.ldb + t.n0), left);
      vb[1] = v[0];
    } else {
      ob.load(vb, rsrc((const float*)P.b[0] + (FORM == kFormDw ? t.seg * P.seg : 0) + k * P.ldb + t.n0), left);
    }
  };
  auto store_b = [&](float* s, const f32x4_t (&v)[NB]) __attribute__((always_inline)) {
    if constexpr (FORM == kFormGlu) {
#pragma unroll
      for (int i = 0; i < NB; ++i) *(f32x4_t*)(s + ob.k[0] * MROW<NB> + 64 * i + ob.mn[0]) = v[i];
    } else {
      ob.store(s, v);
    }
  };
#pragma unroll
  for (int a = 0; a < MB; ++a)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;
  // Slice s sits in LDS buffer s % 3.  In step s, slice s + 2 goes from
  // registers to the buffer that step s - 1 read, slice s + 5 is loaded, and each
  // half slice is read from LDS while the one before it is multiplied; slice
  // s + 1 was stored before the barrier that ended step s - 1.
  struct Half {
    f32x4_t a[MB], b[NB];
  };
  auto read = [&](Half& f, int buf, int q) __attribute__((always_inline)) {
#pragma unroll
    for (int x = 0; x < MB; ++x) f.a[x] = frag<AK, MB>(sa[buf], (wm * MB + x) * 32 + r32, q, half);
#pragma unroll
    for (int x = 0; x < NB; ++x)
      f.b[x] = frag<BKC, NB>(sb[buf], (FORM == kFormGlu ? x * 64 + wn * 32 : (wn * NB + x) * 32) + r32, q, half);
  };
  auto mul = [&](const Half& f) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          acc[mb][nb] = __builtin_amdgcn_mfma_f32_32x32x2f32(f.b[nb][e], f.a[mb][e], acc[mb][nb], 0, 0, 0);
  };
  uint32_t la[4] = {0, 0, 0, 0}, lb[2][4] = {};
  auto fill = [&](auto J, int s) __attribute__((always_inline)) {   // set J to its buffer, then slice s into set J
    constexpr int j = decltype(J)::value;
    if constexpr (MARK) {
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) la[AK ? i : e] |= f32s::cut_off(ra[j][i][e]);
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) lb[FORM == kFormGlu ? i : 0][BKC ? i : e] |= f32s::cut_off(rb[j][i][e]);
    }
    oa.store(sa[j], ra[j]);
    store_b(sb[j], rb[j]);
    load(ra[j], rb[j], s);
  };
  typedef std::integral_constant<int, 0> J0;
  typedef std::integral_constant<int, 1> J1;
  typedef std::integral_constant<int, 2> J2;
  static_assert(kAhead == 3, "three register sets and buffers");
  Half f0, f1;
  auto step = [&](int s, auto J, auto J2nd) __attribute__((always_inline)) {
    constexpr int j = decltype(J)::value;
    fill(J2nd, s + 5);
    read(f1, j, 1);
    mul(f0);
    read(f0, (j + 1) % 3, 0);
    mul(f1);
    __syncthreads();
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) load(ra[j], rb[j], s0 + j);
  int s = s0;
  fill(J0{}, s + 3);
  fill(J1{}, s + 4);
  __syncthreads();
  read(f0, 0, 0);
#pragma unroll 1
  for (; s + 3 <= s1; s += 3) {
    step(s, J0{}, J2{});
    step(s + 1, J1{}, J0{});
    step(s + 2, J2{}, J1{});
  }
  if (s < s1) step(s, J0{}, J2{});
  if (s + 1 < s1) step(s + 1, J1{}, J0{});
  if constexpr (MARK) {   // several threads may write the same word, all of them 1
    uint32_t* mb = marks + 64 * MB;
#pragma unroll
    for (int i = 0; i < (AK ? MB : 4); ++i)
      if (la[i]) marks[AK ? oa.mn[AK ? i : 0] : oa.mn[0] + i] = 1;
#pragma unroll
    for (int m = 0; m < (FORM == kFormGlu ? 2 : 1); ++m)
#pragma unroll
      for (int i = 0; i < (BKC ? NB : 4); ++i)
        if (lb[m][i]) mb[BKC ? ob.mn[BKC ? i : 0] : 64 * m + ob.mn[0] + i] = 1;
  }
}

// The epilogue of a tile whose wave holds MB x NB blocks.
template <int FORM, int MB, int NB>
DEV void f32_store(const DenseParams& P, const DenseTile& t, f32x16_t (&acc)[MB][NB]) {
  constexpr int BM = 64 * MB;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
  const int r32 = lane & 31, half = lane >> 5;
  const int mvalid = (int)(P.M - t.m0 < BM ? P.M - t.m0 : BM);
  // lane l holds row l % 32 and columns 8 i + 4 (l / 32) + 0..3 of each
  // block; one loop body for all blocks, whose registers are picked by
  // uniform branches
#pragma unroll 1
  for (int b = 0; b < (FORM == kFormGlu ? MB : MB * NB); ++b) {
    float v[16], u[16];
#pragma unroll
    for (int c = 0; c < MB * NB; ++c) {
      if (FORM == kFormGlu ? c / NB != b : c != b) continue;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        if (FORM == kFormGlu && c % NB == 1)
          u[r] = acc[c / NB][c % NB][r];
        else
          v[r] = acc[c / NB][c % NB][r];
      }
    }
    const int mb = FORM == kFormGlu ? b : b / NB, nb = FORM == kFormGlu ? 0 : b % NB;
    const int m = (wm * MB + mb) * 32 + r32;
    if (m >= mvalid) continue;
    const AtCols at{t.m0 + m, 8, t.n0 + (FORM == kFormGlu ? wn * 32 : (wn * NB + nb) * 32) + 4 * half};
    if constexpr (FORM == kFormGlu) {
      if (P.S > 1) {
        part<4>(P, t.chunk, 0, at, v);
        part<4>(P, t.chunk, 1, at, u);
      } else {
        emit_glu<float, 4, true>(P, at, v, u);
      }
    } else {
      if (P.S > 1)
        part<4>(P, t.chunk, t.seg, at, v);
      else
        emit<float, FORM, 4, true, false>(P, t.seg, at, v);
    }
  }
}

template <int FORM, int MB, int NB, bool V4>
__global__ __launch_bounds__(256) void dense_f32_kernel(DenseParams P) {
  using namespace f32t;
  __shared__ __attribute__((aligned(16))) float sa[kAhead][OPER<MB>], sb[kAhead][OPER<NB>];
  DenseTile t;
  if (!dense_tile<FORM>(P, 64 * MB, FORM == kFormGlu ? 32 * NB : 64 * NB, BK, t)) return;
  f32x16_t acc[MB][NB];
  f32_loop<FORM, MB, NB, V4, 1, false>(P, t, sa, sb, acc, nullptr);
  f32_store<FORM, MB, NB>(P, t, acc);
}

// ------------------------------------------------- float32 tiles in three parts
// The same 128 x 128 tile (64 columns of both matrices for the gated product)
// at the rate of the bf16 matrix instructions.  A float32 number is the exact
// sum of three bf16 numbers, its significand cut into three runs of 8 bits:
//   x = h + m + l,   h = cut(x),  m = cut(x - h),  l = x - h - m,
// |m| < 2^-7 |x| and |l| < 2^-15 |x|, all of x's sign, so
//   a b = l_a h_b + h_a l_b + m_a m_b + m_a h_b + h_a m_b + h_a h_b + e,
// where e, the three products left out, lies between 0 and 2^-21 a b, 2^-25 a b on
// average: a common factor of the result below the rounding of one float32
// product, beside a part that differs from product to product.  (Against float64,
// 4096^3 normal numbers: 1.02e-6 of the norm, the library's float32 product
// 1.15e-6; 2048^3: 7.1e-7 against 8.1e-7.)  Each product of two bf16
// numbers is exact, the sums are float32.  Six v_mfma_f32_32x32x16_bf16 do the work
// of eight v_mfma_f32_32x32x2f32 in three eighths of their time.
//
// An infinite or NaN number has no such parts: its m is NaN, which reaches every
// sum it takes part in.  A number below 2^-110 may have a bit below 2^-133, the smallest
// bf16 number: then the lower half of x - h - m is not zero, which every split is
// checked for.  And the small parts' products leave the float32 range before the
// numbers' own do.  So every sum of a row or column with a number that is not its three
// parts, and every sum that is not finite, or smaller than 2^-80 and not zero, is computed
// again with the float32 instructions (with its whole tile, whose other sums stay
// as they are: a row's bits do not depend on another row's numbers) and is what a
// float32 product gives.  The check is two of the split's 24 vector instructions per four
// numbers.
//
// A slice is 32 k.  A thread loads 4 groups of four numbers of each operand two
// slices ahead, splits the groups of the next-but-one slice between the
// matrix instructions of the current one, and stores the parts into one of three LDS
// buffers; each part is a [128][32] or [32][128] tile in the layouts of the bf16
// kernels (no bank conflicts).
namespace f32s {
constexpr int BK = 32, PART = 128 * BK * 2, OPER = 3 * PART, BUF = 2 * OPER, NBUF = 3;   // bytes

// The groups of four that a thread loads: K-contiguous, rows tid / 8 + 32 i and
// k = 4 (tid % 8); M/N-contiguous, k = tid / 32 + 8 i and columns 4 (tid % 32);
// the gated product's B, k = tid / 16 + 16 (i % 2) and columns 4 (tid % 16)
// of matrix i / 2.
template <bool KCL, bool GLU, bool V4>
struct Op {
  int k0, n[4];
  uint32_t off[4];
  uint32_t dst[GLU ? 2 : 1];   // LDS byte offset of group 0 in a part (GLU: also of group 2)
  DEV void init(int tid, int64_t ld, int valid) {
    if constexpr (KCL) {
      const int r = tid >> 3;
      k0 = 4 * (tid & 7);
      dst[0] = 2u * (uint32_t)(bf::kc_off(r, k0 >> 3) + (k0 & 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        off[i] = (uint32_t)(((r + 32 * i) * ld + k0) * 4);
        n[i] = r + 32 * i < valid ? 1 : 0;
      }
    } else {
      const int c = GLU ? 4 * (tid & 15) : 4 * (tid & 31);
      k0 = GLU ? tid >> 4 : tid >> 5;
      dst[0] = 2u * (uint32_t)dn::mnc128_off(k0, c);
      if constexpr (GLU) dst[1] = 2u * (uint32_t)dn::mnc128_off(k0, 64 + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        off[i] = (uint32_t)(((k0 + kOf(i)) * ld + c) * 4);
        n[i] = valid - c;
      }
    }
  }
  DEV static int kOf(int i) { return GLU ? 16 * (i & 1) : 8 * i; }
  // group i of a slice with `left` k, from r
  DEV f32x4_t load(__amdgpu_buffer_rsrc_t r, int i, int left) const {
    if constexpr (KCL) return f32t::load4<V4>(r, off[i], n[i] ? left - k0 : 0);
    return f32t::load4<V4>(r, off[i], k0 + kOf(i) < left ? n[i] : 0);
  }
  // group i's place: rows 32 i (K-contiguous) or k rows further, where the
  // swizzles repeat
  DEV uint32_t place(int i) const {
    if constexpr (GLU) return dst[i >> 1] + 4096u * (i & 1);
    return dst[0] + 2048u * i;
  }
};

// The three parts of four numbers; what the last one cuts off goes into `off`.
DEV uint32_t upper_halves(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
DEV void split4(const f32x4_t& x, u32x2_t& h, u32x2_t& m, u32x2_t& l, uint32_t& off) {
  float r[4], q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = x[i] - cut(x[i]);
    q[i] = r[i] - cut(r[i]);
  }
  h = u32x2_t{upper_halves(x[0], x[1]), upper_halves(x[2], x[3])};
  m = u32x2_t{upper_halves(r[0], r[1]), upper_halves(r[2], r[3])};
  l = u32x2_t{upper_halves(q[0], q[1]), upper_halves(q[2], q[3])};
  // Written out as one unit of the schedule: as C the two went in front of the matrix
  // instructions (4096^3: 780 us without the check, 826 in C, 790 so).
  asm("v_or3_b32 %0, %1, %2, %0\n\tv_or3_b32 %0, %3, %4, %0" : "+v"(off) : "v"(q[0]), "v"(q[1]), "v"(q[2]), "v"(q[3]));
}

// Fragment addresses of an operand's two 32-row blocks, relative to a buffer.
template <bool KCL, bool GLU>
struct Addr {
  uint32_t a[4];
  DEV void init(uint32_t base, int first, int lane) {
    if constexpr (KCL) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) a[kk] = base + 2u * (uint32_t)bf::kc_off(first + (lane & 31), 2 * kk + (lane >> 5));
    } else {
      const int g = lane >> 4, i = lane & 15;
      const int k = 8 * (g >> 1) + (i >> 2);
#pragma unroll
      for (int j = 0; j < 4; ++j) {   // block j / 2, rows k + 4 (j % 2)
        const int mn = first + (GLU ? 64 : 32) * (j >> 1) + 16 * (g & 1) + 4 * (i & 3);
        a[j] = base + 2u * (uint32_t)dn::mnc128_off(k + 4 * (j & 1), mn);
      }
    }
  }
  DEV bf16x8_t read(uint32_t buf, int block, int part, int kk) const {
    if constexpr (KCL) {
      const LDS_AS char* p = (const LDS_AS char*)(uintptr_t)(buf + a[kk]);
      return __builtin_bit_cast(bf16x8_t, *(const LDS_AS u32x4_t*)(p + PART * part + 2048 * block));
    } else {
      const LDS_AS char* lo = (const LDS_AS char*)(uintptr_t)(buf + a[2 * block]);
      const LDS_AS char* hi = (const LDS_AS char*)(uintptr_t)(buf + a[2 * block + 1]);
      bf::v4i16 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS bf::v4i16*)(lo + PART * part + 4096 * kk));
      bf::v4i16 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS bf::v4i16*)(hi + PART * part + 4096 * kk));
      const u32x2_t l2 = __builtin_bit_cast(u32x2_t, x), h2 = __builtin_bit_cast(u32x2_t, y);
      return __builtin_bit_cast(bf16x8_t, u32x4_t{l2[0], l2[1], h2[0], h2[1]});
    }
  }
};
// parts of A and B of the six products, smallest first: (l,h) (h,l) (m,m) (m,h) (h,m) (h,h)
constexpr int kPa[6] = {2, 0, 1, 1, 0, 0}, kPb[6] = {0, 2, 1, 0, 1, 0};
}  // namespace f32s

template <int FORM, bool V4>
__global__ __launch_bounds__(256) void dense_f32s_kernel(DenseParams P) {
  using namespace f32s;
  __shared__ __attribute__((aligned(16))) char lds[NBUF * BUF];
  constexpr bool AK = FORM != kFormDw, BKC = FORM == kFormDx, GLU = FORM == kFormGlu;
  DenseTile t;
  if (!dense_tile<FORM>(P, 128, GLU ? 64 : 128, BK, t)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave >> 1, wn = wave & 1;
  const int mvalid = (int)(P.M - t.m0 < 128 ? P.M - t.m0 : 128), nvalid = P.N - t.n0;
  const int steps_seg = (int)((P.K + BK - 1) / BK);
  const uint32_t base = bf::lds_base(lds);
  Op<AK, false, V4> oa;
  Op<BKC, GLU, V4> ob;
  oa.init(tid, P.lda, mvalid);
  ob.init(tid, P.ldb, nvalid);
  Addr<AK, false> fa;
  Addr<BKC, GLU> fb;
  fa.init(base, wm * 64, lane);
  fb.init(base + OPER, GLU ? wn * 32 : wn * 64, lane);
  f32x4_t ra[2][4], rb[2][4];
  struct Src {   // where slice s comes from
    __amdgpu_buffer_rsrc_t a, b, u;
    int left;
  };
  auto src = [&](int s) __attribute__((always_inline)) {
    const bool second = FORM == kFormDx && s >= steps_seg;
    const int64_t k = (int64_t)(second ? s - steps_seg : s) * BK;
    Src q;
    q.left = s < t.s1 ? (int)(P.K - k < BK ? P.K - k : BK) : 0;   // past the last slice: nothing
    q.a = f32t::rsrc((const float*)P.a + (AK ? t.m0 * P.lda + (second ? P.seg : 0) + k : k * P.lda + t.m0));
    q.b = f32t::rsrc((const float*)(second ? P.b[1] : P.b[0]) +
                     (BKC ? t.n0 * P.ldb + k : (FORM == kFormDw ? t.seg * P.seg : 0) + k * P.ldb + t.n0));
    if constexpr (GLU) q.u = f32t::rsrc((const float*)P.b[1] + k * P.ldb + t.n0);
    return q;
  };
  // group u (0..3 of A, 4..7 of B) of a slice
  auto load1 = [&](f32x4_t (&va)[4], f32x4_t (&vb)[4], const Src& q, int u) __attribute__((always_inline)) {
    if (u < 4)
      va[u & 3] = oa.load(q.a, u & 3, q.left);
    else
      vb[u & 3] = ob.load(GLU && u >= 6 ? q.u : q.b, u & 3, q.left);
  };
  auto load = [&](f32x4_t (&va)[4], f32x4_t (&vb)[4], int s) __attribute__((always_inline)) {
    const Src q = src(s);
#pragma unroll
    for (int u = 0; u < 8; ++u) load1(va, vb, q, u);
  };
  uint32_t off = 0;
  // group u of a register set, split, into the buffer at buf
  auto put = [&](const f32x4_t (&va)[4], const f32x4_t (&vb)[4], uint32_t buf, int u) __attribute__((always_inline)) {
    u32x2_t h, m, l;
    split4(u < 4 ? va[u & 3] : vb[u & 3], h, m, l, off);
    LDS_AS char* p = (LDS_AS char*)(uintptr_t)(base + buf + (u < 4 ? oa.place(u & 3) : OPER + ob.place(u & 3)));
    *(LDS_AS u32x2_t*)p = h;
    *(LDS_AS u32x2_t*)(p + PART) = m;
    *(LDS_AS u32x2_t*)(p + 2 * PART) = l;
  };
  struct Frag {
    bf16x8_t a[2][3], b[2][3];
  };
  // third g of a half slice's fragments, in the order the products need them
  auto read3 = [&](Frag& f, uint32_t buf, int kk, int g) __attribute__((always_inline)) {
    const int pa = g == 0 ? 2 : g == 1 ? 0 : 1, pb = g == 0 ? 0 : g == 1 ? 2 : 1;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      f.a[x][pa] = fa.read(buf, x, pa, kk);
      f.b[x][pb] = fb.read(buf, x, pb, kk);
    }
  };
  f32x16_t acc[2][2];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;
  // product j (0..23) of a k half: part pair j / 4, block j % 4
  auto mul6 = [&](const Frag& f, int j0) __attribute__((always_inline)) {
#pragma unroll
    for (int j = j0; j < j0 + 6; ++j) {
      const int q = j >> 2, mb = (j >> 1) & 1, nb = j & 1;
      acc[mb][nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.b[nb][kPb[q]], f.a[mb][kPa[q]], acc[mb][nb], 0, 0, 0);
    }
  };
  // six products with the splitting of one group, its next load and a third of
  // a fragment set between them.  (4096^3: 203 us a round of tiles; 206 us with the
  // reads and loads in one run per half.)
  auto mix = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one matrix instruction
      __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);   // four vector ones
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  Frag f0, f1;
  // Slice s lies in buffer s % 3 (byte offsets c, n, w of slices s, s + 1, s +
  // 2).  In step s the parts of slice s + 2 are stored from the set that holds it,
  // which then loads slice s + 4; slice s + 1 was stored before the barrier that
  // ended step s - 1, so its first half can be read before this step's barrier.
  auto step = [&](f32x4_t (&va)[4], f32x4_t (&vb)[4], int s, uint32_t c, uint32_t n, uint32_t w) __attribute__((always_inline)) {
    const Src q = src(s + 4);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      mul6(u < 4 ? f0 : f1, 6 * (u & 3));
      put(va, vb, w, u);
      load1(va, vb, q, u);
      if (u < 3) read3(f1, c, 1, u);
      if (u >= 4 && u < 7) read3(f0, n, 0, u - 4);
      mix();
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // loads stay in flight
  };
  load(ra[0], rb[0], t.s0);
  load(ra[1], rb[1], t.s0 + 1);
#pragma unroll
  for (int u = 0; u < 8; ++u) put(ra[0], rb[0], 0, u);
  load(ra[0], rb[0], t.s0 + 2);
#pragma unroll
  for (int u = 0; u < 8; ++u) put(ra[1], rb[1], BUF, u);
  load(ra[1], rb[1], t.s0 + 3);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
  for (int g = 0; g < 3; ++g) read3(f0, 0, 0, g);
  uint32_t c = 0, n = BUF, w = 2 * BUF;
  int s = t.s0;
#pragma unroll 1
  for (; s + 2 <= t.s1; s += 2) {
    step(ra[0], rb[0], s, c, n, w);
    step(ra[1], rb[1], s + 1, n, w, c);
    const uint32_t x = c;   // two slices on
    c = w;
    w = n;
    n = x;
  }
  if (s < t.s1) step(ra[0], rb[0], s, c, n, w);
  // One bit a sum: not finite, or between 0 and 2^-80 (sums of rows and columns that
  // do not exist are zeros, which are kept).  Whole words, opaque to the compiler,
  // rather than 64 lane masks that live through the second loop.
  uint32_t bad[2] = {0, 0};
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const uint32_t v = __float_as_uint(acc[a][b][r]) & 0x7fffffffu;
        bad[a] |= (uint32_t)((v >= 0x7f800000u) | (v - 1 < 0x17800000u - 1)) << (16 * b + r);
      }
  asm volatile("" : "+v"(bad[0]), "+v"(bad[1]));
  if (__syncthreads_or((bad[0] | bad[1] | (off & 0xffffu)) != 0)) {
    constexpr int A = f32t::kAhead * f32t::OPER<2>;
    static_assert((2 * A + 256) * 4 <= NBUF * BUF, "the float32 buffers and marks fit");
    float* f = (float*)lds;
    uint32_t* marks = (uint32_t*)(f + 2 * A);
    marks[tid] = 0;
    f32x16_t again[2][2];
    f32_loop<FORM, 2, 2, V4, 2, true>(P, t, (float (*)[f32t::OPER<2>])f, (float (*)[f32t::OPER<2>])(f + A), again, marks);
    __syncthreads();
    // lane l holds rows l % 32 and columns 8 i + 4 (l / 32) + 0..3 of each block (f32_store)
    uint32_t cols = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int col = (GLU ? 64 * b + 32 * wn : 64 * wn + 32 * b) + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        cols |= marks[128 + col] << (16 * b + r);
      }
#pragma unroll
    for (int a = 0; a < 2; ++a) bad[a] |= marks[64 * wm + 32 * a + (lane & 31)] ? ~0u : cols;
    asm volatile("" : "+v"(bad[0]), "+v"(bad[1]));
    // the other sums keep their bits, whatever another row or column holds
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          acc[a][b][r] = bad[a] >> (16 * b + r) & 1 ? again[a][b][r] : acc[a][b][r];
  }
  f32_store<FORM, 2, 2>(P, t, acc);
}

// ------------------------------------------------------------------ few rows
// Weights [K][N] streamed once past at most 16 MT rows of x, mostly in one
// launch and without a workspace (S = 1).  A workgroup owns 64 bytes of every weight row (32 bf16
// or 16 float32 columns) of its chunk; its NW waves take 32-row K steps in turn and add their
// sums in wave order through LDS.  In a step, lane (i = l % 16, g = l / 16) loads
// its 4 bytes of the weights' rows 8 g .. 8 g + 7 and 8 consecutive k of
// each x row i: both go from the loads to the matrix instruction's registers
// directly, with no LDS and no barrier, and DEPTH steps are in flight.
//  bf16     v_mfma_f32_16x16x32_bf16, one per column: a column's 8 k are
//           picked out of the 8 loaded rows with one byte permute per pair.
//  float32  v_mfma_f32_16x16x4f32, 8 per column.
// Rows of x past the last repeat it (their sums are not used).
template <typename T, int FORM, int MT>
struct FewCfg {
  static constexpr int NM = FORM == kFormGlu ? 2 : 1;         // matrices
  static constexpr int CPL = 4 / (int)sizeof(T);              // columns per lane and matrix
  static constexpr int COLS = 16 * CPL;                       // tile columns per matrix
  static constexpr int NW = MT == 1 ? 16 : 8;                 // waves
  static constexpr int DEPTH = sizeof(T) == 2 ? 4 : 3;
};

template <typename T, int FORM, int MT>
__global__ __launch_bounds__((FewCfg<T, FORM, MT>::NW * 64)) void dense_few_kernel(DenseParams P) {
  using Cfg = FewCfg<T, FORM, MT>;
  constexpr int NM = Cfg::NM, CPL = Cfg::CPL, COLS = Cfg::COLS, NW = Cfg::NW, DEPTH = Cfg::DEPTH, RS = NM * COLS + 4;
  constexpr int XW = sizeof(T) == 2 ? 1 : 2;   // 16-byte loads of 8 consecutive k
  __shared__ __attribute__((aligned(16))) float s_acc[NW * 16 * MT * RS];
  // Chunk, then pairs of tiles dealt to the 8 XCDs in turn: the two 64-byte
  // tiles of a 128-byte line share an XCD's L2, and an XCD's tiles lie 1 KiB apart
  // (in one run they would use two of its L2's channels; measured against
  // consecutive tiles: 37 rows of the 2048 x 8192 gated product 15.0 against
  // 16.9 us, 5 rows of 8192 x 2048 unsplit 16.6 against 18.3 us).
  const int tiles = (P.N + COLS - 1) / COLS, tgrid = (tiles + 15) / 16 * 16;
  int b = blockIdx.x;
  if (P.seed) {
    shuffle_delay(P.seed, b);
    b = (int)shuffle_unit(b, (int64_t)tgrid * P.S, P.seed);
  }
  const int chunk = b / tgrid, tb = b - chunk * tgrid;
  const int tile = (tb / 16 * 8 + tb % 8) * 2 + tb / 8 % 2;
  if (tile >= tiles) return;
  const int n0 = tile * COLS;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), i16 = lane & 15, g = lane >> 4;
  const int K = (int)P.K;
  const int all = (K + 31) / 32;
  const int s0 = (int)((int64_t)chunk * all / P.S), steps = (int)((int64_t)(chunk + 1) * all / P.S);
  const int col = n0 + i16 * CPL, ncol = P.N - col;
  f32x4_t acc[NM][CPL][MT];
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int c = 0; c < CPL; ++c)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[m][c][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  struct Step {
    uint32_t w[NM][8];
    typename Vec<T>::raw x[MT][XW];
  };
  const T* xrow[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int row = 16 * t + i16;
    xrow[t] = (const T*)P.a + (int64_t)(row < P.M ? row : (int)P.M - 1) * P.lda;
  }
  auto load = [&](Step& b, int s) __attribute__((always_inline)) {
    const int k = 32 * s + 8 * g;
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int r = 0; r < 8; ++r) b.w[m][r] = *(const u32_any_t*)((const T*)P.b[m] + (int64_t)(k + r) * P.ldb + col);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int h = 0; h < XW; ++h) b.x[t][h] = Vec<T>::load(xrow[t] + k + h * Vec<T>::N, Vec<T>::N);
  };
  auto load_edge = [&](Step& b, int s) __attribute__((always_inline)) {
    const int k = 32 * s + 8 * g;
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        b.w[m][r] = 0u;
        const T* p = (const T*)P.b[m] + (int64_t)(k + r) * P.ldb + col;
        if (k + r < K && ncol >= CPL)
          b.w[m][r] = *(const u32_any_t*)p;
        else if (k + r < K && ncol > 0)
          b.w[m][r] = *(const uint16_t*)p;   // the last of an odd number of bf16 columns
      }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int h = 0; h < XW; ++h) {
        const int kk = k + h * Vec<T>::N;
        b.x[t][h] = typename Vec<T>::raw{};
        if (kk < K) b.x[t][h] = Vec<T>::load(xrow[t] + kk, K - kk);
      }
  };
  auto mma = [&](const Step& b) __attribute__((always_inline)) {
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        if constexpr (sizeof(T) == 2) {
          u32x4_t f;
#pragma unroll
          for (int p = 0; p < 4; ++p)
            f[p] = __builtin_amdgcn_perm(b.w[m][2 * p + 1], b.w[m][2 * p], c ? 0x07060302u : 0x05040100u);
#pragma unroll
          for (int t = 0; t < MT; ++t)
            acc[m][c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, b.x[t][0]),
                                                                   __builtin_bit_cast(bf16x8_t, f), acc[m][c][t], 0, 0, 0);
        } else {
#pragma unroll
          for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int t = 0; t < MT; ++t)
              acc[m][c][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                  __builtin_bit_cast(f32x4_t, b.x[t][r >> 2])[r & 3], __uint_as_float(b.w[m][r]), acc[m][c][t], 0, 0, 0);
        }
      }
  };
  // steps below `whole` lie inside the matrix in both directions
  const int whole = n0 + COLS <= P.N ? min(K / 32, steps) : 0, first = s0 + wave;
  // this wave's whole steps in rounds of DEPTH.  Loads are unconditional, so
  // that the waits can count them: past the last whole step they repeat it, and the last
  // round loads nothing.
  const int n = whole > first ? (whole - first + NW - 1) / NW : 0;
  if (n > 0) {
    Step st[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(st[d], first + (d < n ? d : n - 1) * NW);
    int i = 0;
#pragma unroll 1
    for (; i + DEPTH < n; i += DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        mma(st[d]);
        const int j = i + DEPTH + d;
        load(st[d], first + (j < n ? j : n - 1) * NW);
      }
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (i + d < n) mma(st[d]);
  }
  int s = first + n * NW;
#pragma unroll 1
  for (; s < steps; s += NW) {
    Step b;
    load_edge(b, s);
    mma(b);
  }
  // lane l holds rows 4 g + r and the columns CPL (l % 16) + c of its tiles
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < CPL; ++c)
          s_acc[((wave * MT + t) * 16 + 4 * g + r) * RS + m * COLS + i16 * CPL + c] = acc[m][c][t][r];
  __syncthreads();
  constexpr int QPR = COLS / 4;   // groups of four columns per row and matrix
  for (int o = tid; o < 16 * MT * QPR; o += NW * 64) {
    const int row = o / QPR, c = (o % QPR) * 4;
    if (row >= P.M || n0 + c >= P.N) continue;
    float v[NM][4];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const float* p = s_acc + row * RS + m * COLS + c;
      f32x4_t a = *(const f32x4_t*)p;
#pragma unroll
      for (int w = 1; w < NW; ++w) {
        const f32x4_t b = *(const f32x4_t*)(p + w * 16 * MT * RS);
#pragma unroll
        for (int q = 0; q < 4; ++q) a[q] = a[q] + b[q];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) v[m][q] = a[q];
    }
    if (P.S > 1) {
#pragma unroll
      for (int m = 0; m < NM; ++m) part4(P, chunk, m, row, n0 + c, v[m]);
    } else if constexpr (FORM == kFormGlu) {
      emit4_glu<T>(P, row, n0 + c, v[0], v[NM - 1]);
    } else {
      emit4<T, FORM>(P, 0, row, n0 + c, v[0]);
    }
  }
}

// -------------------------------------------------------------- join of chunks
// One thread per four columns: the chunks' partials in chunk order, then the
// epilogue.
template <typename T, int FORM>
DEV void finish_at(const DenseParams& P, uint32_t block) {
  const uint32_t q = ((uint32_t)P.N + 3) / 4, per = FORM == kFormDw ? q * P.nseg : q;
  const uint32_t i = block * 256u + threadIdx.x;   // a split product has fewer than 2^30 elements
  if (i >= (uint64_t)P.M * per) return;
  const int64_t row = i / per;
  const uint32_t rest = i % per;
  const int seg = rest >= q ? 1 : 0, col = (int)(rest - seg * q) * 4;
  auto sum = [&](int sg, float (&v)[4]) {
    const float* p = P.part + row * P.part_ld + sg * P.part_seg + col;
    f32x4_t a = *(const f32x4_t*)p;
#pragma unroll 4
    for (int s = 1; s < P.S; ++s) {
      const f32x4_t o = *(const f32x4_t*)(p + (int64_t)s * P.M * P.part_ld);
#pragma unroll
      for (int x = 0; x < 4; ++x) a[x] = a[x] + o[x];
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = a[x];
  };
  float v[4];
  sum(seg, v);
  if constexpr (FORM == kFormGlu) {
    float u[4];
    sum(1, u);
    emit4_glu<T>(P, row, col, v, u);
  } else {
    emit4<T, FORM>(P, seg, row, col, v);
  }
}

template <typename T, int FORM>
__global__ __launch_bounds__(256) void dense_finish_kernel(DenseParams P) {
  finish_at<T, FORM>(P, blockIdx.x);
}

// Everything that a backward call joins at its end, in one launch: the chunks
// of dx and of the weight gradients, and the row blocks' column sums.
// Workgroups [0, nx) join dx, [nx, nx + nw) dw, the others add column sums.
template <typename T>
__global__ __launch_bounds__(256) void dense_join_kernel(DenseJoin J) {
  const uint32_t b = blockIdx.x;
  if (b < J.nx)
    finish_at<T, kFormDx>(J.dx, b);
  else if (b < J.nx + J.nw)
    finish_at<T, kFormDw>(J.dw, b - J.nx);
  else
    block_sum16(J.sums, J.blocks, J.cols, J.cols, b - J.nx - J.nw, J.db, J.db_bf16);
}

// ---------------------------------------------------------- elementwise passes
// Up to three matrices copied into rows of whole 16-byte chunks, zeros past
// their columns: a matrix per range of workgroups.
DEV void pack_at(const DensePackParams& P, uint32_t block) {
  int m = 0;
  while (m + 1 < P.n && (int64_t)block >= P.first[m + 1]) ++m;
  // 32 bits: a launch has fewer than 2^32 threads
  const uint32_t q = (uint32_t)P.ldo[m] / 8;
  const uint32_t i = (block - (uint32_t)P.first[m]) * 256u + threadIdx.x;
  if (i >= (uint64_t)P.rows[m] * q) return;
  const int64_t row = i / q;
  const int c = (int)(i % q) * 8, left = P.cols[m] - c;
  u32x4_t r = {0u, 0u, 0u, 0u};
  if (left > 0) r = Vec<uint16_t>::load((const uint16_t*)P.in[m] + row * P.ld[m] + c, left);
  *(u32x4_t*)((uint16_t*)P.out[m] + row * P.ldo[m] + c) = r;
}
__global__ __launch_bounds__(256) void dense_pack_kernel(DensePackParams P) { pack_at(P, blockIdx.x); }

// V elements of a saved pre-activation, zeros past n >= 1
template <typename Z, int V>
DEV void load_z(const Z* p, int n, float* v) {
  constexpr int N = Vec<Z>::N;
#pragma unroll
  for (int i = 0; i < V / N; ++i) {
    typename Vec<Z>::raw r{};
    if (n > i * N) r = Vec<Z>::load(p + i * N, n - i * N);
    Vec<Z>::get(r, v + i * N);
  }
}

// dz = dy act'(z), or dg = da u act'(g) and du = da act(g).  A workgroup owns
// 64 V columns and a block of rows; its 4 waves take the rows in turn, and
// their column sums of the unrounded dz are added in wave order.  Workgroups
// past `grid` copy unaligned operands in the same launch.
//
// For bf16 storage dz, dg and du are rounded to bf16, since the products multiply bf16
// numbers (as the expert layer rounds dh); float32 ones would take two bf16 parts, twice
// the products' time.  It adds one rounding, 0.0017 of the norm, to the gradients'
// own: 0.0023 against float64 instead of 0.0017 (4096 x 2048 x 8192 gated).  The bias
// gradient sums the unrounded dz.
template <typename T, typename Z, bool GLU>
__global__ __launch_bounds__(256) void dense_ew_kernel(DenseEwParams P, DensePackParams K, uint32_t grid) {
  if (blockIdx.x >= grid) {
    pack_at(K, blockIdx.x - grid);
    return;
  }
  constexpr int V = Vec<T>::N, CT = 64 * V;
  __shared__ float s_sum[3][CT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cT = (P.pad + CT - 1) / CT;
  const int64_t units = (int64_t)P.blocks * cT;
  const int64_t L = map_unit(blockIdx.x, units, P.seed);
  if (L < 0) return;
  const int64_t blk = L / cT;
  const int col = (int)(L % cT) * CT + lane * V;
  const int64_t r0 = blk * P.rows / P.blocks, r1 = (blk + 1) * P.rows / P.blocks;
  const int n = P.cols - col, no = P.pad - col;
  const bool need_z = GLU || P.act != kActNone;
  float sum[V];
#pragma unroll
  for (int q = 0; q < V; ++q) sum[q] = 0.f;
  // R rows at a time, loaded before any is used; a wave's columns are whole
  // except in the last column tile
  constexpr int R = 2;
  auto rows = [&](int64_t row, int count, auto WHOLE) __attribute__((always_inline)) {
    constexpr bool whole = decltype(WHOLE)::value;
    float d[R][V], z[R][V], u[R][V];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int q = 0; q < V; ++q) d[i][q] = z[i][q] = u[i][q] = 0.f;
      if (i >= count || (!whole && n <= 0)) continue;
      const int64_t r = row + 4 * i;
      const int m = whole ? V : n;
      Vec<T>::get(Vec<T>::load((const T*)P.dy + r * P.lddy + col, m), d[i]);
      if (need_z) load_z<Z, V>((const Z*)P.z[0] + r * P.ldz + col, m, z[i]);
      if (GLU) load_z<Z, V>((const Z*)P.z[1] + r * P.ldz + col, m, u[i]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i >= count) continue;
      // past the row every load gave 0, and act(0) or act'(0) times 0 is 0
      float o0[V], o1[V];
      if (need_z) {
        float v[V], dv[V];
        act_df_n<sizeof(T) == 4, V>(P.act, z[i], v, dv);
#pragma unroll
        for (int q = 0; q < V; ++q) {
          o0[q] = GLU ? d[i][q] * u[i][q] * dv[q] : d[i][q] * dv[q];
          o1[q] = d[i][q] * v[q];
        }
      } else {
#pragma unroll
        for (int q = 0; q < V; ++q) o0[q] = o1[q] = d[i][q];
      }
      const int64_t at = (row + 4 * i) * P.ldo + col;
      const int m = whole ? V : no;
#pragma unroll
      for (int q = 0; q < V; ++q) sum[q] = sum[q] + o0[q];
      if (P.out[0]) Vec<T>::store((T*)P.out[0] + at, o0, m);
      if (GLU) Vec<T>::store((T*)P.out[1] + at, o1, m);
    }
  };
  if (no > 0) {
    const bool whole = (col - lane * V) + CT <= P.cols;   // uniform
    int64_t row = r0 + wave;
    if (whole) {
      for (; row + 4 * (R - 1) < r1; row += 4 * R) rows(row, R, std::true_type{});
      for (; row < r1; row += 4) rows(row, 1, std::true_type{});
    } else {
      for (; row < r1; row += 4) rows(row, 1, std::false_type{});
    }
  }
  if (GLU || !P.part) return;
  if (wave > 0)
#pragma unroll
    for (int q = 0; q < V; ++q) s_sum[wave - 1][q * 64 + lane] = sum[q];
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int q = 0; q < V; ++q) {
      float v = sum[q];
#pragma unroll
      for (int w = 0; w < 3; ++w) v = v + s_sum[w][q * 64 + lane];
      if (col + q < P.cols) P.part[blk * P.cols + col + q] = v;
    }
  }
}

__global__ __launch_bounds__(256) void dense_zero_kernel(uint16_t* p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0;
}

// -------------------------------------------------------------------- launches
DenseShape dense_shape(int form, bool bf16, int tile) {
  static constexpr DenseShape kBf16[kDenseBf16Tiles] = {{256, 256, 32}, {128, 256, 32}, {128, 128, 64}, {64, 64, 64}};
  static constexpr DenseShape kF32[kDenseF32Tiles] = {{128, 128, 32}, {64, 64, 16}};
  DenseShape s = bf16 ? kBf16[tile] : kF32[tile];
  // half the columns of both matrices; the 64-row tiles are twice as wide
  if (form == kFormGlu && s.bm > 64) s.bn /= 2;
  return s;
}

bool dense_short(const DenseParams& P, int form) {
  const int64_t steps = (P.K + dn::SBK - 1) / dn::SBK * (form == kFormDx ? P.nseg : 1);
  return steps <= 2 * (int64_t)P.S;
}
bool dense_v4(const DenseParams& P, int form) {
  const bool ka = form != kFormDw, kb = form == kFormDx;   // K-contiguous operands
  return (ka ? P.K : P.M) % 4 == 0 && (kb ? P.K : P.N) % 4 == 0;
}

template <int FORM, bool V4>
static void dense_f32_launch(const DenseParams& P, int tile, int64_t grid, hipStream_t st) {
  if (tile == 0)
    dense_f32s_kernel<FORM, V4><<<grid, 256, 0, st>>>(P);
  else
    dense_f32_kernel<FORM, 1, FORM == kFormGlu ? 2 : 1, V4><<<grid, 256, 0, st>>>(P);
}

template <int FORM>
static void dense_gemm_launch(const DenseParams& P, bool bf16, int tile, int64_t grid, hipStream_t st) {
  if (!bf16) {
    if (dense_v4(P, FORM))
      dense_f32_launch<FORM, true>(P, tile, grid, st);
    else
      dense_f32_launch<FORM, false>(P, tile, grid, st);
    return;
  }
  switch (tile) {
    case 0: dense_bf16_kernel<FORM, 128><<<grid, 256, 0, st>>>(P); break;
    case 1: dense_bf16_kernel<FORM, 64><<<grid, 256, 0, st>>>(P); break;
    case 2: dense_bf16_small_kernel<FORM, 2, 2, false><<<grid, 256, 0, st>>>(P); break;
    default: {
      constexpr int NB = FORM == kFormGlu ? 2 : 1;
      if (dense_short(P, FORM))
        dense_bf16_small_kernel<FORM, 1, NB, true><<<grid, 256, 0, st>>>(P);
      else
        dense_bf16_small_kernel<FORM, 1, NB, false><<<grid, 256, 0, st>>>(P);
    }
  }
}

hipError_t launch_dense_gemm(const DenseParams& P, int form, bool bf16, int tile, hipStream_t st) {
  const DenseShape sh = dense_shape(form, bf16, tile);
  const int64_t tiles = (P.M + sh.bm - 1) / sh.bm * ((P.N + sh.bn - 1) / sh.bn) * (form == kFormDw ? P.nseg : 1);
  const int64_t grid = grid_for_units(tiles * P.S);
  switch (form) {
    case kFormLinear: dense_gemm_launch<kFormLinear>(P, bf16, tile, grid, st); break;
    case kFormGlu: dense_gemm_launch<kFormGlu>(P, bf16, tile, grid, st); break;
    case kFormDx: dense_gemm_launch<kFormDx>(P, bf16, tile, grid, st); break;
    default: dense_gemm_launch<kFormDw>(P, bf16, tile, grid, st); break;
  }
  return hipGetLastError();
}

template <typename T, int FORM, int MT>
static void dense_few_launch(const DenseParams& P, hipStream_t st) {
  using Cfg = FewCfg<T, FORM, MT>;
  const int tiles = (P.N + Cfg::COLS - 1) / Cfg::COLS;
  dense_few_kernel<T, FORM, MT><<<(tiles + 15) / 16 * 16 * P.S, Cfg::NW * 64, 0, st>>>(P);
}

template <int FORM>
static void dense_few_form(const DenseParams& P, bool bf16, hipStream_t st) {
  if (!bf16 && P.M <= 16)
    dense_few_launch<float, FORM, 1>(P, st);
  else if (!bf16)
    dense_few_launch<float, FORM, 2>(P, st);
  else if (P.M <= 16)
    dense_few_launch<uint16_t, FORM, 1>(P, st);
  else if (P.M <= 32)
    dense_few_launch<uint16_t, FORM, 2>(P, st);
  else if (P.M <= 48)
    dense_few_launch<uint16_t, FORM, 3>(P, st);
  else
    dense_few_launch<uint16_t, FORM, 4>(P, st);
}

hipError_t launch_dense_few(const DenseParams& P, int form, bool bf16, hipStream_t st) {
  if (form == kFormGlu)
    dense_few_form<kFormGlu>(P, bf16, st);
  else
    dense_few_form<kFormLinear>(P, bf16, st);
  return hipGetLastError();
}

static uint32_t finish_blocks(const DenseParams& P, int form) {
  return (uint32_t)((P.M * ((P.N + 3) / 4) * (form == kFormDw ? P.nseg : 1) + 255) / 256);
}

template <typename T>
static void dense_finish_launch(const DenseParams& P, int form, int64_t grid, hipStream_t st) {
  switch (form) {
    case kFormLinear: dense_finish_kernel<T, kFormLinear><<<grid, 256, 0, st>>>(P); break;
    default: dense_finish_kernel<T, kFormGlu><<<grid, 256, 0, st>>>(P); break;
  }
}

hipError_t launch_dense_finish(const DenseParams& P, int form, bool bf16, hipStream_t st) {
  const int64_t grid = finish_blocks(P, form);
  if (bf16)
    dense_finish_launch<uint16_t>(P, form, grid, st);
  else
    dense_finish_launch<float>(P, form, grid, st);
  return hipGetLastError();
}

void DensePackParams::add(const void* src, int64_t r, int c, int64_t l, void* dst, int64_t lo) {
  if (n == 0) first[0] = 0;
  in[n] = src;
  rows[n] = r;
  cols[n] = c;
  ld[n] = l;
  out[n] = dst;
  ldo[n] = lo;
  first[n + 1] = first[n] + (r * (lo / 8) + 255) / 256;
  ++n;
}

hipError_t launch_dense_pack(const DensePackParams& P, hipStream_t st) {
  if (P.n == 0) return hipSuccess;
  dense_pack_kernel<<<P.first[P.n], 256, 0, st>>>(P);
  return hipGetLastError();
}

// Row blocks of the elementwise pass.  With column sums about 512 workgroups
// (every block adds a row of partials to write and read again; 4096 x 2048
// bf16: 4 MB of them with 2048 workgroups, 1 MB with 512), else about 2048; at
// least 4 rows each.
int dense_ew_blocks(int64_t rows, int cols, bool bf16, bool sums) {
  const int ct = bf16 ? 512 : 256;
  int64_t b = (sums ? 512 : 2048) / ((cols + ct - 1) / ct);
  const int64_t most = (rows + 3) / 4;
  if (b > most) b = most;
  return (int)(b < 1 ? 1 : b > 512 ? 512 : b);
}

template <typename T, typename Z>
static void dense_ew_launch(const DenseEwParams& P, const DensePackParams& K, bool glu, uint32_t grid, hipStream_t st) {
  const uint32_t all = grid + (K.n ? (uint32_t)K.first[K.n] : 0);
  if (glu)
    dense_ew_kernel<T, Z, true><<<all, 256, 0, st>>>(P, K, grid);
  else
    dense_ew_kernel<T, Z, false><<<all, 256, 0, st>>>(P, K, grid);
}

hipError_t launch_dense_ew(const DenseEwParams& P, const DensePackParams& K, bool glu, bool bf16, hipStream_t st) {
  const int ct = bf16 ? 512 : 256;
  const uint32_t grid = (uint32_t)grid_for_units((int64_t)P.blocks * ((P.pad + ct - 1) / ct));
  if (!bf16)
    dense_ew_launch<float, float>(P, K, glu, grid, st);
  else if (P.z_f32)
    dense_ew_launch<uint16_t, float>(P, K, glu, grid, st);
  else
    dense_ew_launch<uint16_t, uint16_t>(P, K, glu, grid, st);
  return hipGetLastError();
}

hipError_t launch_dense_join(const DenseParams& dx, const DenseParams& dw, const float* sums, int blocks, int cols,
                             void* db, bool db_bf16, bool bf16, hipStream_t st) {
  DenseJoin J{dx, dw, 0, 0, sums, blocks, cols, db, db_bf16};
  if (dx.S > 1) J.nx = finish_blocks(dx, kFormDx);
  if (dw.S > 1) J.nw = finish_blocks(dw, kFormDw);
  const uint32_t grid = J.nx + J.nw + (db ? (uint32_t)(cols + 15) / 16 : 0);
  if (grid == 0) return hipSuccess;
  if (bf16)
    dense_join_kernel<uint16_t><<<grid, 256, 0, st>>>(J);
  else
    dense_join_kernel<float><<<grid, 256, 0, st>>>(J);
  return hipGetLastError();
}

hipError_t launch_dense_zero(void* p, int64_t n16, hipStream_t st) {
  dense_zero_kernel<<<(n16 + 255) / 256, 256, 0, st>>>((uint16_t*)p, n16);
  return hipGetLastError();
}

}  // namespace moedet
