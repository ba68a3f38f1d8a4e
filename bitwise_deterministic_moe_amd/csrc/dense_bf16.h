// bf16 main loop of the dense matrix operators: the ring of gemm_bf16.h
// (32-row K slices copied by DMA into LDS slots, the loads of later
// slices spread between the MFMAs) with a tile of 256 or 128 rows, a B tile
// that may come from two matrices, K tails and K segments.
//
// Tile (2 WTM) x 256, K slice 32, 4 waves in a 2x2 grid, each wave WTM x 128 as blocks
// of v_mfma_f32_32x32x16_bf16.
//
// LDS layouts besides KC and MNC of gemm_bf16.h:
//  MNC tile of 128 columns: [32 k][128], rows of 256 bytes; chunk c (8
//      elements) of row k sits at c ^ 4*(k&3): the four k rows that a transpose read
//      takes then lie in four different 64-byte quarters of the row, and rows
//      k+8 follow a cycle later.
//  MNC tile of 64 columns (small tiles): [32 k][64], rows of 128 bytes; chunk c of
//      row k sits at c ^ 4*((k>>1)&1): four 64-byte quarters of two rows.
//  GLU the B tile of the gated product: a 128-column tile of wg, then one of
//      wu.  The wave wn holds columns 64 wn .. 64 wn + 63 of both, so a
//      lane ends with g and u of the same element.
#pragma once

#include "gemm_bf16.h"

namespace moedet {
namespace dn {

using bf::kOOB;
using bf::KC;
using bf::MNC;
constexpr int GLU = 2;
constexpr int BK = bf::BK, BN = 256, BOPER = BN * BK;

template <int WTM>
constexpr int kAOper = 2 * WTM * BK;             // elements of an A slot
template <int WTM>
constexpr int kSlot = kAOper<WTM> + BOPER;       // elements of a ring slot
// Ring slots: 4 of 32 KiB, or 6 of 24 KiB for the 128-row tile, whose slices are
// multiplied in half the time while the loads take as long.
template <int WTM>
constexpr int kSlots = WTM == 128 ? 4 : 6;
template <int WTM>
constexpr int kRingBytes = kSlots<WTM> * kSlot<WTM> * 2;
template <int WTM>
constexpr int kALoads = WTM / 32;                // 16-byte loads per thread of an A slice

// chunk swizzle of row k in an MNC tile of 128 or 64 columns
template <int W>
DEV int mnc_swz(int k) {
  return W == 256 ? bf::mnc_swz(k) : W == 128 ? (k & 3) << 2 : ((k >> 1) & 1) << 2;
}
DEV int mnc128_off(int k, int mn) { return k * 128 + (((mn >> 3) ^ ((k & 3) << 2)) << 3) + (mn & 7); }

// Fragment read addresses of one operand.  Per lane, the LDS byte addresses
// of the reads that differ by more than a constant, in the even ring slots;
// every read is one of them plus a constant that fits the instruction's
// 16-bit offset (slot parity, k half, block), so the loop, unrolled over the slots,
// spends no instruction on addresses.  The sets past the first go through
// an asm add so that they stay in registers.
//  KC   the two k halves (the swizzle is the same for rows 32 apart)
//  MNC  rows k and k + 4 of each 32-column block
//  GLU  rows k and k + 4 of the two blocks of a matrix; wu 8 KiB past wg
template <int L, int NBLK, int NS>
struct FragAddr {
  static constexpr int N = L == KC ? 2 : L == MNC ? 2 * NBLK : 4;
  uint32_t at[NS / 2][N];
  template <int W>
  DEV static uint32_t mnc_at(int col, int lane, int hi) {
    const int g = lane >> 4, i = lane & 15;
    const int k = 8 * (g >> 1) + (i >> 2) + 4 * hi, mn = col + 16 * (g & 1) + 4 * (i & 3);
    return 2u * (uint32_t)(W == 256 ? bf::mnc_off(k, mn) : mnc128_off(k, mn));
  }
  // base: byte address of the operand in slot 0; first: first row or column of
  // the wave's blocks; W: columns of an MNC tile
  template <int W>
  DEV void init(uint32_t base, int first, int lane, uint32_t two_slots) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if constexpr (L == KC)
        at[0][j] = base + 2u * (uint32_t)bf::kc_off(first + (lane & 31), 2 * j + (lane >> 5));
      else
        at[0][j] = base + mnc_at<W>(first + 32 * (j >> 1), lane, j & 1);
#pragma unroll
      for (int p = 1; p < NS / 2; ++p) asm("v_add_u32 %0, %2, %1" : "=v"(at[p][j]) : "v"(at[p - 1][j]), "s"(two_slots));
    }
  }
  // block b, k half kk, in slot sl (constants); slot: bytes of a slot
  template <int W, int SLOT_BYTES>
  DEV bf16x8_t read(int b, int kk, int sl) const {
    const uint32_t* set = at[sl >> 1];
    const uint32_t so = (uint32_t)(sl & 1) * SLOT_BYTES;
    if constexpr (L == KC) {
      const LDS_AS char* p = (const LDS_AS char*)(uintptr_t)set[kk];
      return __builtin_bit_cast(bf16x8_t, *(const LDS_AS u32x4_t*)(p + so + (uint32_t)b * 2048u));
    } else {
      const int j = L == GLU ? 2 * (b & 1) : 2 * b;
      const uint32_t off = so + (uint32_t)kk * (16u * W * 2u) + (L == GLU ? (uint32_t)(b >> 1) * 8192u : 0u);
      const LDS_AS char* plo = (const LDS_AS char*)(uintptr_t)set[j];
      const LDS_AS char* phi = (const LDS_AS char*)(uintptr_t)set[j + 1];
      bf::v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS bf::v4i16*)(plo + off));
      bf::v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS bf::v4i16*)(phi + off));
      const u32x2_t l2 = __builtin_bit_cast(u32x2_t, lo), h2 = __builtin_bit_cast(u32x2_t, hi);
      return __builtin_bit_cast(bf16x8_t, u32x4_t{l2[0], l2[1], h2[0], h2[1]});
    }
  }
};

// ------------------------------------------------------------------ loaders
// K-contiguous operand of ROWS tile rows (rows of `cols` readable elements):
// wave-load j fills LDS rows 16 j .. 16 j + 15.
template <int NL>
struct KcOp {
  bf::i32x4_t rs;
  uint32_t voff[NL];
  DEV void init(const void* base, int64_t extent, int wave, int lane, int valid, int64_t ld) {
    rs = bf::make_rsrc(base, (uint32_t)extent);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int r = 16 * (wave * NL + i) + (lane >> 2);
      const int c = (lane & 3) ^ bf::kc_swz(r);
      voff[i] = r < valid ? (uint32_t)(r * ld * 2) + (uint32_t)c * 16u : kOOB;
    }
  }
  // 16-byte chunk of a slice that this lane loads (the same in every load)
  DEV static int chunk(int lane) { return (lane & 3) ^ ((lane >> 4) & 3); }
  DEV void issue(uint32_t lds, int wave, int i, bool ok, uint32_t soff) const {
    bf::dma16(rs, lds + (uint32_t)(wave * NL + i) * 1024u, ok ? voff[i] : kOOB, soff);
  }
};

// M/N-contiguous operand of W columns: wave-load j fills 1 KiB of LDS rows.
// Rows past the operand lie past its extent and read zeros.
template <int W, int NL>
struct MncOp {
  bf::i32x4_t rs;
  uint32_t voff[NL];   // row offset in slice 0 plus column offset, or kOOB for columns past `valid`
  DEV void init(const void* base, int64_t extent, int wave, int lane, int valid, int64_t ld) {
    init(base, extent, wave, lane, 0, valid, ld);
  }
  // the W columns from column c0 of the tile
  DEV void init(const void* base, int64_t extent, int wave, int lane, int c0, int valid, int64_t ld) {
    rs = bf::make_rsrc(base, (uint32_t)extent);
    constexpr int LPR = W / 8;          // lanes per k row
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int k = (64 / LPR) * (wave * NL + i) + lane / LPR;
      const int c = (lane & (LPR - 1)) ^ mnc_swz<W>(k);
      voff[i] = c0 + 8 * c < valid ? (uint32_t)(k * ld * 2) + (uint32_t)(c0 * 2 + c * 16) : kOOB;
    }
  }
  DEV void issue(uint32_t lds, int wave, int i, uint32_t slice_off) const {
    bf::dma16(rs, lds + (uint32_t)(wave * NL + i) * 1024u, voff[i] + slice_off, 0u);
  }
};

// ----------------------------------------------------------------- main loop
template <int N>
DEV void wait_vm_barrier() {
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <int AL, int BL, int WTM>
struct TileAddr {
  static constexpr int WB = BL == GLU ? 128 : 256, SB = kSlot<WTM> * 2;
  FragAddr<AL, WTM / 32, kSlots<WTM>> a;
  FragAddr<BL, 4, kSlots<WTM>> b;
  DEV void init(uint32_t ring, int wm, int wn, int lane) {
    a.template init<2 * WTM>(ring, wm * WTM, lane, 2u * SB);
    b.template init<WB>(ring + kAOper<WTM> * 2, wn * (BL == GLU ? 64 : 128), lane, 2u * SB);
  }
  // the fragment that group g of the phase reads (bf::kGrpA, kGrpB)
  DEV void load(bf::Frags& f, int kk, int sl, int g) const {
    if (bf::kGrpA[g] >= 0) {
      if (bf::kGrpA[g] < WTM / 32) f.a[bf::kGrpA[g]] = a.template read<2 * WTM, SB>(bf::kGrpA[g], kk, sl);
    } else {
      f.b[bf::kGrpB[g]] = b.template read<WB, SB>(bf::kGrpB[g], kk, sl);
    }
  }
};

// One of the two products of group g (bf::mma2).
template <int NMB, bool FIRST = false>
DEV void mma1(const bf::Frags& f, f32x16_t (&acc)[4][4], int g, int j) {
  const int mb = bf::kGrpM[g], nb = bf::kGrpN[g] + j;
  if (mb >= NMB) return;
  const f32x16_t zero = {};
  acc[mb][nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.b[nb], f.a[mb], FIRST ? zero : acc[mb][nb], 0, 0, 0);
}

// nsteps >= 1 slices.  issue(s, slot, i): load i of slice s into the slot at
// that LDS address, i < kALoads of A, then 4 of B; slices at or past nsteps
// must read zeros (their loads keep the count of outstanding loads the same
// in every step).  The order of waits and reads is bf::mainloop's: in step s the
// B loads of slice s + NS - 2 go out while k-half 0 is multiplied; then slice
// s + 1 has landed, and the A loads of slice s + NS - 1 go out while k-half 1 is.
template <int AL, int BL, int WTM, class Issue>
DEV void mainloop(uint32_t ring, int nsteps, Issue issue, f32x16_t (&acc)[4][4], int wm, int wn, int lane) {
  constexpr int LA = kALoads<WTM>, L = LA + 4, NMB = WTM / 32, SB = kSlot<WTM> * 2, NS = kSlots<WTM>;
  auto addr = [&](int sl) { return ring + (uint32_t)sl * SB; };
#pragma unroll
  for (int s = 0; s < NS - 2; ++s)
#pragma unroll
    for (int i = 0; i < L; ++i) issue(s, addr(s), i);
#pragma unroll
  for (int i = 0; i < LA; ++i) issue(NS - 2, addr(NS - 2), i);
  TileAddr<AL, BL, WTM> ta;
  ta.init(ring, wm, wn, lane);
  wait_vm_barrier<L*(NS - 3) + LA>();  // slice 0 landed
  bf::Frags f0, f1;
#pragma unroll
  for (int g = 0; g < 8; ++g) ta.load(f0, 0, 0, g);
  // step s in slot sl = s % NS
  auto phase1 = [&](int s, auto first, int sl) __attribute__((always_inline)) {
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      ta.load(f1, 1, sl, g);
      __builtin_amdgcn_sched_barrier(0);
      mma1<NMB, decltype(first)::value>(f0, acc, g, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (g & 1) issue(s + NS - 2, addr((sl + NS - 2) % NS), LA + (g >> 1));
      __builtin_amdgcn_sched_barrier(0);
      mma1<NMB, decltype(first)::value>(f0, acc, g, 1);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto phase2 = [&](int s, int sl) __attribute__((always_inline)) {
    wait_vm_barrier<L*(NS - 3)>();  // slice s+1 landed; slot of slice s-1 free
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      ta.load(f0, 0, (sl + 1) % NS, g);
      __builtin_amdgcn_sched_barrier(0);
      mma1<NMB>(f1, acc, g, 0);
      __builtin_amdgcn_sched_barrier(0);
      if ((g & 1) && (g >> 1) < LA) issue(s + NS - 1, addr((sl + NS - 1) % NS), g >> 1);
      __builtin_amdgcn_sched_barrier(0);
      mma1<NMB>(f1, acc, g, 1);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // past the last slice the next slot holds zeros, read and never multiplied
  phase1(0, bf::BoolC<true>{}, 0);
  phase2(0, 0);
  int s = 1;
#pragma unroll 1
  for (; s + NS <= nsteps; s += NS) {
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      phase1(s + j, bf::BoolC<false>{}, (1 + j) % NS);
      phase2(s + j, (1 + j) % NS);
    }
  }
#pragma unroll
  for (int j = 0; j < NS - 1; ++j) {
    if (s + j < nsteps) {
      phase1(s + j, bf::BoolC<false>{}, (1 + j) % NS);
      phase2(s + j, (1 + j) % NS);
    }
  }
  bf::block_barrier();
}

// ----------------------------------------------------------------- small tiles
// Tile (64 MB) x (64 NB) (the gated product: 64 columns of both matrices, NB =
// 2), K slice 64 as two halves of 32 in the layouts above, 4 waves in a 2x2 grid
// that hold one 32 x 32 block of each 64 x 64 part.  For products with too few
// tiles of 128 x 256 to fill the device: more workgroups, a short first slice and a
// short epilogue, paid for with more reads of the caches, which bound them
// (2048^3 with 128 x 128: 24 us, 720 TF, 0.3 GB through the L2s, 13 TB/s; 512^3 with 64 x 64: 5.9 us,
// of it 4.5 us launch, first slice and epilogue).
// One barrier a slice: the reads of the slot that is filled next were waited for
// before it.  More slots are no faster (1024^3: 8.2 us with 4, 8.4 with 5, 8.6 with
// 6), products between the reads one at a time are (128 x 128, 2048^3:
// 24.7 -> 23.0 us).
constexpr int SBK = 64;
template <int MB, int NB, bool SHORT>
struct Small {
  static constexpr int PARTS = MB + NB;
  // Ring slots.  SHORT: contractions of at most two slices a workgroup, where
  // five workgroups a CU (three of the gated product) hide each other's first loads
  // and stores (backward of 2048 x 8192 with 33 rows, of it the weight gradient two
  // thirds: 36.6 -> 27.8 us, 25.8 with non-temporal stores)
  static constexpr int NS = SHORT ? 2 : MB == 1 && NB == 2 ? 3 : 4;
  // Fragments are read one slice ahead of their products (512 x 2048 x 2048 with
  // 64 x 64: 12.1 -> 11.1 us), but not where that needs a fourth slot and
  // leaves room for one workgroup a CU (gated, 1024 x 2048 x 8192: 85 and 106 us)
  static constexpr bool AHEAD = NS == 4;
  static constexpr uint32_t HALF = 4096 * PARTS, SLOT = 2 * HALF;
  static constexpr int RING = NS * SLOT;                     // 64, 72 or 128 KiB; SHORT 32 or 48
};

// One operand's fragment addresses in the first slot's first half.
template <int L>
struct SmallAddr {
  uint32_t at[2];
  DEV void init(uint32_t base, int first, int lane) {
    if constexpr (L == KC) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) at[kk] = base + 2u * (uint32_t)bf::kc_off(first + (lane & 31), 2 * kk + (lane >> 5));
    } else {
      const int g = lane >> 4, i = lane & 15, k = 8 * (g >> 1) + (i >> 2), mn = first + 16 * (g & 1) + 4 * (i & 3);
      at[0] = base + 2u * (uint32_t)(k * 64 + (((mn >> 3) ^ mnc_swz<64>(k)) << 3) + (mn & 7));
    }
  }
  // k quarter kk of the half at byte offset off
  DEV bf16x8_t read(uint32_t off, int kk) const {
    if constexpr (L == KC) {
      return __builtin_bit_cast(bf16x8_t, *(const LDS_AS u32x4_t*)((const LDS_AS char*)(uintptr_t)(at[kk] + off)));
    } else {
      const LDS_AS char* p = (const LDS_AS char*)(uintptr_t)(at[0] + off) + kk * 2048;
      bf::v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS bf::v4i16*)p);
      bf::v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS bf::v4i16*)(p + 512));
      const u32x2_t l2 = __builtin_bit_cast(u32x2_t, lo), h2 = __builtin_bit_cast(u32x2_t, hi);
      return __builtin_bit_cast(bf16x8_t, u32x4_t{l2[0], l2[1], h2[0], h2[1]});
    }
  }
};

// K-contiguous operand in parts of 64 tile rows, of each of which a wave loads 16.
template <int NP>
struct KcPart {
  bf::i32x4_t rs;
  uint32_t voff[NP];
  DEV void init(const void* base, int64_t extent, int wave, int lane, int valid, int64_t ld) {
    rs = bf::make_rsrc(base, (uint32_t)extent);
    const int r = 16 * wave + (lane >> 2), c = (lane & 3) ^ bf::kc_swz(r);
#pragma unroll
    for (int p = 0; p < NP; ++p)
      voff[p] = 64 * p + r < valid ? (uint32_t)((64 * p + r) * ld * 2) + (uint32_t)c * 16u : kOOB;
  }
};

// issue(h, addr, i): load i (the parts of A, then those of B) of half slice h to
// addr; half slices past 2 nsteps may hold anything.
template <int AL, int BL, int MB, int NB, bool SHORT, class Issue>
DEV void small_mainloop(uint32_t ring, int nsteps, Issue issue, f32x16_t (&acc)[MB][NB], int wm, int wn, int lane) {
  using S = Small<MB, NB, SHORT>;
  constexpr uint32_t HALF = S::HALF, SB = S::SLOT, END = S::NS * SB;
  constexpr int L = 2 * S::PARTS, NS = S::NS;
  auto fill = [&](int s, uint32_t off) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < S::PARTS; ++i) issue(2 * s + h, ring + off + h * HALF + i * 4096, i);
  };
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) fill(s, s * SB);
  SmallAddr<AL> aa;
  SmallAddr<BL> ba;
  aa.init(ring, wm * 32, lane);
  ba.init(ring + 4096 * MB, wn * 32, lane);
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[m][n][r] = 0.f;
  struct Frag {
    bf16x8_t a[4][MB], b[4][NB];
  } f0, f1;
  // fragment k of a slice, in the order of their use
  constexpr int NR = 4 * S::PARTS, NM = 4 * MB * NB;
  auto read = [&](Frag& f, uint32_t off, int k) __attribute__((always_inline)) {
    const int q = k / S::PARTS, i = k % S::PARTS;
    const uint32_t o = off + (q >> 1) * HALF;
    if (i < MB)
      f.a[q][i < MB ? i : 0] = aa.read(o + i * 4096, q & 1);
    else
      f.b[q][i < MB ? 0 : i - MB] = ba.read(o + (i - MB) * 4096, q & 1);
  };
  uint32_t at = S::AHEAD ? SB : 0, free = (NS - 1) * SB;   // slot that is read, slot that is filled
  auto step = [&](int s, Frag& f, Frag& g) __attribute__((always_inline)) {
    // the slice that is read landed in every wave's part, and slot `free` was read
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NS - 2 - S::AHEAD) * L) : "memory");
    if constexpr (!S::AHEAD) {
#pragma unroll
      for (int k = 0; k < NR; ++k) read(f, at, k);
      fill(s + NS - 1, free);
    }
    // one product at a time between the reads and loads of later slices
#pragma unroll
    for (int j = 0; j < NM; ++j) {
      const int q = j / (MB * NB), m = j / NB % MB, n = j % NB;
      acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.b[q][n], f.a[q][m], acc[m][n], 0, 0, 0);
      if constexpr (S::AHEAD) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = j * NR / NM; k < (j + 1) * NR / NM; ++k) read(g, at, k);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = j * L / NM; k < (j + 1) * L / NM; ++k)
          issue(2 * (s + NS - 1) + k / S::PARTS, ring + free + k / S::PARTS * HALF + k % S::PARTS * 4096, k % S::PARTS);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    at = at + SB == END ? 0 : at + SB;
    free = free + SB == END ? 0 : free + SB;
  };
  if constexpr (S::AHEAD) {
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((NS - 2) * L) : "memory");
#pragma unroll
    for (int k = 0; k < NR; ++k) read(f0, 0, k);
  }
  int s = 0;
#pragma unroll 1
  for (; s + 2 <= nsteps; s += 2) {
    step(s, f0, f1);
    step(s + 1, f1, f0);
  }
  if (s < nsteps) step(s, f0, f1);
  bf::block_barrier();
}

}  // namespace dn
}  // namespace moedet
