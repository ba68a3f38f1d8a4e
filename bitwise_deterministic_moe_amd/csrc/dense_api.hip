// Host side of the dense operators' C ABI (declared in include/moedet.h):
// argument checks, workspace layout, and the choice of kernel and split from
// sizes alone.
#include <cstdarg>
#include <cstdio>

#include "../../include/moedet.h"
#include "dense.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moedet {
namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// ------------------------------------------------------------------ description
constexpr int64_t kMaxLd = (int64_t)1 << 20;

struct Dense {
  bool bf16;
  int nm;             // weight matrices: 1 linear, 2 gated
  int64_t T;
  int D, F;
  int64_t es;
  int act;
  int any;            // moe_any bits
};
constexpr int kAnyBits = MOE_ANY_X | MOE_ANY_W | MOE_ANY_Y | MOE_ANY_REST;

moe_status check(const moe_dense* p, int nm, Dense* d) {
  if (!p) return MOE_ERR_NULL;
  if (p->dtype != MOE_F32 && p->dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (p->grad_dtype != MOE_F32 && p->grad_dtype != p->dtype) return MOE_ERR_DTYPE;
  if (p->z_dtype != MOE_F32 && p->z_dtype != p->dtype) return MOE_ERR_DTYPE;
  d->any = p->act & kAnyBits;
  d->act = p->act - d->any;
  if (d->act < MOE_ACT_NONE || d->act > MOE_ACT_GELU) return MOE_ERR_MODE;
  if (p->rows < 0 || p->rows >= (int64_t)1 << 31 || p->d_in < 1 || p->d_out < 1) return MOE_ERR_SHAPE;
  if (p->d_in >= kMaxLd || p->d_out >= kMaxLd) return MOE_ERR_SHAPE;
  if (p->ldx < p->d_in || p->ldw < p->d_out || p->ldy < p->d_out || p->ldz < p->d_out) return MOE_ERR_SHAPE;
  if (p->ldx >= kMaxLd || p->ldw >= kMaxLd || p->ldy >= kMaxLd || p->ldz >= kMaxLd || p->ldr < 0 || p->ldr >= kMaxLd)
    return MOE_ERR_SHAPE;
  d->bf16 = p->dtype == MOE_BF16;
  d->es = d->bf16 ? 2 : 4;
  // a copied weight matrix has rows of d_out rounded up to 8, no longer than ldw + 7
  if ((int64_t)p->d_in * up(p->ldw, 8) * d->es >= (int64_t)1 << 31) return MOE_ERR_SHAPE;
  d->nm = nm;
  d->T = p->rows;
  d->D = p->d_in;
  d->F = p->d_out;
  return MOE_OK;
}

// Whether a base address is a multiple of 16 bytes, or of `es` where the call allows it.
bool based(const Dense& d, const void* p, int any, int64_t es) {
  return ((uintptr_t)p & (uintptr_t)(d.any & any ? es - 1 : 15)) == 0;
}

// A bf16 matrix that the tile kernels read in place: whole 16-byte chunks.
bool direct(const Dense& d, int64_t cols, int64_t ld, int any) {
  return !d.bf16 || (cols % 8 == 0 && ld % 8 == 0 && !(d.any & any));
}
bool direct_x(const Dense& d, const moe_dense* p) { return direct(d, d.D, p->ldx, MOE_ANY_X); }
bool direct_w(const Dense& d, const moe_dense* p) { return direct(d, d.F, p->ldw, MOE_ANY_W); }

// --------------------------------------------------------- tile and split choice
struct Choice {
  int tile, S;
};
constexpr int kCUs = 256;
constexpr int64_t kMaxPartialBytes = (int64_t)1 << 30;
constexpr int64_t kMaxUnits = ((int64_t)1 << 24) - 8;   // workgroups of 256 in a launch

// A tile's cost in microseconds, measured on this card, by dense_shape's
// numbers.  `fixed`: launch, first slice, epilogue.  Per K slice and workgroup:
// `alone` while at most half of the CUs have one, `busy` when all do (they share the
// caches' bandwidth); where several workgroups fit on a CU (`shares`), `alone`
// for one and `busy` for each of several.
//   bf16     256 x 256: 0.77 (8192^3) to 0.85; 128 x 256: 0.48 (4096 x 8192 x 2048),
//            0.36 on half the CUs; 128 x 128 (slices of 64): 0.54 (2048^3), 0.38;
//            64 x 64 (of 64): 0.2 alone, 0.23 each of two, 1.6 of it for both
//            matrices of the gated product.
//            512^3 takes 5.9 us with the 64 x 64 tile, 9 with 128 x 128 and 13.6
//            with 128 x 256; 2048^3 35, 24 and 31; 4096 x 2048 x 8192 240,
//            167 and 125 (with 256 x 256)
//   float32  128 x 128 in three parts: 1.54 (4096^3); 64 x 64 (slices of 16): 0.27 of
//            several.  They meet near 1024^3: 50 us and 27 us forward, at 2048^3
//            107 us and 147 us
struct TileCost {
  double alone, busy, fixed;
  bool shares;
};
constexpr TileCost kBf16Tiles[] = {{0.7, 0.8, 9.0, false}, {0.36, 0.48, 8.0, false}, {0.38, 0.52, 5.8, false}, {0.2, 0.23, 4.5, true}};
constexpr TileCost kF32Tiles[] = {{1.5, 1.5, 9.0, false}, {0.38, 0.27, 6.0, true}};

double estimate(const TileCost& c, int64_t wgs, int64_t steps, double width, int64_t S, double out_elems) {
  const double per_cu = (double)((wgs + kCUs - 1) / kCUs);
  double slice, t = c.fixed;
  if (c.shares) {
    slice = per_cu * c.busy > c.alone ? per_cu * c.busy : c.alone;
  } else {
    const double over = 2.0 * (double)wgs / kCUs - 1;
    slice = per_cu * (over <= 0 ? c.alone : over >= 1 ? c.busy : c.alone + over * (c.busy - c.alone));
    // later rounds pay their epilogue again
    t += (per_cu - 1) * 0.6 * c.fixed;
  }
  t += (double)steps * width * slice;
  // float32 partials written and read, mostly in the caches, and the launch that
  // joins them
  if (S > 1) t += (double)S * out_elems * 8.0 / 1e7 + 3.0;
  return t;
}

// Whether one launch copies x into rows of ld elements, beside the weights and the
// elementwise pass (together at most 2^22 workgroups).
bool copies_fit(const Dense& d, int64_t ld) { return d.T * (ld / 8) / 256 < kMaxUnits - (1 << 22); }

// Tile and number of K chunks of one product: the cheapest estimate.  S = 0 if
// no tile covers it in one launch.
Choice choose(const Dense& d, int form, int64_t M, int64_t N, int nseg, int64_t K, int64_t ld_max) {
  const double outs = (double)M * N * (form == kFormDw ? nseg : form == kFormGlu ? 2 : 1);
  // the weight gradient's bf16 operands are addressed by 32-bit offsets from
  // the chunk's first row
  int64_t smin = 1;
  if (form == kFormDw && d.bf16) smin = (K + 64) * ld_max * 2 / ((int64_t)1 << 30) + 1;
  Choice best{0, 0};
  double tb = 0;
  for (int i = 0; i < (d.bf16 ? kDenseBf16Tiles : kDenseF32Tiles); ++i) {
    const TileCost& c = d.bf16 ? kBf16Tiles[i] : kF32Tiles[i];
    const DenseShape sh = dense_shape(form, d.bf16, i);
    const int64_t steps = (K + sh.bk - 1) / sh.bk * (form == kFormDx ? nseg : 1);
    // the 64-row tile of the gated product is twice as wide as high
    const double width = form == kFormGlu && sh.bm == 64 ? (d.bf16 ? 1.6 : 2) : 1;
    const int64_t tiles = (M + sh.bm - 1) / sh.bm * ((N + sh.bn - 1) / sh.bn * (form == kFormDw ? nseg : 1));
    const int64_t smax = smin > 32 ? smin : 32;
    for (int64_t S = smin; S <= smax; ++S) {
      if (S > smin && (steps / S < 4 || S * outs * 4 > kMaxPartialBytes || tiles * (S - 1) >= 4 * kCUs)) break;
      if (tiles * S > kMaxUnits) break;
      const double t = estimate(c, tiles * S, (steps + S - 1) / S, width, S, outs);
      if (best.S == 0 || t < tb * 0.98) {
        best = Choice{i, (int)S};
        tb = t;
      }
    }
  }
  return best;
}

// Chunks of K of the few-row kernels.  A workgroup streams about 40 KB/us and
// the device 4.6 TB/s; a launch of them takes 3 us beside the stream, and
// partials with their join 4.5 us more (measured: 64 strips of 8192 x 2048
// bf16 16.6 us unsplit; 256 in four chunks 10.5 us with the join).  Two row blocks of
// float32 products halve a workgroup's rate (4096 x 1024, 32 rows: 20.9 us unsplit,
// 12.2 us in chunks).
int few_chunks(const Dense& d) {
  const double strip = (double)d.D * 64 * d.nm;
  const int cols = 64 / (int)d.es;
  const int64_t tiles = (d.F + cols - 1) / cols, steps = (d.D + 31) / 32;
  const double all = (double)d.D * d.F * d.es * d.nm / 4.6e6;
  int64_t S = kCUs / tiles;
  if (S > steps / 16) S = steps / 16;
  if (S < 2) return 1;
  const double rate = !d.bf16 && d.T > 16 ? 20e3 : 40e3;
  const double t1 = strip / rate > all ? strip / rate : all;
  const double tS = 4.5 + (strip / S / rate > all ? strip / S / rate : all);
  return tS < t1 ? (int)S : 1;
}
bool few(const Dense& d, const moe_dense* p) {
  return d.T <= few_rows(d.bf16, d.nm, !direct_w(d, p));
}

// ------------------------------------------------------------- workspace layout
struct FwdPlan {
  bool few, pack_x, pack_w;
  Choice ch;
  int64_t ldx, ldw;          // row distances that the kernel reads
  int64_t part_seg, part_ld;
  size_t x, w, part, total;  // byte offsets
};

FwdPlan fwd_plan(const moe_dense* p, const Dense& d) {
  FwdPlan f{};
  const int form = d.nm == 2 ? kFormGlu : kFormLinear;
  f.few = few(d, p);
  f.ldx = p->ldx;
  f.ldw = p->ldw;
  size_t o = 0;
  if (d.T == 0) return f;
  if (f.few) {
    f.pack_x = d.bf16 && d.T >= kFewCopyRows && (p->ldx % 8 || (d.any & MOE_ANY_X));
    f.ch = Choice{0, few_chunks(d)};
  } else {
    f.pack_x = !direct_x(d, p);
    f.pack_w = !direct_w(d, p);
    f.ch = choose(d, form, d.T, d.F, 1, d.D, 0);
  }
  if (f.pack_x) {
    f.ldx = up(d.D, 8);
    if (!copies_fit(d, f.ldx)) f.ch.S = 0;
    f.x = o;
    o += align_up((size_t)d.T * f.ldx * 2);
  }
  if (f.pack_w) {
    f.ldw = up(d.F, 8);
    f.w = o;
    o += align_up((size_t)d.nm * d.D * f.ldw * 2);
  }
  f.part_seg = up(d.F, 4);
  f.part_ld = d.nm * f.part_seg;
  f.part = o;
  if (f.ch.S > 1) o += align_up((size_t)f.ch.S * d.T * f.part_ld * 4);
  f.total = o;
  return f;
}

struct BwdPlan {
  bool pack_x, pack_w, make_dz;
  Choice dx, dw;
  int64_t ldx, ldw, lddz, segdz;
  int64_t dx_ld, dw_seg;
  int ew_blocks;
  size_t x, w, dz, colsum, part_dx, part_dw, total;
};

BwdPlan bwd_plan(const moe_dense* p, const Dense& d) {
  BwdPlan b{};
  b.ldx = p->ldx;
  b.ldw = p->ldw;
  b.lddz = p->ldy;
  size_t o = 0;
  if (d.T == 0) return b;
  b.pack_x = !direct_x(d, p);
  b.pack_w = !direct_w(d, p);
  b.make_dz = d.nm == 2 || d.act != MOE_ACT_NONE || !direct(d, d.F, p->ldy, MOE_ANY_Y);
  if (b.pack_x) {
    b.ldx = up(d.D, 8);
    b.x = o;
    o += align_up((size_t)d.T * b.ldx * 2);
  }
  if (b.pack_w) {
    b.ldw = up(d.F, 8);
    b.w = o;
    o += align_up((size_t)d.nm * d.D * b.ldw * 2);
  }
  if (b.make_dz) {
    b.segdz = up(d.F, 32);
    b.lddz = d.nm * b.segdz;
    b.dz = o;
    o += align_up((size_t)d.T * b.lddz * d.es);
  }
  b.ew_blocks = dense_ew_blocks(d.T, d.F, d.bf16, d.nm == 1);
  b.colsum = o;
  if (d.nm == 1) o += align_up((size_t)b.ew_blocks * d.F * 4);
  b.dx = choose(d, kFormDx, d.T, d.D, d.nm, d.F, 0);
  b.dw = choose(d, kFormDw, d.D, d.F, d.nm, d.T, b.ldx > b.lddz ? b.ldx : b.lddz);
  if (b.pack_x && !copies_fit(d, b.ldx)) b.dx.S = 0;
  b.dx_ld = up(d.D, 4);
  b.dw_seg = up(d.F, 4);
  // both products' partials live until the joining launch at the end
  b.part_dx = o;
  if (b.dx.S > 1) o += align_up((size_t)b.dx.S * d.T * b.dx_ld * 4);
  b.part_dw = o;
  if (b.dw.S > 1) o += align_up((size_t)b.dw.S * d.D * d.nm * b.dw_seg * 4);
  b.total = o;
  return b;
}

moe_status workspace_size(const moe_dense* p, int nm, size_t* fwd, size_t* bwd) {
  Dense d;
  const moe_status s = check(p, nm, &d);
  if (s != MOE_OK) return s;
  if (fwd) *fwd = fwd_plan(p, d).total;
  if (bwd) *bwd = bwd_plan(p, d).total;
  return MOE_OK;
}

// ------------------------------------------------------------------ kernel names
struct Names {
  char* at;
  size_t left;
  bool fits = true;
  void add(const char* format, ...) {
    va_list v;
    va_start(v, format);
    const int n = vsnprintf(at, left, format, v);
    va_end(v);
    fits = fits && n >= 0 && (size_t)n < left;
    if (fits) {
      at += n;
      left -= n;
    }
  }
};

void add_product(Names& o, const char* name, const Dense& d, int form, const Choice& c, int64_t M, int64_t N, int nseg, int64_t K) {
  DenseParams P{};
  P.M = M;
  P.N = (int)N;
  P.K = K;
  P.nseg = nseg;
  P.S = c.S;
  static const char* const kBf16[kDenseBf16Tiles] = {"256x256", "128x256", "128x128", "64x64"};
  static const char* const kF32[kDenseF32Tiles] = {"128x128_parts", "64x64_f32"};
  o.add("%s_%s", name, d.bf16 ? kBf16[c.tile] : kF32[c.tile]);
  if (d.bf16 && c.tile == kDenseBf16Tiles - 1 && dense_short(P, form)) o.add("_short");
  if (!d.bf16 && !dense_v4(P, form)) o.add("_odd");
  if (c.S > 1) o.add("_split%d", c.S);
}

moe_status stage_names(const moe_dense* p, int nm, int call, char* names, size_t bytes) {
  Dense d;
  const moe_status s = check(p, nm, &d);
  if (s != MOE_OK) return s;
  if (call < 0 || call > 2) return MOE_ERR_MODE;
  if (!names) return MOE_ERR_NULL;
  if (bytes < 1) return MOE_ERR_WORKSPACE;
  Names o{names, bytes};
  o.add("");
  const bool db = nm == 1 && call == 1;
  if (d.T == 0) {
    if (call) o.add(nm == 2 ? "zero,zero" : db ? "zero,zero" : "zero");
  } else if (call == 0) {
    const FwdPlan f = fwd_plan(p, d);
    if (!f.ch.S) return MOE_ERR_SHAPE;
    const int form = nm == 2 ? kFormGlu : kFormLinear;
    const char* name = nm == 2 ? "glu" : "linear";
    if (f.pack_x || f.pack_w) o.add("copy,");
    if (f.few) {
      o.add("%s_few%d", name, (int)up(d.T, 16));
      if (f.ch.S > 1) o.add("_split%d", f.ch.S);
    } else {
      add_product(o, name, d, form, f.ch, d.T, d.F, 1, d.D);
    }
    if (f.ch.S > 1) o.add(",join");
  } else {
    const BwdPlan b = bwd_plan(p, d);
    if (!b.dx.S || !b.dw.S) return MOE_ERR_SHAPE;
    const bool copies = b.pack_x || b.pack_w;
    if (b.make_dz || db)
      o.add(!copies ? "%s," : "%s_copy,", b.make_dz ? "dz" : "sums");
    else if (copies)
      o.add("copy,");
    add_product(o, "dx", d, kFormDx, b.dx, d.T, d.D, nm, d.F);
    o.add(",");
    add_product(o, "dw", d, kFormDw, b.dw, d.D, d.F, nm, d.T);
    if (b.dx.S > 1 || b.dw.S > 1 || db) o.add(",join");
  }
  return o.fits ? MOE_OK : MOE_ERR_WORKSPACE;
}

moe_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return MOE_OK;
  if (!ws) return MOE_ERR_NULL;
  if (have < need || ((uintptr_t)ws & (kAlign - 1))) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

#define MOE_TRY(x)                               \
  do {                                           \
    if ((x) != hipSuccess) return MOE_ERR_HIP;   \
  } while (0)

// The copies of x and the weights into whole 16-byte rows, where they need
// one; x and w then point to them.
DensePackParams plan_copies(const Dense& d, const moe_dense* p, bool px, bool pw, int64_t ldx, int64_t ldw, char* wx,
                            char* ww, const void*& x, const void* (&w)[2]) {
  DensePackParams K{};
  if (px) {
    K.add(x, d.T, d.D, p->ldx, wx, ldx);
    x = wx;
  }
  if (pw) {
    for (int m = 0; m < d.nm; ++m) {
      char* o = ww + (size_t)m * d.D * ldw * 2;
      K.add(w[m], d.D, d.F, p->ldw, o, ldw);
      w[m] = o;
    }
  }
  return K;
}

moe_status forward(const moe_dense* p, int nm, const void* x, const void* w0, const void* w1, const void* bias,
                   const void* residual, void* y, void* z0, void* z1, void* ws, size_t ws_bytes, hipStream_t st) {
  Dense d;
  moe_status s = check(p, nm, &d);
  if (s != MOE_OK) return s;
  if (residual && p->ldr < d.F) return MOE_ERR_SHAPE;
  if (nm == 2 && (z0 == nullptr) != (z1 == nullptr)) return MOE_ERR_NULL;
  if (d.T == 0) return MOE_OK;
  if (!x || !w0 || !w1 || !y) return MOE_ERR_NULL;
  const int64_t zs = p->z_dtype == MOE_F32 ? 4 : 2;
  if (!based(d, x, MOE_ANY_X, d.es) || !based(d, w0, MOE_ANY_W, d.es) || !based(d, w1, MOE_ANY_W, d.es) ||
      !based(d, y, MOE_ANY_Y, d.es) || !based(d, residual, MOE_ANY_REST, d.es) || !based(d, z0, MOE_ANY_REST, zs) ||
      !based(d, z1, MOE_ANY_REST, zs) || ((uintptr_t)bias & (d.es - 1)))
    return MOE_ERR_SHAPE;
  const FwdPlan f = fwd_plan(p, d);
  if (!f.ch.S) return MOE_ERR_SHAPE;
  if ((s = check_ws(ws, ws_bytes, f.total)) != MOE_OK) return s;
  const void* w[2] = {w0, w1};
  MOE_TRY(launch_dense_pack(
      plan_copies(d, p, f.pack_x, f.pack_w, f.ldx, f.ldw, (char*)ws + f.x, (char*)ws + f.w, x, w), st));
  const int form = nm == 2 ? kFormGlu : kFormLinear;
  DenseParams P{};
  P.M = d.T;
  P.N = d.F;
  P.K = d.D;
  P.nseg = 1;
  P.a = x;
  P.lda = f.ldx;
  P.b[0] = w[0];
  P.b[1] = w[1];
  P.ldb = f.ldw;
  P.S = f.ch.S;
  P.part = (float*)((char*)ws + f.part);
  P.part_ld = f.part_ld;
  P.part_seg = (int)f.part_seg;
  P.bias = bias;
  P.add = residual;
  P.ldadd = p->ldr;
  P.c[0] = y;
  P.ldc = p->ldy;
  P.z[0] = z0;
  P.z[1] = z1;
  P.ldz = p->ldz;
  P.z_f32 = p->z_dtype == MOE_F32;
  P.act = d.act;
  P.seed = p->debug_shuffle_seed;
  if (f.few)
    MOE_TRY(launch_dense_few(P, form, d.bf16, st));
  else
    MOE_TRY(launch_dense_gemm(P, form, d.bf16, f.ch.tile, st));
  if (P.S > 1) MOE_TRY(launch_dense_finish(P, form, d.bf16, st));
  return MOE_OK;
}

moe_status backward(const moe_dense* p, int nm, const void* dy, const void* x, const void* w0, const void* w1,
                    const void* z0, const void* z1, const void* dx_add, void* dx, void* dw0, void* dw1, void* db,
                    void* ws, size_t ws_bytes, hipStream_t st) {
  Dense d;
  moe_status s = check(p, nm, &d);
  if (s != MOE_OK) return s;
  if (dx_add && p->ldr < d.D) return MOE_ERR_SHAPE;
  const bool g32 = p->grad_dtype == MOE_F32;
  const int64_t gs = g32 ? 4 : 2;
  if (!dw0 || !dw1) return MOE_ERR_NULL;
  const bool need_z = nm == 2 || d.act != MOE_ACT_NONE;
  if (d.T > 0 && (!dy || !x || !w0 || !w1 || !dx || (need_z && (!z0 || !z1)))) return MOE_ERR_NULL;
  const int64_t zs = p->z_dtype == MOE_F32 ? 4 : 2;
  if (!based(d, dy, MOE_ANY_Y, d.es) || !based(d, x, MOE_ANY_X, d.es) || !based(d, w0, MOE_ANY_W, d.es) ||
      !based(d, w1, MOE_ANY_W, d.es) || !based(d, dx_add, MOE_ANY_REST, d.es) || !based(d, dx, MOE_ANY_REST, d.es) ||
      !based(d, dw0, MOE_ANY_REST, gs) || !based(d, dw1, MOE_ANY_REST, gs) || ((uintptr_t)db & (gs - 1)))
    return MOE_ERR_SHAPE;
  if (need_z && (!based(d, z0, MOE_ANY_REST, zs) || !based(d, z1, MOE_ANY_REST, zs))) return MOE_ERR_SHAPE;
  if (d.T == 0) {
    const int64_t n16 = (int64_t)d.D * d.F * gs / 2;
    MOE_TRY(launch_dense_zero(dw0, n16, st));
    if (nm == 2) MOE_TRY(launch_dense_zero(dw1, n16, st));
    if (db) MOE_TRY(launch_dense_zero(db, d.F * gs / 2, st));
    return MOE_OK;
  }
  const BwdPlan b = bwd_plan(p, d);
  if (!b.dx.S || !b.dw.S) return MOE_ERR_SHAPE;
  if ((s = check_ws(ws, ws_bytes, b.total)) != MOE_OK) return s;
  char* base = (char*)ws;
  const void* w[2] = {w0, w1};
  const DensePackParams K = plan_copies(d, p, b.pack_x, b.pack_w, b.ldx, b.ldw, base + b.x, base + b.w, x, w);
  const void* dz = dy;
  if (b.make_dz || db) {
    DenseEwParams E{};
    E.rows = d.T;
    E.cols = d.F;
    E.dy = dy;
    E.lddy = p->ldy;
    E.z[0] = z0;
    E.z[1] = z1;
    E.ldz = p->ldz;
    E.z_f32 = p->z_dtype == MOE_F32;
    E.act = d.act;
    if (b.make_dz) {
      E.out[0] = base + b.dz;
      E.out[1] = base + b.dz + b.segdz * d.es;
      dz = E.out[0];
    }
    E.ldo = b.lddz;
    E.pad = b.make_dz ? (int)b.segdz : d.F;
    E.part = db ? (float*)(base + b.colsum) : nullptr;
    E.blocks = b.ew_blocks;
    E.seed = p->debug_shuffle_seed;
    MOE_TRY(launch_dense_ew(E, K, nm == 2, d.bf16, st));
  } else {
    MOE_TRY(launch_dense_pack(K, st));
  }
  DenseParams P{};
  P.M = d.T;
  P.N = d.D;
  P.K = d.F;
  P.nseg = nm;
  P.a = dz;
  P.lda = b.lddz;
  P.seg = b.segdz;
  P.b[0] = w[0];
  P.b[1] = w[1];
  P.ldb = b.ldw;
  P.S = b.dx.S;
  P.part = (float*)(base + b.part_dx);
  P.part_ld = b.dx_ld;
  P.add = dx_add;
  P.ldadd = p->ldr;
  P.c[0] = dx;
  P.ldc = d.D;
  P.seed = p->debug_shuffle_seed;
  MOE_TRY(launch_dense_gemm(P, kFormDx, d.bf16, b.dx.tile, st));
  DenseParams W{};
  W.M = d.D;
  W.N = d.F;
  W.K = d.T;
  W.nseg = nm;
  W.a = x;
  W.lda = b.ldx;
  W.b[0] = dz;
  W.ldb = b.lddz;
  W.seg = b.segdz;
  W.S = b.dw.S;
  W.part = (float*)(base + b.part_dw);
  W.part_seg = (int)b.dw_seg;
  W.part_ld = nm * b.dw_seg;
  W.c[0] = dw0;
  W.c[1] = dw1;
  W.ldc = d.F;
  W.c_f32 = g32;
  W.seed = p->debug_shuffle_seed;
  MOE_TRY(launch_dense_gemm(W, kFormDw, d.bf16, b.dw.tile, st));
  return hip_status(launch_dense_join(P, W, (const float*)(base + b.colsum), b.ew_blocks, d.F, db, !g32 && d.bf16, d.bf16, st));
}

// --------------------------------------------------------------------- layer norm
moe_status check_norm(moe_dtype dtype, int64_t rows, int64_t cols) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (rows < 0 || cols < 1 || cols > kNormMaxCols || rows >= (int64_t)1 << 40) return MOE_ERR_SHAPE;
  return MOE_OK;
}
bool ld_ok(int64_t rows, int64_t cols, int64_t ld) { return ld >= cols && ld < ((int64_t)1 << 40) / (rows < 1 ? 1 : rows); }

}  // namespace
}  // namespace moedet

using namespace moedet;

MOE_API moe_status moe_layernorm_fwd(const void* x, const void* weight, const void* bias, moe_dtype dtype,
                                     int64_t rows, int64_t cols, int64_t ldx, float eps, void* y, float* mean,
                                     float* rstd, uint64_t debug_shuffle_seed, void* stream) {
  const moe_status s = check_norm(dtype, rows, cols);
  if (s != MOE_OK) return s;
  if (!ld_ok(rows, cols, ldx) || !(eps >= 0.f && eps < __builtin_inff())) return MOE_ERR_SHAPE;
  if ((mean == nullptr) != (rstd == nullptr)) return MOE_ERR_NULL;
  if (rows == 0) return MOE_OK;
  if (!x || !y) return MOE_ERR_NULL;
  const uintptr_t em = dtype == MOE_BF16 ? 1 : 3;
  if (((uintptr_t)x | (uintptr_t)weight | (uintptr_t)bias | (uintptr_t)y) & em) return MOE_ERR_SHAPE;
  if (((uintptr_t)mean | (uintptr_t)rstd) & 3) return MOE_ERR_SHAPE;
  NormParams P{};
  P.x = x;
  P.weight = weight;
  P.bias = bias;
  P.rows = rows;
  P.ldx = ldx;
  P.cols = (int)cols;
  P.eps = eps;
  P.y = y;
  P.mean = mean;
  P.rstd = rstd;
  P.seed = debug_shuffle_seed;
  return hip_status(launch_norm_fwd(P, dtype == MOE_BF16, (hipStream_t)stream));
}

MOE_API moe_status moe_layernorm_workspace_size(int64_t rows, int64_t cols, size_t* bwd_bytes) {
  const moe_status s = check_norm(MOE_F32, rows, cols);
  if (s != MOE_OK) return s;
  if (!bwd_bytes) return MOE_ERR_NULL;
  // float32 rows may take more blocks than bf16 rows
  *bwd_bytes = rows == 0 ? 0 : align_up((size_t)norm_bwd_blocks(rows, cols, false) * 2 * cols * 4);
  return MOE_OK;
}

MOE_API moe_status moe_layernorm_bwd(const void* dy, const void* x, const void* weight, const float* mean,
                                     const float* rstd, const void* dx_add, moe_dtype dtype, int64_t rows,
                                     int64_t cols, int64_t lddy, int64_t ldx, int64_t ldadd, void* dx,
                                     float* dweight, float* dbias, void* ws, size_t ws_bytes,
                                     uint64_t debug_shuffle_seed, void* stream) {
  moe_status s = check_norm(dtype, rows, cols);
  if (s != MOE_OK) return s;
  if (!ld_ok(rows, cols, lddy) || !ld_ok(rows, cols, ldx) || (dx_add && !ld_ok(rows, cols, ldadd))) return MOE_ERR_SHAPE;
  if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return MOE_ERR_NULL;
  const uintptr_t em = dtype == MOE_BF16 ? 1 : 3;
  if (((uintptr_t)dy | (uintptr_t)x | (uintptr_t)weight | (uintptr_t)dx_add | (uintptr_t)dx) & em) return MOE_ERR_SHAPE;
  if (((uintptr_t)mean | (uintptr_t)rstd | (uintptr_t)dweight | (uintptr_t)dbias) & 3) return MOE_ERR_SHAPE;
  hipStream_t st = (hipStream_t)stream;
  if (rows == 0) {
    if (dweight) MOE_TRY(launch_dense_zero(dweight, 2 * cols, st));
    if (dbias) MOE_TRY(launch_dense_zero(dbias, 2 * cols, st));
    return MOE_OK;
  }
  const bool bf16 = dtype == MOE_BF16;
  const int blocks = norm_bwd_blocks(rows, cols, bf16);
  const bool sums = dweight || dbias;
  if (sums && (s = check_ws(ws, ws_bytes, (size_t)blocks * 2 * cols * 4)) != MOE_OK) return s;
  NormParams P{};
  P.x = x;
  P.weight = weight;
  P.dy = dy;
  P.add = dx_add;
  P.rows = rows;
  P.ldx = ldx;
  P.lddy = lddy;
  P.ldadd = ldadd;
  P.cols = (int)cols;
  P.y = dx;
  P.mean = const_cast<float*>(mean);
  P.rstd = const_cast<float*>(rstd);
  P.part = sums ? (float*)ws : nullptr;
  P.blocks = blocks;
  P.seed = debug_shuffle_seed;
  MOE_TRY(launch_norm_bwd(P, bf16, st));
  if (sums) MOE_TRY(launch_block_sums(P.part, blocks, 2 * cols, (int)cols, dweight, dbias, st));
  return MOE_OK;
}

// ------------------------------------------------------------ linear and gated
MOE_API moe_status moe_linear_workspace_size(const moe_dense* p, size_t* fwd_bytes, size_t* bwd_bytes) {
  return workspace_size(p, 1, fwd_bytes, bwd_bytes);
}

MOE_API moe_status moe_glu_workspace_size(const moe_dense* p, size_t* fwd_bytes, size_t* bwd_bytes) {
  return workspace_size(p, 2, fwd_bytes, bwd_bytes);
}

MOE_API moe_status moe_linear_stage_names(const moe_dense* p, int call, char* names, size_t bytes) {
  return stage_names(p, 1, call, names, bytes);
}

MOE_API moe_status moe_glu_stage_names(const moe_dense* p, int call, char* names, size_t bytes) {
  return stage_names(p, 2, call, names, bytes);
}

MOE_API moe_status moe_linear_fwd(const moe_dense* p, const void* x, const void* w, const void* bias,
                                  const void* residual, void* y, void* z, void* ws, size_t ws_bytes, void* stream) {
  return forward(p, 1, x, w, w, bias, residual, y, z, nullptr, ws, ws_bytes, (hipStream_t)stream);
}

MOE_API moe_status moe_linear_bwd(const moe_dense* p, const void* dy, const void* x, const void* w, const void* z,
                                  const void* dx_add, void* dx, void* dw, void* db, void* ws, size_t ws_bytes,
                                  void* stream) {
  return backward(p, 1, dy, x, w, w, z, z, dx_add, dx, dw, dw, db, ws, ws_bytes, (hipStream_t)stream);
}

MOE_API moe_status moe_glu_fwd(const moe_dense* p, const void* x, const void* wg, const void* wu, void* a, void* g,
                               void* u, void* ws, size_t ws_bytes, void* stream) {
  return forward(p, 2, x, wg, wu, nullptr, nullptr, a, g, u, ws, ws_bytes, (hipStream_t)stream);
}

MOE_API moe_status moe_glu_bwd(const moe_dense* p, const void* da, const void* x, const void* wg, const void* wu,
                               const void* g, const void* u, const void* dx_add, void* dx, void* dwg, void* dwu,
                               void* ws, size_t ws_bytes, void* stream) {
  return backward(p, 2, da, x, wg, wu, g, u, dx_add, dx, dwg, dwu, nullptr, ws, ws_bytes, (hipStream_t)stream);
}
