// Host side of the C ABI of the products in 8-bit integers (declared in
// include/moedet.h): argument checks, workspace, and the choice of kernel from
// sizes alone.
#include <cstdio>

#include "../../include/moedet.h"
#include "int8.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moedet {
namespace {

constexpr size_t kWsAlign = 256;
constexpr int64_t kMaxLd = (int64_t)1 << 20;
constexpr int64_t kMaxElems = (int64_t)1 << 40;

moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
size_t align_up(size_t v) { return (v + kWsAlign - 1) / kWsAlign * kWsAlign; }
bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }
int size_of(int dtype) { return dtype == MOE_F32 ? 4 : dtype == MOE_BF16 ? 2 : 1; }
int up16(int64_t n) { return (int)((n + 15) / 16 * 16); }

constexpr int kCUs = 256;

// The kernel of a product: few rows (ks > 0, fused: x is quantised by it), or a tile and the
// chunks of its contraction.  Of experts, p->rows are the rows that x has room for: how many there are is
// known on the GPU alone.  (About 2050 rows of 4 experts, 2048 x 2048, in an x of as many 28.6 us, of 65536
// rows 39.9, of 360448 60: larger tiles, and workgroups without a tile.)
struct Choice {
  int ks, tile, S;
  bool fused;
};

// A tile's cost in microseconds, fitted to the times in int8.h: `each` a slice of each of
// the workgroups that share a CU, `alone` one by itself, `fixed` the launch, first
// slice and epilogue of a round.
struct TileCost {
  double alone, each, fixed;
  int shares;               // workgroups a CU
};
constexpr TileCost kTiles[kInt8Tiles] = {{1.0, 1.45, 12.0, 1}, {0.52, 0.47, 8.5, 2}, {0.26, 0.27, 5.5, 2}, {0.46, 0.286, 6.3, 3}, {0.44, 0.2, 4.0, 5}, {0.24, 0.18, 3.3, 2}};

double estimate(int i, double tiles, double steps, int act) {
  const TileCost& c = kTiles[i];
  const double per_cu = tiles / kCUs;
  // a SiLU or GELU epilogue has nothing beside it here (8192 x 2048 x 1024 with GELU 31 us, with
  // tiles of 128 x 128 31; without 23 and 27)
  if (c.shares == 1)
    return (double)(int64_t)(per_cu + 0.999) * (c.fixed + (act >= MOE_ACT_SILU ? 4.0 : 0.0) + steps * (per_cu <= 0.5 ? c.alone : c.each));
  const double full = per_cu / c.shares;   // rounds of a full CU
  const double slice = per_cu * c.each > c.alone ? per_cu * c.each : c.alone;
  return c.fixed * (full < 1 ? 1 : 0.4 + 0.6 * full) + steps * slice;
}

Choice choose(const moe_int8* p, int64_t K) {
  const int64_t rows = p->rows, N = p->d_out, groups = p->num_local ? p->num_local : 1;
  Choice best{0, 0, 1, false};
  // 16 rows and fewer of one matrix (16 x 2048 x 2048 5.3 us, with a tile 7.1), and experts
  // of up to 3 rows were they spread evenly, stream the weights (4 tokens of 22 experts of 512, 352 MB:
  // 60 us, with tiles 66; 16 tokens, 1079 MB: 178 and 205; but 800 rows of 64 experts 82 and 55).
  if (p->num_local ? rows <= 3 * groups : rows <= 16) {
    // a wave to 16 weight rows where that fills the device, else four (22 experts of
    // 2048 x 2048: 17.8 and 19.8 us; 1 x 2048 x 2048: 8 and 4.5)
    const int64_t waves = (N + 15) / 16 * (p->num_local ? rows : 1);
    best.ks = waves >= 2048 ? 1 : 4;
    best.fused = p->x_dtype == p->dtype && (p->num_local || rows <= kInt8FusedRows) && (p->num_local ? 16 : rows) * K <= kInt8FusedBytes;
    return best;
  }
  double least = -1;
  for (int i = 0; i < kInt8Tiles; ++i) {
    const Int8Shape& sh = kInt8Shapes[i];
    const double nT = (double)((N + sh.bn - 1) / sh.bn);
    // experts leave half a tile each on average
    double mT = (double)((rows + sh.bm - 1) / sh.bm);
    if (groups > 1) mT = (double)rows / sh.bm + 0.5 * (double)(groups < rows ? groups : rows);
    const int64_t steps = (K + kInt8Slice - 1) / kInt8Slice;
    for (int S = 1; S <= 8; S *= 2) {
      // the 64 x 64 tile of one matrix may be split while workgroups are few
      if (S > 1 && (i != kInt8Tiles - 1 || p->num_local || steps / S < 4 || mT * nT * S > 2 * kCUs)) break;
      double t = estimate(i, mT * nT * S, (double)((steps + S - 1) / S), p->act);
      // the sums written and read, and the join
      if (S > 1) t += 3.2 + (double)S * (double)rows * (double)N * 8.0 / 3e6;
      // the weights at 5.2 TB/s; of tiles that reach that, the quickest
      const double stream = (double)groups * (double)N * (double)K / 5.2e6;
      t = (t > stream ? t : stream) + 0.1 * t;
      if (least < 0 || t < least) {
        best.tile = i;
        best.S = S;
        least = t;
      }
    }
  }
  return best;
}

// Workgroups that a launch may need at most.
int64_t units(const moe_int8* p, const Choice& c) {
  const int64_t bm = c.ks ? 16 : kInt8Shapes[c.tile].bm, bn = c.ks ? 64 / c.ks : kInt8Shapes[c.tile].bn;
  int64_t mT = p->rows / bm + (p->num_local ? p->num_local : 1);
  if (mT > p->rows) mT = p->rows;
  return mT * ((p->d_out + bn - 1) / bn) * c.S;
}

moe_status check(const moe_int8* p) {
  if (!p) return MOE_ERR_NULL;
  if (p->x_dtype != MOE_F32 && p->x_dtype != MOE_BF16 && p->x_dtype != MOE_I8) return MOE_ERR_DTYPE;
  if (p->dtype != MOE_F32 && p->dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (p->act < MOE_ACT_NONE || p->act > MOE_ACT_GELU) return MOE_ERR_MODE;
  if (p->rows < 0 || p->rows >= (int64_t)1 << 31) return MOE_ERR_SHAPE;
  if (p->d_in < 1 || p->d_in > kInt8MaxK || p->d_out < 1 || p->d_out >= kMaxLd) return MOE_ERR_SHAPE;
  if (p->num_local < 0 || p->num_local > kInt8MaxGroups) return MOE_ERR_SHAPE;
  if (p->ldx < p->d_in || p->ldx >= kMaxLd || p->ldy < p->d_out || p->ldy >= kMaxLd || p->ldr < 0 || p->ldr >= kMaxLd) return MOE_ERR_SHAPE;
  if (p->x_dtype == MOE_I8 && (p->d_in % 16 || p->ldx % 16)) return MOE_ERR_SHAPE;
  const Choice c = choose(p, up16(p->d_in));
  if (units(p, c) > kMaxGrid) return MOE_ERR_SHAPE;
  if (p->x_dtype != MOE_I8 && !c.fused && int8_quantize_grid(p->rows, up16(p->d_in), p->x_dtype == MOE_BF16) > kMaxGrid) return MOE_ERR_SHAPE;
  return MOE_OK;
}

// Workspace: codes and scales of x, then the sums of a split contraction.
struct Plan {
  Choice c;
  int K;
  int64_t part_ld;
  size_t scales, part, total;   // byte offsets
};
Plan plan(const moe_int8* p) {
  Plan w{};
  w.K = up16(p->d_in);
  w.c = choose(p, w.K);
  if (p->rows == 0) return w;
  size_t o = 0;
  if (p->x_dtype != MOE_I8 && !w.c.fused) {
    o = align_up((size_t)p->rows * w.K);
    w.scales = o;
    o += align_up((size_t)p->rows * 4);
  }
  if (w.c.S > 1) {
    w.part_ld = ((int64_t)p->d_out + 3) / 4 * 4;
    w.part = o;
    o += align_up((size_t)w.c.S * p->rows * w.part_ld * 4);
  }
  w.total = o;
  return w;
}

moe_status product(const moe_int8* p, const void* x, const float* x_scales, const int8_t* w_codes, const float* w_scales,
                   const void* bias, const void* residual, const int32_t* offsets, void* y, void* ws, size_t ws_bytes,
                   hipStream_t st) {
  if (p->rows == 0) return MOE_OK;
  const bool codes = p->x_dtype == MOE_I8;
  if (!x || !w_codes || !w_scales || !y || (codes && !x_scales)) return MOE_ERR_NULL;
  const int es = size_of(p->dtype);
  if (!aligned(x, codes ? 16 : size_of(p->x_dtype)) || !aligned(x_scales, 4) || !aligned(w_codes, 16) || !aligned(w_scales, 4) ||
      !aligned(bias, es) || !aligned(residual, es) || !aligned(y, es) || !aligned(offsets, 4))
    return MOE_ERR_SHAPE;
  if (residual && p->ldr < p->d_out) return MOE_ERR_SHAPE;
  const Plan w = plan(p);
  if (w.total && !ws) return MOE_ERR_NULL;
  if (w.total && (ws_bytes < w.total || !aligned(ws, kWsAlign))) return MOE_ERR_WORKSPACE;
  const int K = w.K;
  Int8Params P{};
  P.d.M = p->rows;
  P.d.N = p->d_out;
  P.d.K = K;
  P.d.nseg = 1;
  P.d.S = w.c.S;
  P.d.bias = bias;
  P.d.add = residual;
  P.d.ldadd = p->ldr;
  P.d.c[0] = y;
  P.d.ldc = p->ldy;
  P.d.act = p->act;
  P.d.seed = p->debug_shuffle_seed;
  P.a = (const int8_t*)x;
  P.lda = p->ldx;
  P.sa = x_scales;
  P.b = w_codes;
  P.sb = w_scales;
  P.offsets = offsets;
  P.groups = offsets ? p->num_local : 1;
  const bool bf16 = p->dtype == MOE_BF16;
  P.part = (int32_t*)((char*)ws + w.part);
  P.part_ld = w.part_ld;
  if (w.c.fused) {
    P.x = x;
    P.ldx = p->ldx;
    P.xcols = p->d_in;
  } else if (!codes) {
    Int8QuantParams Q{};
    Q.x = x;
    Q.rows = p->rows;
    Q.ldx = p->ldx;
    Q.cols = p->d_in;
    Q.cols16 = K;
    Q.limit = offsets ? offsets + p->num_local : nullptr;
    Q.codes = (int8_t*)ws;
    Q.scales = (float*)((char*)ws + w.scales);
    Q.seed = p->debug_shuffle_seed;
    const hipError_t e = launch_int8_quantize(Q, p->x_dtype == MOE_BF16, st);
    if (e != hipSuccess) return hip_status(e);
    P.a = Q.codes;
    P.lda = K;
    P.sa = Q.scales;
  }
  return hip_status(w.c.ks ? launch_int8_few(P, bf16, w.c.ks, st) : launch_int8_tiles(P, bf16, w.c.tile, st));
}

}  // namespace
}  // namespace moedet

using namespace moedet;

MOE_API moe_status moe_int8_quantize(const void* x, moe_dtype dtype, int64_t rows, int64_t cols, int64_t ldx,
                                     int8_t* codes, float* scales, uint64_t debug_shuffle_seed, void* stream) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (rows < 0 || rows >= (int64_t)1 << 31 || cols < 1 || cols > kInt8MaxK || ldx < cols || ldx >= kMaxElems) return MOE_ERR_SHAPE;
  if (rows * (double)ldx > (double)kMaxElems || int8_quantize_grid(rows, up16(cols), dtype == MOE_BF16) > kMaxGrid) return MOE_ERR_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales) return MOE_ERR_NULL;
  if (!aligned(x, size_of(dtype)) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_SHAPE;
  Int8QuantParams P{};
  P.x = x;
  P.rows = rows;
  P.ldx = ldx;
  P.cols = (int)cols;
  P.cols16 = up16(cols);
  P.codes = codes;
  P.scales = scales;
  P.seed = debug_shuffle_seed;
  return hip_status(launch_int8_quantize(P, dtype == MOE_BF16, (hipStream_t)stream));
}

MOE_API moe_status moe_int8_quantize_t(const void* w, moe_dtype dtype, int64_t batch, int64_t rows, int64_t cols,
                                       int8_t* codes, float* scales, uint64_t debug_shuffle_seed, void* stream) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (batch < 0 || rows < 1 || rows > kInt8MaxK || cols < 1 || cols >= kMaxLd) return MOE_ERR_SHAPE;
  if (batch * (double)rows * (double)cols > (double)kMaxElems) return MOE_ERR_SHAPE;
  if (int8_quantize_t_grid(batch, (int)cols) > kMaxGrid / 2) return MOE_ERR_SHAPE;   // workgroups of 512 threads
  if (batch == 0) return MOE_OK;
  if (!w || !codes || !scales) return MOE_ERR_NULL;
  if (!aligned(w, size_of(dtype)) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_SHAPE;
  Int8QuantTParams P{};
  P.w = w;
  P.batch = batch;
  P.rows = (int)rows;
  P.cols = (int)cols;
  P.rows16 = up16(rows);
  P.codes = codes;
  P.scales = scales;
  P.seed = debug_shuffle_seed;
  return hip_status(launch_int8_quantize_t(P, dtype == MOE_BF16, (hipStream_t)stream));
}

MOE_API moe_status moe_int8_workspace_size(const moe_int8* p, size_t* bytes) {
  const moe_status s = check(p);
  if (s != MOE_OK) return s;
  if (!bytes) return MOE_ERR_NULL;
  *bytes = plan(p).total;
  return MOE_OK;
}

MOE_API moe_status moe_int8_stage_names(const moe_int8* p, char* names, size_t bytes) {
  const moe_status s = check(p);
  if (s != MOE_OK) return s;
  if (!names) return MOE_ERR_NULL;
  if (bytes < 1) return MOE_ERR_WORKSPACE;
  static const char* const kNames[kInt8Tiles] = {"256x256", "128x128", "128x64_deep", "128x64", "64x64", "64x64_deep"};   // kInt8Shapes
  const Choice c = choose(p, up16(p->d_in));
  const char* kind = p->num_local ? "experts" : "linear";
  const char* first = p->x_dtype == MOE_I8 || c.fused ? "" : "quantize,";
  int n;
  if (p->rows == 0)
    n = snprintf(names, bytes, "%s", "");
  else if (c.ks)
    n = snprintf(names, bytes, "%s%s_few%d%s", first, kind, c.ks, c.fused ? "_quantize" : "");
  else if (c.S > 1)
    n = snprintf(names, bytes, "%s%s_%s_split%d,join", first, kind, kNames[c.tile], c.S);
  else
    n = snprintf(names, bytes, "%s%s_%s", first, kind, kNames[c.tile]);
  return n >= 0 && (size_t)n < bytes ? MOE_OK : MOE_ERR_WORKSPACE;
}

MOE_API moe_status moe_int8_linear(const moe_int8* p, const void* x, const float* x_scales, const int8_t* w_codes,
                                   const float* w_scales, const void* bias, const void* residual, void* y, void* ws,
                                   size_t ws_bytes, void* stream) {
  const moe_status s = check(p);
  if (s != MOE_OK) return s;
  if (p->num_local != 0) return MOE_ERR_SHAPE;
  return product(p, x, x_scales, w_codes, w_scales, bias, residual, nullptr, y, ws, ws_bytes, (hipStream_t)stream);
}

MOE_API moe_status moe_int8_experts(const moe_int8* p, const void* x, const float* x_scales, const int8_t* w_codes,
                                    const float* w_scales, const void* bias, const int32_t* offsets, void* y, void* ws,
                                    size_t ws_bytes, void* stream) {
  const moe_status s = check(p);
  if (s != MOE_OK) return s;
  if (p->num_local < 1) return MOE_ERR_SHAPE;
  if (!offsets) return MOE_ERR_NULL;
  return product(p, x, x_scales, w_codes, w_scales, bias, nullptr, offsets, y, ws, ws_bytes, (hipStream_t)stream);
}
