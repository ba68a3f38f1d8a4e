// Host side of the C ABI of the products in 8-bit integers (declared in
// include/moedet.h): argument checks, workspace, and the choice of kernel from
// sizes alone.
#include "../../include/moedet.h"
#include "int8.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moedet {
namespace {

constexpr size_t kWsAlign = 256;
constexpr int64_t kMaxLd = (int64_t)1 << 20;
constexpr int64_t kMaxElems = (int64_t)1 << 40;
constexpr int64_t kMaxUnits = ((int64_t)1 << 24) - 8;

moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
size_t align_up(size_t v) { return (v + kWsAlign - 1) / kWsAlign * kWsAlign; }
bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }
int size_of(int dtype) { return dtype == MOE_F32 ? 4 : dtype == MOE_BF16 ? 2 : 1; }
int up16(int64_t n) { return (int)((n + 15) / 16 * 16); }

// A kernel of the product: few rows (mt > 0) or a tile.
struct Choice {
  int mt, tile;
};

// Tiles' costs as in the bf16 operators (choose in dense_api.hip), per slice of 64
// codes (128 in the small tiles): alone while at most half of the CUs have one, busy when
// all do.
struct TileCost {
  double alone, busy, fixed;
  bool shares;
};
constexpr TileCost kTiles[kInt8Tiles] = {{0.7, 0.8, 9.0, false}, {0.36, 0.48, 8.0, false}, {0.38, 0.52, 5.8, false}, {0.2, 0.23, 4.5, true}};
constexpr int kCUs = 256;

Choice choose(int64_t rows, int64_t N, int64_t K, int64_t groups) {
  // rows that share a matrix, were they spread evenly
  const int64_t each = (rows + groups - 1) / groups;
  if (each <= 16) return {1, 0};
  if (each <= 32) return {2, 0};
  Choice best{0, -1};
  double least = 0;
  for (int i = 0; i < kInt8Tiles; ++i) {
    const TileCost& c = kTiles[i];
    const DenseShape sh = dense_shape(kFormLinear, true, i);
    const int64_t tiles = groups * ((each + sh.bm - 1) / sh.bm) * ((N + sh.bn - 1) / sh.bn);
    const double steps = (double)((K / 2 + sh.bk - 1) / sh.bk);
    const double per_cu = (double)((tiles + kCUs - 1) / kCUs);
    double slice, t = c.fixed;
    if (c.shares) {
      slice = per_cu * c.busy > c.alone ? per_cu * c.busy : c.alone;
    } else {
      const double over = 2.0 * (double)tiles / kCUs - 1;
      slice = per_cu * (over <= 0 ? c.alone : over >= 1 ? c.busy : c.alone + over * (c.busy - c.alone));
      t += (per_cu - 1) * 0.6 * c.fixed;
    }
    t += steps * slice;
    if (best.tile < 0 || t < least) {
      best.tile = i;
      least = t;
    }
  }
  return best;
}

// Workgroups that a launch may need at most.
int64_t units(const Choice& c, int64_t rows, int64_t N, int64_t groups) {
  const DenseShape sh = c.mt ? DenseShape{16 * c.mt, 16, 64} : dense_shape(kFormLinear, true, c.tile);
  int64_t mT = rows / sh.bm + groups;
  if (mT > rows) mT = rows;
  return mT * ((N + sh.bn - 1) / sh.bn);
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
  const int64_t groups = p->num_local ? p->num_local : 1;
  if (units(choose(p->rows, p->d_out, up16(p->d_in), groups), p->rows, p->d_out, groups) > kMaxUnits) return MOE_ERR_SHAPE;
  return MOE_OK;
}

size_t codes_bytes(const moe_int8* p) { return align_up((size_t)p->rows * up16(p->d_in)); }
size_t ws_need(const moe_int8* p) {
  return p->x_dtype == MOE_I8 || p->rows == 0 ? 0 : codes_bytes(p) + align_up((size_t)p->rows * 4);
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
  const size_t need = ws_need(p);
  if (need && !ws) return MOE_ERR_NULL;
  if (need && (ws_bytes < need || !aligned(ws, kWsAlign))) return MOE_ERR_WORKSPACE;
  const int K = up16(p->d_in);
  Int8Params P{};
  P.d.M = p->rows;
  P.d.N = p->d_out;
  P.d.K = K;
  P.d.nseg = P.d.S = 1;
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
  if (!codes) {
    Int8QuantParams Q{};
    Q.x = x;
    Q.rows = p->rows;
    Q.ldx = p->ldx;
    Q.cols = p->d_in;
    Q.cols16 = K;
    Q.limit = offsets ? offsets + p->num_local : nullptr;
    Q.codes = (int8_t*)ws;
    Q.scales = (float*)((char*)ws + codes_bytes(p));
    Q.seed = p->debug_shuffle_seed;
    if (launch_int8_quantize(Q, p->x_dtype == MOE_BF16, st) != hipSuccess) return MOE_ERR_HIP;
    P.a = Q.codes;
    P.lda = K;
    P.sa = Q.scales;
  }
  const Choice c = choose(p->rows, p->d_out, K, P.groups);
  const bool bf16 = p->dtype == MOE_BF16;
  return hip_status(c.mt ? launch_int8_few(P, bf16, c.mt, st) : launch_int8_tiles(P, bf16, c.tile, st));
}

}  // namespace
}  // namespace moedet

using namespace moedet;

MOE_API moe_status moe_int8_quantize(const void* x, moe_dtype dtype, int64_t rows, int64_t cols, int64_t ldx,
                                     int8_t* codes, float* scales, uint64_t debug_shuffle_seed, void* stream) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (rows < 0 || rows >= (int64_t)1 << 31 || cols < 1 || cols > kInt8MaxK || ldx < cols || ldx >= kMaxElems) return MOE_ERR_SHAPE;
  if (rows * (double)ldx > (double)kMaxElems) return MOE_ERR_SHAPE;
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
  if (batch * (double)rows * (double)cols > (double)kMaxElems || batch * (double)((cols + 63) / 64) > (double)kMaxUnits)
    return MOE_ERR_SHAPE;
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
  *bytes = ws_need(p);
  return MOE_OK;
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
