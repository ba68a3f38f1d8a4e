// Host side of the C ABI of the pieces of an expert layer (declared in
// include/moedet.h): the sort, the rows' copies and sums, and dropout.
#include <cmath>

#include "../../include/moedet.h"
#include "rows.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moedet {
namespace {

constexpr size_t kWsAlign = 256;
constexpr int64_t kMaxCols = (int64_t)1 << 24;
constexpr int64_t kMaxElems = (int64_t)1 << 40;

moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

int elem_bytes(int dtype) {
  switch (dtype) {
    case MOE_F32: return 4;
    case MOE_BF16: return 2;
    case MOE_I8:
    case MOE_U8: return 1;
    default: return 0;
  }
}
bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

moe_status check_slots(int64_t tokens, int32_t top_k) {
  if (tokens < 0 || top_k < 1 || tokens > ((int64_t)0x7fffffff) / top_k) return MOE_ERR_SHAPE;
  return MOE_OK;
}

moe_status check_sort(int64_t tokens, int32_t top_k, int32_t num_local) {
  const moe_status s = check_slots(tokens, top_k);
  if (s != MOE_OK) return s;
  return num_local < 1 || num_local > kSortMaxLocal ? MOE_ERR_SHAPE : MOE_OK;
}

size_t sort_ws(int64_t n, int local) {
  int64_t chunk;
  int chunks;
  sort_chunks(n, local, &chunk, &chunks);
  if (chunks == 1) return 0;
  return ((size_t)chunks * local * 4 + kWsAlign - 1) / kWsAlign * kWsAlign;
}

// What the four row calls share; `dtypes`: whether one-byte types are allowed.
moe_status check_rows(const void* token_side, int dtype, bool bytes, int64_t tokens, int32_t top_k, int32_t cols,
                      int64_t ld, int64_t nrows, const int32_t* slot_row) {
  const int es = elem_bytes(dtype);
  if (es == 0 || (es == 1 && !bytes)) return MOE_ERR_DTYPE;
  moe_status s = check_slots(tokens, top_k);
  if (s != MOE_OK) return s;
  if (cols < 1 || cols > kMaxCols || ld < cols || nrows < 0 || nrows > 0x7fffffff) return MOE_ERR_SHAPE;
  if (ld > kMaxElems || tokens * (double)ld > (double)kMaxElems || nrows * (double)cols > (double)kMaxElems) return MOE_ERR_SHAPE;
  if (tokens > 0 && (!token_side || !slot_row)) return MOE_ERR_NULL;
  if (!aligned(token_side, es) || !aligned(slot_row, 4)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

moe_status sum_rows(const void* rows, int dtype, int64_t tokens, int32_t top_k, int32_t cols, int64_t nrows,
                    const int32_t* slot_row, const float* prob, const void* add, int64_t ldadd, void* y, uint64_t seed,
                    void* stream) {
  moe_status s = check_rows(y, dtype, false, tokens, top_k, cols, cols, nrows, slot_row);
  if (s != MOE_OK) return s;
  const int es = elem_bytes(dtype);
  if (add && (ldadd < cols || ldadd > kMaxElems || tokens * (double)ldadd > (double)kMaxElems)) return MOE_ERR_SHAPE;
  if (!aligned(rows, es) || !aligned(prob, 4) || !aligned(add, es)) return MOE_ERR_SHAPE;
  if (tokens == 0) return MOE_OK;
  RowsParams P{};
  P.tokens = tokens;
  P.k = top_k;
  P.cols = cols;
  P.nrows = nrows;
  P.slot_row = slot_row;
  P.prob = prob;
  P.rows = rows;
  P.add = add;
  P.ldadd = ldadd;
  P.out = y;
  P.seed = seed;
  if (unpermute_grid(P, dtype == MOE_BF16) > kMaxGrid) return MOE_ERR_SHAPE;
  if (nrows > 0 && !rows) return MOE_ERR_NULL;
  return hip_status(launch_unpermute(P, dtype == MOE_BF16, (hipStream_t)stream));
}

moe_status dropout(const void* x, const void* add, int dtype, int64_t rows, int64_t cols, int64_t ldx, int64_t ldadd,
                   double p, const uint64_t* rng, void* y, uint64_t seed, void* stream) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
  const int es = elem_bytes(dtype);
  if (!(p >= 0.0 && p <= 1.0)) return MOE_ERR_SHAPE;
  if (rows < 0 || cols < 1 || cols > 0x7fffffff || ldx < cols || (add && ldadd < cols)) return MOE_ERR_SHAPE;
  if (ldx > kMaxElems || rows * (double)ldx > (double)kMaxElems) return MOE_ERR_SHAPE;
  if (add && (ldadd > kMaxElems || rows * (double)ldadd > (double)kMaxElems)) return MOE_ERR_SHAPE;
  if (rows == 0) return MOE_OK;
  DropoutParams P{};
  P.rows = rows;
  P.cols = (int)cols;
  P.x = x;
  P.ldx = ldx;
  P.add = add;
  P.ldadd = ldadd;
  P.y = y;
  P.rng = rng;
  const uint64_t limit = (uint64_t)std::nearbyint(p * 4294967296.0);
  P.limit = (uint32_t)limit;
  P.all = limit >> 32;
  P.scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f;
  P.seed = seed;
  if (dropout_grid(P, dtype == MOE_BF16) > kMaxGrid) return MOE_ERR_SHAPE;
  if (!x || !y || !rng) return MOE_ERR_NULL;
  if (!aligned(x, es) || !aligned(y, es) || !aligned(add, es) || !aligned(rng, 8)) return MOE_ERR_SHAPE;
  return hip_status(launch_dropout(P, dtype == MOE_BF16, (hipStream_t)stream));
}

}  // namespace
}  // namespace moedet

using namespace moedet;

MOE_API moe_status moe_sort_workspace_size(int64_t tokens, int32_t top_k, int32_t num_local, size_t* bytes) {
  const moe_status s = check_sort(tokens, top_k, num_local);
  if (s != MOE_OK) return s;
  if (!bytes) return MOE_ERR_NULL;
  *bytes = sort_ws(tokens * top_k, num_local);
  return MOE_OK;
}

MOE_API moe_status moe_sort(const void* topk_idx, moe_dtype idx_dtype, int64_t tokens, int32_t top_k,
                            int32_t expert_begin, int32_t num_local, int32_t* slot_row, int32_t* offsets,
                            int32_t* row_src, void* ws, size_t ws_bytes, uint64_t debug_shuffle_seed, void* stream) {
  if (idx_dtype != MOE_I32 && idx_dtype != MOE_I64) return MOE_ERR_DTYPE;
  const moe_status s = check_sort(tokens, top_k, num_local);
  if (s != MOE_OK) return s;
  if (expert_begin < 0) return MOE_ERR_SHAPE;
  const int64_t n = tokens * top_k;
  if (!offsets || (n > 0 && (!topk_idx || !slot_row))) return MOE_ERR_NULL;
  if (!aligned(topk_idx, idx_dtype == MOE_I64 ? 8 : 4) || !aligned(slot_row, 4) || !aligned(offsets, 4) || !aligned(row_src, 4))
    return MOE_ERR_SHAPE;
  const size_t need = sort_ws(n, num_local);
  if (need && !ws) return MOE_ERR_NULL;
  if (need && (ws_bytes < need || !aligned(ws, kWsAlign))) return MOE_ERR_WORKSPACE;
  SortParams P{};
  P.idx = topk_idx;
  P.wide = idx_dtype == MOE_I64;
  P.n = n;
  P.begin = expert_begin;
  P.local = num_local;
  sort_chunks(n, num_local, &P.chunk, &P.chunks);
  P.hist = (int32_t*)ws;
  P.slot_row = slot_row;
  P.offsets = offsets;
  P.row_src = row_src;
  P.seed = debug_shuffle_seed;
  return hip_status(launch_sort(P, (hipStream_t)stream));
}

MOE_API moe_status moe_permute_fwd(const void* x, moe_dtype dtype, int64_t tokens, int32_t top_k, int32_t cols,
                                   int64_t ldx, const int32_t* slot_row, int64_t nrows, void* rows,
                                   uint64_t debug_shuffle_seed, void* stream) {
  const moe_status s = check_rows(x, dtype, true, tokens, top_k, cols, ldx, nrows, slot_row);
  if (s != MOE_OK) return s;
  const int es = elem_bytes(dtype);
  if (!aligned(rows, es)) return MOE_ERR_SHAPE;
  if (tokens == 0 || nrows == 0) return MOE_OK;
  RowsParams P{};
  P.tokens = tokens;
  P.k = top_k;
  P.cols = cols;
  P.nrows = nrows;
  P.slot_row = slot_row;
  P.x = x;
  P.ldx = ldx;
  P.out = rows;
  P.seed = debug_shuffle_seed;
  if (permute_grid(P, es) > kMaxGrid) return MOE_ERR_SHAPE;
  if (!rows) return MOE_ERR_NULL;
  return hip_status(launch_permute(P, es, (hipStream_t)stream));
}

MOE_API moe_status moe_permute_bwd(const void* drows, moe_dtype dtype, int64_t tokens, int32_t top_k, int32_t cols,
                                   const int32_t* slot_row, int64_t nrows, const void* dx_add, int64_t ldadd, void* dx,
                                   uint64_t debug_shuffle_seed, void* stream) {
  return sum_rows(drows, dtype, tokens, top_k, cols, nrows, slot_row, nullptr, dx_add, ldadd, dx, debug_shuffle_seed, stream);
}

MOE_API moe_status moe_unpermute_fwd(const void* rows, moe_dtype dtype, int64_t tokens, int32_t top_k, int32_t cols,
                                     const int32_t* slot_row, int64_t nrows, const float* prob, const void* residual,
                                     int64_t ldr, void* y, uint64_t debug_shuffle_seed, void* stream) {
  return sum_rows(rows, dtype, tokens, top_k, cols, nrows, slot_row, prob, residual, ldr, y, debug_shuffle_seed, stream);
}

MOE_API moe_status moe_unpermute_bwd(const void* dy, int64_t lddy, const void* rows, moe_dtype dtype, int64_t tokens,
                                     int32_t top_k, int32_t cols, const int32_t* slot_row, int64_t nrows,
                                     const float* prob, void* drows, float* dprob, uint64_t debug_shuffle_seed,
                                     void* stream) {
  const moe_status s = check_rows(dy, dtype, false, tokens, top_k, cols, lddy, nrows, slot_row);
  if (s != MOE_OK) return s;
  const int es = elem_bytes(dtype);
  if (!aligned(rows, es) || !aligned(drows, es) || !aligned(prob, 4) || !aligned(dprob, 4)) return MOE_ERR_SHAPE;
  if (tokens == 0) return MOE_OK;
  RowsParams P{};
  P.tokens = tokens;
  P.k = top_k;
  P.cols = cols;
  P.nrows = nrows;
  P.slot_row = slot_row;
  P.prob = prob;
  P.x = dy;
  P.ldx = lddy;
  P.rows = rows;
  P.out = drows;
  P.dprob = dprob;
  P.seed = debug_shuffle_seed;
  if (unpermute_bwd_grid(P, dtype == MOE_BF16) > kMaxGrid) return MOE_ERR_SHAPE;
  if (!prob || (nrows > 0 && (!drows || (dprob && !rows)))) return MOE_ERR_NULL;
  return hip_status(launch_unpermute_bwd(P, dtype == MOE_BF16, (hipStream_t)stream));
}

MOE_API moe_status moe_dropout_fwd(const void* x, const void* residual, moe_dtype dtype, int64_t rows, int64_t cols,
                                   int64_t ldx, int64_t ldr, double p, const uint64_t* rng, void* y,
                                   uint64_t debug_shuffle_seed, void* stream) {
  return dropout(x, residual, dtype, rows, cols, ldx, ldr, p, rng, y, debug_shuffle_seed, stream);
}

MOE_API moe_status moe_dropout_bwd(const void* dy, moe_dtype dtype, int64_t rows, int64_t cols, int64_t lddy, double p,
                                   const uint64_t* rng, void* dx, uint64_t debug_shuffle_seed, void* stream) {
  return dropout(dy, nullptr, dtype, rows, cols, lddy, 0, p, rng, dx, debug_shuffle_seed, stream);
}
