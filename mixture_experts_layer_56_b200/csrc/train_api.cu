// C ABI of the training operators (include/moe.h): validation, workspace
// carving and launches on the caller's stream.
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "mm_sm100.h"
#include "train_kernels.h"

namespace moe {
namespace {

inline bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
template <typename... P> bool any_null(P... p) { return ((p == nullptr) || ...); }
template <typename... P> bool any_misaligned(P... p) { return (misaligned(p) || ...); }

inline bool known_dtype(int32_t t) { return t == MOE_DTYPE_F32 || t == MOE_DTYPE_BF16; }

constexpr size_t kStatusBytes = 256;  // the status word at the workspace's start
constexpr int32_t kMaxSide = 1 << 24;
// Rows per group, on average, below which the products take the matrix's rows
// as the tile's: see run_ragged_rows.
constexpr int64_t kFewRows = 512;

int validate(const moe_grouped_shape_t* s) {
  if (!s) return MOE_ERR_NULLPTR;
  if (!known_dtype(s->dtype)) return MOE_ERR_DTYPE;
  if (s->rows < 0 || s->rows > 0x7fffffffll - 511 || s->n_groups < 1 ||
      s->n_groups > sm100::kMmMaxGroups || s->n < 1 || s->n > kMaxSide || s->k < 1 ||
      s->k > kMaxSide)
    return MOE_ERR_SHAPE;
  if (s->dtype == MOE_DTYPE_BF16 && (s->n % 8 != 0 || s->k % 8 != 0)) return MOE_ERR_SHAPE;
  if (s->flags & ~(MOE_GROUPED_DW_F32 | MOE_GROUPED_DW_ACCUMULATE)) return MOE_ERR_SHAPE;
  if ((s->flags & MOE_GROUPED_DW_ACCUMULATE) && s->dtype == MOE_DTYPE_BF16 &&
      !(s->flags & MOE_GROUPED_DW_F32))
    return MOE_ERR_SHAPE;
  // tile numbers are int32, TMA strides below 2^40 bytes
  const int64_t nt = (s->n + 63) / 64, kt = (s->k + 63) / 64, rt = (s->rows + 63) / 64 + s->n_groups;
  const int64_t wide = nt > kt ? nt : kt, side = s->n > s->k ? s->n : s->k;
  if (rt * wide > 0x7fffffffll || s->n_groups * nt * kt > 0x7fffffffll) return MOE_ERR_SHAPE;
  if (s->rows * side >= (1ll << 38) || static_cast<int64_t>(s->n) * s->k >= (1ll << 38))
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

int validate(const moe_swiglu_shape_t* s) {
  if (!s) return MOE_ERR_NULLPTR;
  if (!known_dtype(s->dtype)) return MOE_ERR_DTYPE;
  if (s->rows < 0 || s->rows > 0x7fffffffll || s->inter < 64 || s->inter % 64 != 0 ||
      s->inter > kMaxSide)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

int validate(const moe_norm_shape_t* s) {
  if (!s) return MOE_ERR_NULLPTR;
  if (!known_dtype(s->dtype)) return MOE_ERR_DTYPE;
  if (s->T < 0 || s->T > 0x7fffffffll || s->d < 1 || s->d > kMaxSide || !std::isfinite(s->eps) ||
      s->eps < 0.0f)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

int validate(const moe_ortho_shape_t* s) {
  if (!s) return MOE_ERR_NULLPTR;
  if (!known_dtype(s->dtype)) return MOE_ERR_DTYPE;
  if (s->n_mats < 0 || s->n_mats > 65535 || s->rows < 1 || s->rows > 65536 || s->cols < 1 ||
      s->cols > 65536 || s->steps < 1 || s->steps > 16)
    return MOE_ERR_SHAPE;
  const int64_t rt = (s->rows + 255) / 256, ct = (s->cols + 255) / 256;
  if (s->n_mats * rt * ct > 0x7fffffffll) return MOE_ERR_SHAPE;
  return MOE_OK;
}

// pairs of CTAs for at most `tiles` tiles
int pairs_for(int64_t tiles, int sms) {
  const int64_t most = sms / 2;
  return static_cast<int>(tiles < most ? tiles : most);
}

int64_t ragged_row_blocks(const moe_grouped_shape_t& s) {
  return (s.rows + 255) / 256 + (s.rows < s.n_groups ? s.rows : s.n_groups);
}

// The bf16 products of ragged rows: forward (in = X) and dX (in = dY).
//
// Two ways round.  With the groups' rows as the tile's 256 rows, a group's last
// tile costs a whole one, and where groups have few rows every tile is mostly
// empty and keeps the tensor cores busy for longer than the weights' stream
// takes.  With the matrix's rows in their place the groups' rows are columns,
// which come in steps of 32: 64 groups of 2816 x 2048 with 12 rows each on
// average take 116 us (0.98 of the HBM rate) for 146, with 96 rows 128 for 151,
// with 200 rows 170 for 186.  From some 500 rows on there is nothing between
// them but the output's transposition (16 groups of 4096 rows: 375 for 372 us),
// which short reductions show sooner (8 groups of 256 rows of 2048 x 256: 9.9 us
// for 8.1).
int run_ragged_rows(const moe_grouped_shape_t& s, bool dx, const void* in, const int32_t* offsets,
                    const void* W, void* out, void* ws, int sms, cudaStream_t st) {
  using namespace sm100;
  const int32_t n = dx ? s.k : s.n, k = dx ? s.n : s.k;  // of the product
  const uint64_t k64 = k, rows = s.rows, wn = s.n, wk = s.k;
  const bool swap = s.rows < (k < 512 ? 112 : kFewRows) * s.n_groups;
  MmArgs a{};
  a.offsets = offsets;
  a.rows = static_cast<int32_t>(s.rows);
  a.groups = s.n_groups;
  a.k = k;
  a.out = out;
  a.ld = n;
  a.status = static_cast<int32_t*>(ws);
  CUtensorMap ma, mb, tail;
  if (swap) {
    a.m = n;
    // enough columns for most groups' rows, and fewer where that many tiles
    // leave pairs idle
    const int64_t some = s.rows < s.n_groups ? s.rows : s.n_groups, bands = (n + 255) / 256;
    a.tn = s.rows <= 32                  ? 32
           : s.rows <= 48ll * s.n_groups  ? 64
           : s.rows <= 112ll * s.n_groups ? 128
                                          : 256;
    while (a.tn > 64 && bands * (s.rows / (a.tn / 2) + some) <= sms / 2) a.tn /= 2;
    const int layout = dx ? kMmTT : kMmNT;
    if (!make_map_16bit(&ma, false, W, wk, wn, s.n_groups, wk, wn * wk, mm_box_a(layout)) ||
        !make_map_16bit(&mb, false, in, k64, rows, 1, k64, rows * k64, mm_box_b(layout, a.tn)) ||
        (a.tn == 256 && !make_map_16bit(&tail, false, in, k64, rows, 1, k64, rows * k64, 32)))
      return MOE_ERR_CUDA;
    return launch_mm(layout, kMmRaggedN, kMmStoreTBf16, ma, mb, a,
                     pairs_for(bands * (s.rows / a.tn + some), sms), st, &tail);
  }
  const int layout = dx ? kMmNN : kMmNT;
  a.n = n;
  a.tn = mm_tile_width(n, ragged_row_blocks(s), sms / 2);
  if (!make_map_16bit(&ma, false, in, k64, rows, 1, k64, rows * k64, mm_box_a(layout)) ||
      !make_map_16bit(&mb, false, W, wk, wn, s.n_groups, wk, wn * wk, mm_box_b(layout, a.tn)))
    return MOE_ERR_CUDA;
  return launch_mm(layout, kMmRaggedM, kMmStoreBf16, ma, mb, a,
                   pairs_for(ragged_row_blocks(s) * ((n + a.tn - 1) / a.tn), sms), st);
}

int check_grouped(const moe_grouped_shape_t& s, const void* in, const int32_t* offsets,
                  const void* other, const void* out, const void* ws, size_t ws_bytes) {
  if (any_null(in, offsets, other, out, ws)) return MOE_ERR_NULLPTR;
  if (any_misaligned(in, static_cast<const void*>(offsets), other, out, ws)) return MOE_ERR_ALIGN;
  if (ws_bytes < kStatusBytes) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_grouped_workspace_size(const moe_grouped_shape_t* shape, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULLPTR;
  if (int rc = validate(shape)) return rc;
  *bytes = kStatusBytes;
  return MOE_OK;
}

int moe_grouped_matmul(const moe_grouped_shape_t* shape, const void* X, const int32_t* offsets,
                       const void* W, void* Y, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (int rc = validate(shape)) return rc;
  const moe_grouped_shape_t& s = *shape;
  if (s.rows == 0) return MOE_OK;
  if (int rc = check_grouped(s, X, offsets, W, Y, ws, ws_bytes)) return rc;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  StageScope sg(MOE_KERNEL_GROUPED_FWD, st);
  if (s.dtype == MOE_DTYPE_F32)
    return launch_grouped_f32(kGroupedFwd, static_cast<const float*>(X),
                              static_cast<const float*>(W), offsets, s.n_groups, s.rows, s.n, s.k,
                              static_cast<float*>(Y), false, sms, st);
  return run_ragged_rows(s, false, X, offsets, W, Y, ws, sms, st);
}

int moe_grouped_matmul_dx(const moe_grouped_shape_t* shape, const void* dY, const int32_t* offsets,
                          const void* W, void* dX, void* ws, size_t ws_bytes,
                          moe_stream_t stream) {
  if (int rc = validate(shape)) return rc;
  const moe_grouped_shape_t& s = *shape;
  if (s.rows == 0) return MOE_OK;
  if (int rc = check_grouped(s, dY, offsets, W, dX, ws, ws_bytes)) return rc;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  StageScope sg(MOE_KERNEL_GROUPED_DX, st);
  if (s.dtype == MOE_DTYPE_F32)
    return launch_grouped_f32(kGroupedDx, static_cast<const float*>(dY),
                              static_cast<const float*>(W), offsets, s.n_groups, s.rows, s.n, s.k,
                              static_cast<float*>(dX), false, sms, st);
  return run_ragged_rows(s, true, dY, offsets, W, dX, ws, sms, st);
}

int moe_grouped_matmul_dw(const moe_grouped_shape_t* shape, const void* dY, const void* X,
                          const int32_t* offsets, void* dW, void* ws, size_t ws_bytes,
                          moe_stream_t stream) {
  using namespace sm100;
  if (int rc = validate(shape)) return rc;
  const moe_grouped_shape_t& s = *shape;
  const bool add = (s.flags & MOE_GROUPED_DW_ACCUMULATE) != 0;
  const bool f32_out = s.dtype == MOE_DTYPE_F32 || (s.flags & MOE_GROUPED_DW_F32);
  if (s.rows == 0 && add) return MOE_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int sms = 0;
  if (s.rows == 0) {
    // every group is empty
    if (!dW) return MOE_ERR_NULLPTR;
    if (misaligned(dW)) return MOE_ERR_ALIGN;
    if (int rc = require_device(&sms)) return rc;
    StageScope sg(MOE_KERNEL_GROUPED_DW, st);
    return launch_zero(dW, static_cast<size_t>(s.n_groups) * s.n * s.k * (f32_out ? 4 : 2), st);
  }
  if (int rc = check_grouped(s, dY, offsets, X, dW, ws, ws_bytes)) return rc;
  if (int rc = require_device(&sms)) return rc;
  StageScope sg(MOE_KERNEL_GROUPED_DW, st);
  if (s.dtype == MOE_DTYPE_F32)
    return launch_grouped_f32(kGroupedDw, static_cast<const float*>(dY),
                              static_cast<const float*>(X), offsets, s.n_groups, s.rows, s.n, s.k,
                              static_cast<float*>(dW), add, sms, st);
  const uint64_t n = s.n, k = s.k, rows = s.rows;
  const int64_t bands = static_cast<int64_t>(s.n_groups) * ((s.n + 255) / 256);
  const int32_t tn = mm_tile_width(s.k, bands, sms / 2);
  CUtensorMap ma, mb;
  if (!make_map_16bit(&ma, false, dY, n, rows, 1, n, rows * n, mm_box_a(kMmTN)) ||
      !make_map_16bit(&mb, false, X, k, rows, 1, k, rows * k, mm_box_b(kMmTN, tn)))
    return MOE_ERR_CUDA;
  MmArgs a{};
  a.offsets = offsets;
  a.rows = static_cast<int32_t>(s.rows);
  a.groups = s.n_groups;
  a.m = s.n;
  a.n = s.k;
  a.tn = tn;
  a.out = dW;
  a.ld = s.k;
  a.out_stride = static_cast<int64_t>(s.n) * s.k;
  a.status = static_cast<int32_t*>(ws);
  const int epi = add ? kMmAddF32 : (f32_out ? kMmStoreF32 : kMmStoreBf16);
  const int64_t tiles = bands * ((s.k + a.tn - 1) / a.tn);
  return launch_mm(kMmTN, kMmRaggedK, epi, ma, mb, a, pairs_for(tiles, sms), st);
}

int moe_swiglu(const moe_swiglu_shape_t* shape, const void* gu, void* a, moe_stream_t stream) {
  if (int rc = validate(shape)) return rc;
  if (shape->rows == 0) return MOE_OK;
  if (any_null(gu, static_cast<const void*>(a))) return MOE_ERR_NULLPTR;
  if (any_misaligned(gu, static_cast<const void*>(a))) return MOE_ERR_ALIGN;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  StageScope sg(MOE_KERNEL_SWIGLU, st);
  return launch_swiglu(shape->dtype, gu, shape->rows, shape->inter, a, st);
}

int moe_swiglu_backward(const moe_swiglu_shape_t* shape, const void* gu, const void* da, void* dgu,
                        moe_stream_t stream) {
  if (int rc = validate(shape)) return rc;
  if (shape->rows == 0) return MOE_OK;
  if (any_null(gu, da, static_cast<const void*>(dgu))) return MOE_ERR_NULLPTR;
  if (any_misaligned(gu, da, static_cast<const void*>(dgu))) return MOE_ERR_ALIGN;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  StageScope sg(MOE_KERNEL_SWIGLU_BACKWARD, st);
  return launch_swiglu_backward(shape->dtype, gu, da, shape->rows, shape->inter, dgu, st);
}

int moe_layer_norm(const moe_norm_shape_t* shape, const void* x, const float* gamma,
                   const float* beta, void* y, float* mean, float* rstd, moe_stream_t stream) {
  if (int rc = validate(shape)) return rc;
  if (shape->T == 0) return MOE_OK;
  if (!x || !gamma || !y) return MOE_ERR_NULLPTR;
  if (misaligned(x) || misaligned(gamma) || misaligned(y) || (beta && misaligned(beta)) ||
      (mean && misaligned(mean)) || (rstd && misaligned(rstd)))
    return MOE_ERR_ALIGN;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  StageScope sg(MOE_KERNEL_LAYER_NORM, st);
  return launch_layer_norm(shape->dtype, x, gamma, beta, shape->T, shape->d, shape->eps, y, mean,
                           rstd, sms, st);
}

int moe_layer_norm_workspace_size(const moe_norm_shape_t* shape, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULLPTR;
  if (int rc = validate(shape)) return rc;
  // two fp32 partial rows per block of the backward pass
  const int64_t parts = norm_partial_rows(shape->dtype, shape->T, shape->d, kNormMaxSms);
  *bytes = (static_cast<size_t>(2 * parts) * shape->d * 4 + 255) / 256 * 256;
  return MOE_OK;
}

int moe_layer_norm_backward(const moe_norm_shape_t* shape, const void* dy, const void* x,
                            const float* gamma, const float* mean, const float* rstd, void* dx,
                            float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                            moe_stream_t stream) {
  if (int rc = validate(shape)) return rc;
  if (!dgamma) return MOE_ERR_NULLPTR;
  if (misaligned(dgamma) || (dbeta && misaligned(dbeta))) return MOE_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int sms = 0;
  if (shape->T == 0) {
    if (int rc = require_device(&sms)) return rc;
    StageScope sg(MOE_KERNEL_LAYER_NORM_BACKWARD, st);
    const size_t bytes = static_cast<size_t>(shape->d) * 4;
    if (int rc = launch_zero(dgamma, bytes, st)) return rc;
    return dbeta ? launch_zero(dbeta, bytes, st) : MOE_OK;
  }
  if (!dy || !x || !gamma || !mean || !rstd || !dx || !ws) return MOE_ERR_NULLPTR;
  if (misaligned(dy) || misaligned(x) || misaligned(gamma) || misaligned(mean) ||
      misaligned(rstd) || misaligned(dx) || misaligned(ws))
    return MOE_ERR_ALIGN;
  size_t need = 0;
  if (int rc = moe_layer_norm_workspace_size(shape, &need)) return rc;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  if (int rc = require_device(&sms)) return rc;
  StageScope sg(MOE_KERNEL_LAYER_NORM_BACKWARD, st);
  const int parts = norm_partial_rows(shape->dtype, shape->T, shape->d,
                                      sms < kNormMaxSms ? sms : kNormMaxSms);
  return launch_layer_norm_backward(shape->dtype, dy, x, gamma, mean, rstd, shape->T, shape->d, dx,
                                    dgamma, dbeta, static_cast<float*>(ws), parts, st);
}

int moe_orthogonalize_workspace_size(const moe_ortho_shape_t* shape, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULLPTR;
  if (int rc = validate(shape)) return rc;
  *bytes = ortho_layout(shape->n_mats, shape->rows, shape->cols).total;
  return MOE_OK;
}

int moe_orthogonalize(const moe_ortho_shape_t* shape, const float* coef, const void* M, void* O,
                      void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (int rc = validate(shape)) return rc;
  const moe_ortho_shape_t& s = *shape;
  if (s.n_mats == 0) return MOE_OK;
  if (any_null(M, static_cast<const void*>(O), static_cast<const void*>(ws))) return MOE_ERR_NULLPTR;
  if (any_misaligned(M, static_cast<const void*>(O), static_cast<const void*>(ws)))
    return MOE_ERR_ALIGN;
  if (ws_bytes < ortho_layout(s.n_mats, s.rows, s.cols).total) return MOE_ERR_WORKSPACE;
  float c[3 * 16];
  for (int i = 0; i < s.steps; ++i) {
    c[3 * i] = coef ? coef[3 * i] : 3.4445f;
    c[3 * i + 1] = coef ? coef[3 * i + 1] : -4.7750f;
    c[3 * i + 2] = coef ? coef[3 * i + 2] : 2.0315f;
  }
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  StageScope sg(MOE_KERNEL_ORTHOGONALIZE, st);
  return launch_orthogonalize(s.dtype, M, O, s.n_mats, s.rows, s.cols, s.steps, c, ws, sms, st);
}

}  // extern "C"
