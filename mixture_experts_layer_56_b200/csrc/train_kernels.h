// Launch wrappers of the training operators' kernels (host interface).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// MOE_OK and the SM count if the current device is a B200 (api.cu)
int require_device(int* sms);

// fp32 grouped products on CUDA cores (grouped_f32.cu)
enum GroupedDir { kGroupedFwd = 0, kGroupedDx = 1, kGroupedDw = 2 };
int launch_grouped_f32(int dir, const float* a, const float* b, const int32_t* offsets, int groups,
                       int64_t rows, int n, int k, float* out, bool accumulate, int sms,
                       cudaStream_t st);

// layer norm (norm.cu)
int launch_layer_norm(int dtype, const void* x, const float* gamma, const float* beta, int64_t T,
                      int d, float eps, void* y, float* mean, float* rstd, int sms,
                      cudaStream_t st);
// SMs that a backward pass's workspace is sized for, so that its size needs no
// device (148 on a B200)
constexpr int kNormMaxSms = 160;
// rows of each of the two fp32 [rows, d] partial buffers of the backward pass
int norm_partial_rows(int dtype, int64_t T, int d, int sms);
int launch_layer_norm_backward(int dtype, const void* dy, const void* x, const float* gamma,
                               const float* mean, const float* rstd, int64_t T, int d, void* dx,
                               float* dgamma, float* dbeta, float* part, int part_rows,
                               cudaStream_t st);

// SwiGLU on packed gate/up columns (swiglu.cu)
int launch_swiglu(int dtype, const void* gu, int64_t rows, int inter, void* a, cudaStream_t st);
int launch_swiglu_backward(int dtype, const void* gu, const void* da, int64_t rows, int inter,
                           void* dgu, cudaStream_t st);

// Newton-Schulz (ortho.cu)
struct OrthoLayout {
  size_t status, partial, hi0, hi1, lo, gram, poly, dgram, dpoly, total;
  int parts;          // partial sums of squares per matrix
  int64_t ldx, ldm;   // row pitches of X and of the m x m matrices, elements
  int m;              // min(rows, cols)
};
OrthoLayout ortho_layout(int mats, int rows, int cols);
// small matrices: one kernel, no workspace but the status word (ortho_small.cu)
bool ortho_small_fits(int rows, int cols);
int launch_ortho_small(int dtype, const void* M, void* O, int mats, int rows, int cols, int steps,
                       const float* coef, float scale, int32_t* status, cudaStream_t st);
int launch_orthogonalize(int dtype, const void* M, void* O, int mats, int rows, int cols, int steps,
                         const float* coef, void* ws, int sms, cudaStream_t st);

}  // namespace moe
