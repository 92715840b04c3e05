// SwiGLU on packed gate/up columns and its gradient.  A row holds, for every
// block of 64 intermediate columns, 64 gate values and then the 64 up values
// (the row order of moe_pack_w13, which the gate/up product leaves in the
// columns).
//
//   a  = g s u,  s = 1 / (1 + e^-g)
//   dg = da u s (1 + g (1 - s)),  du = da g s
//
// Bound by memory: 3 (5) values per output element, each moved once in
// 16-byte pieces; arithmetic in fp32, one rounding on the store.  bf16, 57344 x
// 896: 50 us, 6.1 TB/s (0.94 of a copy's rate); backward, 98304 x 1408: 197 us,
// 7.0 TB/s (what L2 still holds of the last call's output need not be written).
// A thread does one piece of each operand, so that a grid of many blocks keeps
// enough loads in flight; a loop over a resident grid was no faster.
#include <cuda_runtime.h>

#include "common.cuh"
#include "train_kernels.h"

namespace moe {

namespace {

// bf16 results: ex2.approx and rcp.approx, a few fp32 ulp, far below the
// store's rounding.  Below g = -87.3, where s would be subnormal, and where e^-g
// overflows it is 0, off by 2^-126 at most.
__device__ __forceinline__ float sigmoid_of(float g, bf16) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}
__device__ __forceinline__ float sigmoid_of(float g, float) { return 1.0f / (1.0f + expf(-g)); }

template <typename T, bool BWD>
__global__ void __launch_bounds__(256)
swiglu_kernel(const T* gu, const T* __restrict__ da, int64_t pieces, int per_row,
              T* out) {  // the gradient may overwrite gu
  constexpr int N = Vec16<T>::N;
  constexpr int PB = 64 / N;  // pieces per block of 64
  pdl_wait();
  pdl_trigger();
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t p = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; p < pieces; p += step) {
    const int64_t row = p / per_row;
    const int c = static_cast<int>(p - row * per_row);
    const int64_t at = (row * per_row * 2 + (c / PB) * 2 * PB + c % PB) * N;
    float g[N], u[N], x[N];
    Vec16<T>::load(gu + at, g);
    Vec16<T>::load(gu + at + 64, u);
    if (!BWD) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = g[i] * sigmoid_of(g[i], T()) * u[i];
      Vec16<T>::store(out + p * N, x);
    } else {
      Vec16<T>::load(da + p * N, x);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float s = sigmoid_of(g[i], T());
        const float dg = x[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
        u[i] = x[i] * g[i] * s;
        g[i] = dg;
      }
      Vec16<T>::store(out + at, g);
      Vec16<T>::store(out + at + 64, u);
    }
  }
}

template <typename T, bool BWD>
int launch_impl(const void* gu, const void* da, int64_t rows, int inter, void* out,
                cudaStream_t st) {
  const int per_row = inter / Vec16<T>::N;
  const int64_t pieces = rows * per_row;
  const int64_t blocks = (pieces + 255) / 256;
  const int grid = static_cast<int>(blocks < (1 << 20) ? blocks : (1 << 20));
  return launch_k(swiglu_kernel<T, BWD>, dim3(grid), dim3(256), 0, st, 1,
                  static_cast<const T*>(gu), static_cast<const T*>(da), pieces, per_row,
                  static_cast<T*>(out));
}

}  // namespace

int launch_swiglu(int dtype, const void* gu, int64_t rows, int inter, void* a, cudaStream_t st) {
  return dtype == MOE_DTYPE_BF16 ? launch_impl<bf16, false>(gu, nullptr, rows, inter, a, st)
                                 : launch_impl<float, false>(gu, nullptr, rows, inter, a, st);
}

int launch_swiglu_backward(int dtype, const void* gu, const void* da, int64_t rows, int inter,
                           void* dgu, cudaStream_t st) {
  return dtype == MOE_DTYPE_BF16 ? launch_impl<bf16, true>(gu, da, rows, inter, dgu, st)
                                 : launch_impl<float, true>(gu, da, rows, inter, dgu, st);
}

}  // namespace moe
