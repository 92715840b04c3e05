// Layer norm over the model width, forward and backward, in fp32:
//
//   mu = mean x, s = 1 / sqrt(mean (x - mu)^2 + eps), h = (x - mu) s
//   y  = h gamma + beta
//   dx = s (v - mean v - h mean(v h)), v = dy gamma
//   dgamma = sum_t dy h,  dbeta = sum_t dy
//
// Bound by memory.  A row is read once and held in registers: a group of
// 32..512 threads per row, kVals values each, so that the variance is taken
// about the mean (a second pass over registers) rather than as a difference of
// sums.  The backward pass runs a fixed set of blocks over all rows; a thread
// keeps the same columns for every row and carries their dgamma and dbeta sums
// in registers, written once per block and added up in a fixed order by a
// second kernel (no atomics: the same bits every run).  Rows too wide for the
// registers take kernels that read them more than once.
#include <cuda_runtime.h>

#include "common.cuh"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr int kMaxGroup = 512;  // threads per row

template <typename T> struct NormCfg;
template <> struct NormCfg<bf16> { static constexpr int kVals = 16; };
template <> struct NormCfg<float> { static constexpr int kVals = 8; };

// A thread's kVals values of a row: 16-byte pieces t, t + TPR, ... (VEC) or
// single elements t, t + TPR, ...; those past the row are 0.
template <typename T, bool VEC>
struct RowSlice {
  static constexpr int V = NormCfg<T>::kVals;
  static constexpr int N = Vec16<T>::N;
  static constexpr int P = V / N;

  // column of value i
  __device__ __forceinline__ static int col(int i, int t, int tpr) {
    return VEC ? (t + (i / N) * tpr) * N + i % N : t + i * tpr;
  }
  template <typename S>
  __device__ __forceinline__ static void load_f32(const S* p, int d, int t, int tpr, float fill,
                                                  float* v) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = col(i, t, tpr);
      v[i] = c < d ? to_f32(p[c]) : fill;
    }
  }
  __device__ __forceinline__ static void load(const T* p, int d, int t, int tpr, float* v) {
    if (VEC) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int c = (t + i * tpr) * N;
        if (c < d) {
          Vec16<T>::load(p + c, v + i * N);
        } else {
#pragma unroll
          for (int j = 0; j < N; ++j) v[i * N + j] = 0.0f;
        }
      }
    } else {
      load_f32(p, d, t, tpr, 0.0f, v);
    }
  }
  __device__ __forceinline__ static void store(T* p, int d, int t, int tpr, const float* v) {
    if (VEC) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int c = (t + i * tpr) * N;
        if (c < d) Vec16<T>::store(p + c, v + i * N);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = col(i, t, tpr);
        if (c < d) p[c] = from_f32<T>(v[i]);
      }
    }
  }
};

// Sum over the group of TPR threads that holds this thread (every thread of
// the block calls it; `red` is used by no other call until a block barrier).
template <int TPR>
__device__ __forceinline__ float group_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    const int w0 = warp / W * W;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += red[w0 + i];
  }
  return v;
}

template <int TPR> constexpr int block_of() { return TPR > 256 ? TPR : 256; }

template <typename T, bool VEC, int TPR>
__global__ void __launch_bounds__(block_of<TPR>())
norm_fwd_kernel(const T* x, const float* __restrict__ gamma,
                const float* __restrict__ beta, int64_t rows, int d, float eps,
                T* y, float* __restrict__ mean, float* __restrict__ rstd) {
  using S = RowSlice<T, VEC>;
  constexpr int V = S::V;
  constexpr int RG = block_of<TPR>() / TPR;
  __shared__ float red[2][block_of<TPR>() / 32];
  pdl_wait();
  pdl_trigger();
  const int t = threadIdx.x % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * RG + threadIdx.x / TPR;
  const bool live = row < rows;
  float v[V];
  if (live) {
    S::load(x + row * d, d, t, TPR, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) s += v[i];
  const float mu = group_sum<TPR>(s, red[0]) / d;
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = S::col(i, t, TPR) < d ? v[i] - mu : 0.0f;
    q += v[i] * v[i];
  }
  const float rs = 1.0f / sqrtf(group_sum<TPR>(q, red[1]) / d + eps);
  if (!live) return;
  float g[V];
  S::load_f32(gamma, d, t, TPR, 0.0f, g);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = v[i] * rs * g[i];
  if (beta != nullptr) {
    S::load_f32(beta, d, t, TPR, 0.0f, g);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += g[i];
  }
  S::store(y + row * d, d, t, TPR, v);
  if (t == 0) {
    if (mean != nullptr) mean[row] = mu;
    if (rstd != nullptr) rstd[row] = rs;
  }
}

// Rows that the registers do not hold: three reads of x.
template <typename T>
__global__ void __launch_bounds__(512)
norm_fwd_wide_kernel(const T* x, const float* __restrict__ gamma,
                     const float* __restrict__ beta, int d, float eps, T* y,
                     float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float red[2][16];
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const T* p = x + row * d;
  float s = 0.0f;
  for (int c = threadIdx.x; c < d; c += 512) s += to_f32(p[c]);
  const float mu = group_sum<512>(s, red[0]) / d;
  float q = 0.0f;
  for (int c = threadIdx.x; c < d; c += 512) {
    const float h = to_f32(p[c]) - mu;
    q += h * h;
  }
  const float rs = 1.0f / sqrtf(group_sum<512>(q, red[1]) / d + eps);
  for (int c = threadIdx.x; c < d; c += 512) {
    const float h = (to_f32(p[c]) - mu) * rs * gamma[c];
    y[row * d + c] = from_f32<T>(beta != nullptr ? h + beta[c] : h);
  }
  if (threadIdx.x == 0) {
    if (mean != nullptr) mean[row] = mu;
    if (rstd != nullptr) rstd[row] = rs;
  }
}

template <typename T, bool VEC, int TPR>
__global__ void __launch_bounds__(block_of<TPR>(), TPR > 256 ? 1 : 2)
norm_bwd_kernel(const T* dy, const T* __restrict__ x, const float* __restrict__ gamma,
                const float* __restrict__ mean, const float* __restrict__ rstd, int64_t rows,
                int d, T* dx, float* __restrict__ part) {
  using S = RowSlice<T, VEC>;
  constexpr int V = S::V;
  constexpr int B = block_of<TPR>();
  constexpr int RG = B / TPR;
  __shared__ float red[2][2][B / 32];
  __shared__ float acc[RG > 1 ? B * V : 1];
  pdl_wait();
  pdl_trigger();
  const int t = threadIdx.x % TPR;
  const int grp = threadIdx.x / TPR;
  float g[V], dg[V], db[V];
  S::load_f32(gamma, d, t, TPR, 0.0f, g);
#pragma unroll
  for (int i = 0; i < V; ++i) dg[i] = db[i] = 0.0f;
  const float inv_d = 1.0f / d;
  int buf = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * RG; base < rows;
       base += static_cast<int64_t>(gridDim.x) * RG, buf ^= 1) {
    const int64_t row = base + grp;
    const bool live = row < rows;
    float h[V], v[V];
    float rs = 0.0f;
    if (live) {
      S::load(x + row * d, d, t, TPR, h);
      S::load(dy + row * d, d, t, TPR, v);
      const float mu = mean[row];
      rs = rstd[row];
#pragma unroll
      for (int i = 0; i < V; ++i) h[i] = (h[i] - mu) * rs;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) h[i] = v[i] = 0.0f;
    }
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      // past the row dy and gamma are 0, and h is not used
      dg[i] += v[i] * h[i];
      db[i] += v[i];
      v[i] *= g[i];
      s1 += v[i];
      s2 += v[i] * h[i];
    }
    // one barrier for both sums: the next row's use of this buffer is behind
    // the barrier of the row between
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, o);
      s2 += __shfl_xor_sync(0xffffffffu, s2, o);
    }
    if (TPR > 32) {
      constexpr int W = TPR / 32;
      const int warp = threadIdx.x >> 5;
      if ((threadIdx.x & 31) == 0) {
        red[buf][0][warp] = s1;
        red[buf][1][warp] = s2;
      }
      __syncthreads();
      const int w0 = warp / W * W;
      s1 = s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        s1 += red[buf][0][w0 + i];
        s2 += red[buf][1][w0 + i];
      }
    }
    s1 *= inv_d;
    s2 *= inv_d;
    if (live) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = rs * (v[i] - s1 - h[i] * s2);
      S::store(dx + row * d, d, t, TPR, v);
    }
  }
  // this block's sums: part[0] dgamma, part[1] dbeta, [gridDim.x, d] each
  float* pg = part + static_cast<int64_t>(blockIdx.x) * d;
  float* pb = part + (static_cast<int64_t>(gridDim.x) + blockIdx.x) * d;
  if (RG == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = S::col(i, t, TPR);
      if (c < d) {
        pg[c] = dg[i];
        pb[c] = db[i];
      }
    }
  } else {
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = S::col(i, t, TPR);
        if (c < d) acc[grp * TPR * V + c] = pass ? db[i] : dg[i];
      }
      __syncthreads();
      for (int c = threadIdx.x; c < d; c += B) {
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < RG; ++r) s += acc[r * TPR * V + c];
        (pass ? pb : pg)[c] = s;
      }
    }
  }
}

// Wide rows: dx in one kernel (two reads of x and dy; dx may be dy) ...
template <typename T>
__global__ void __launch_bounds__(512)
norm_bwd_wide_kernel(const T* dy, const T* __restrict__ x,
                     const float* __restrict__ gamma, const float* __restrict__ mean,
                     const float* __restrict__ rstd, int d, T* dx) {
  __shared__ float red[2][16];
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const float mu = mean[row], rs = rstd[row];
  float s1 = 0.0f, s2 = 0.0f;
  for (int c = threadIdx.x; c < d; c += 512) {
    const float v = to_f32(dy[row * d + c]) * gamma[c];
    s1 += v;
    s2 += v * ((to_f32(x[row * d + c]) - mu) * rs);
  }
  s1 = group_sum<512>(s1, red[0]) / d;
  s2 = group_sum<512>(s2, red[1]) / d;
  for (int c = threadIdx.x; c < d; c += 512) {
    const float v = to_f32(dy[row * d + c]) * gamma[c];
    const float h = (to_f32(x[row * d + c]) - mu) * rs;
    dx[row * d + c] = from_f32<T>(rs * (v - s1 - h * s2));
  }
}

// ... and the column sums in another, a thread per column and slice of rows.
template <typename T>
__global__ void __launch_bounds__(256)
norm_bwd_cols_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                     const float* __restrict__ mean, const float* __restrict__ rstd, int64_t rows,
                     int d, float* __restrict__ part) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= d) return;
  float g = 0.0f, b = 0.0f;
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const float v = to_f32(dy[row * d + c]);
    g += v * ((to_f32(x[row * d + c]) - mean[row]) * rstd[row]);
    b += v;
  }
  part[static_cast<int64_t>(blockIdx.y) * d + c] = g;
  part[(static_cast<int64_t>(gridDim.y) + blockIdx.y) * d + c] = b;
}

// dgamma, dbeta = column sums of the blocks' partial rows, 32 columns by 8
// slices of the rows per block, added in a fixed order.
__global__ void __launch_bounds__(256)
norm_bwd_reduce_kernel(const float* __restrict__ part, int part_rows, int d,
                       float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float red[8][33];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float* p = part + static_cast<int64_t>(blockIdx.y) * part_rows * d;
  float s = 0.0f;
  if (c < d)
    for (int r = slice; r < part_rows; r += 8) s += p[static_cast<int64_t>(r) * d + c];
  red[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < d) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][lane];
    float* out = blockIdx.y ? dbeta : dgamma;
    if (out != nullptr) out[c] = s;
  }
}

// threads per row that hold d values, or 0 (too wide)
template <typename T>
int group_of(int d) {
  for (int tpr = 32; tpr <= kMaxGroup; tpr *= 2)
    if (d <= tpr * NormCfg<T>::kVals) return tpr;
  return 0;
}

template <typename T>
int part_rows_of(int64_t T_, int d, int sms) {
  const int tpr = group_of<T>(d);
  if (tpr == 0) return static_cast<int>(T_ < 64 ? T_ : 64);
  const int rg = tpr > 256 ? 1 : 256 / tpr;
  const int64_t blocks = (T_ + rg - 1) / rg;
  const int64_t most = static_cast<int64_t>(sms) * (tpr > 256 ? 1 : 2);
  return static_cast<int>(blocks < most ? blocks : most);
}

template <typename T, bool VEC, int TPR>
int fwd_impl(const T* x, const float* gamma, const float* beta, int64_t rows, int d, float eps,
             T* y, float* mean, float* rstd, cudaStream_t st) {
  constexpr int RG = block_of<TPR>() / TPR;
  return launch_k(norm_fwd_kernel<T, VEC, TPR>, dim3(static_cast<unsigned>((rows + RG - 1) / RG)),
                  dim3(block_of<TPR>()), 0, st, 1, x, gamma, beta, rows, d, eps, y, mean, rstd);
}

template <typename T, bool VEC>
int fwd_group(const T* x, const float* gamma, const float* beta, int64_t rows, int d, float eps,
              T* y, float* mean, float* rstd, cudaStream_t st) {
  switch (group_of<T>(d)) {
    case 32: return fwd_impl<T, VEC, 32>(x, gamma, beta, rows, d, eps, y, mean, rstd, st);
    case 64: return fwd_impl<T, VEC, 64>(x, gamma, beta, rows, d, eps, y, mean, rstd, st);
    case 128: return fwd_impl<T, VEC, 128>(x, gamma, beta, rows, d, eps, y, mean, rstd, st);
    case 256: return fwd_impl<T, VEC, 256>(x, gamma, beta, rows, d, eps, y, mean, rstd, st);
    case 512: return fwd_impl<T, VEC, 512>(x, gamma, beta, rows, d, eps, y, mean, rstd, st);
  }
  return launch_k(norm_fwd_wide_kernel<T>, dim3(static_cast<unsigned>(rows)), dim3(512), 0, st, 1,
                  x, gamma, beta, d, eps, y, mean, rstd);
}

template <typename T>
int fwd_typed(const void* x, const float* gamma, const float* beta, int64_t rows, int d, float eps,
              void* y, float* mean, float* rstd, cudaStream_t st) {
  const T* xt = static_cast<const T*>(x);
  T* yt = static_cast<T*>(y);
  return d % Vec16<T>::N == 0 ? fwd_group<T, true>(xt, gamma, beta, rows, d, eps, yt, mean, rstd, st)
                              : fwd_group<T, false>(xt, gamma, beta, rows, d, eps, yt, mean, rstd, st);
}

template <typename T, bool VEC, int TPR>
int bwd_impl(const T* dy, const T* x, const float* gamma, const float* mean, const float* rstd,
             int64_t rows, int d, T* dx, float* part, int part_rows, cudaStream_t st) {
  return launch_k(norm_bwd_kernel<T, VEC, TPR>, dim3(part_rows), dim3(block_of<TPR>()), 0, st, 1,
                  dy, x, gamma, mean, rstd, rows, d, dx, part);
}

template <typename T, bool VEC>
int bwd_group(const T* dy, const T* x, const float* gamma, const float* mean, const float* rstd,
              int64_t rows, int d, T* dx, float* part, int part_rows, cudaStream_t st) {
  switch (group_of<T>(d)) {
    case 32: return bwd_impl<T, VEC, 32>(dy, x, gamma, mean, rstd, rows, d, dx, part, part_rows, st);
    case 64: return bwd_impl<T, VEC, 64>(dy, x, gamma, mean, rstd, rows, d, dx, part, part_rows, st);
    case 128: return bwd_impl<T, VEC, 128>(dy, x, gamma, mean, rstd, rows, d, dx, part, part_rows, st);
    case 256: return bwd_impl<T, VEC, 256>(dy, x, gamma, mean, rstd, rows, d, dx, part, part_rows, st);
    case 512: return bwd_impl<T, VEC, 512>(dy, x, gamma, mean, rstd, rows, d, dx, part, part_rows, st);
  }
  // the column sums first: dx may be dy
  if (int rc = launch_k(norm_bwd_cols_kernel<T>, dim3((d + 255) / 256, part_rows), dim3(256), 0, st,
                        1, dy, x, mean, rstd, rows, d, part))
    return rc;
  return launch_k(norm_bwd_wide_kernel<T>, dim3(static_cast<unsigned>(rows)), dim3(512), 0, st, 1,
                  dy, x, gamma, mean, rstd, d, dx);
}

template <typename T>
int bwd_typed(const void* dy, const void* x, const float* gamma, const float* mean,
              const float* rstd, int64_t rows, int d, void* dx, float* part, int part_rows,
              cudaStream_t st) {
  const T *dt = static_cast<const T*>(dy), *xt = static_cast<const T*>(x);
  T* o = static_cast<T*>(dx);
  return d % Vec16<T>::N == 0
             ? bwd_group<T, true>(dt, xt, gamma, mean, rstd, rows, d, o, part, part_rows, st)
             : bwd_group<T, false>(dt, xt, gamma, mean, rstd, rows, d, o, part, part_rows, st);
}

}  // namespace

int launch_layer_norm(int dtype, const void* x, const float* gamma, const float* beta, int64_t T,
                      int d, float eps, void* y, float* mean, float* rstd, cudaStream_t st) {
  return dtype == MOE_DTYPE_BF16
             ? fwd_typed<bf16>(x, gamma, beta, T, d, eps, y, mean, rstd, st)
             : fwd_typed<float>(x, gamma, beta, T, d, eps, y, mean, rstd, st);
}

int norm_partial_rows(int dtype, int64_t T, int d, int sms) {
  return dtype == MOE_DTYPE_BF16 ? part_rows_of<bf16>(T, d, sms) : part_rows_of<float>(T, d, sms);
}

int launch_layer_norm_backward(int dtype, const void* dy, const void* x, const float* gamma,
                               const float* mean, const float* rstd, int64_t T, int d, void* dx,
                               float* dgamma, float* dbeta, float* part, int part_rows,
                               cudaStream_t st) {
  const int rc = dtype == MOE_DTYPE_BF16
                     ? bwd_typed<bf16>(dy, x, gamma, mean, rstd, T, d, dx, part, part_rows, st)
                     : bwd_typed<float>(dy, x, gamma, mean, rstd, T, d, dx, part, part_rows, st);
  if (rc) return rc;
  return launch_k(norm_bwd_reduce_kernel, dim3((d + 31) / 32, dbeta != nullptr ? 2 : 1), dim3(256),
                  0, st, 1, static_cast<const float*>(part), part_rows, d, dgamma, dbeta);
}

}  // namespace moe
