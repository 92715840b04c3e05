// Layer norm over the model width, forward and backward, in fp32:
//
//   mu = mean x, s = 1 / sqrt(mean (x - mu)^2 + eps), h = (x - mu) s
//   y  = h gamma + beta
//   dx = s (v - mean v - h mean(v h)), v = dy gamma
//   dgamma = sum_t dy h,  dbeta = sum_t dy
//
// Bound by memory: 32768 x 4096 bf16 forward 88 to 97 us (5.5 to 6.1 TB/s, 0.85 to
// 0.93 of the measured copy rate), backward 143 to 148 us (5.5 TB/s, 0.84).
//
// A row is read once and held in registers: a group of 32 to 512 threads per
// row, kVals values each, so that the variance is taken about the mean (a second
// pass over registers) rather than as a difference of sums.  A fixed set of
// blocks takes the rows in turn, the next two rows on their way from memory
// while one is worked on (one block per row, without that, took 345 us forward).
// In the backward pass a thread keeps the same columns for every row and carries
// their dgamma and dbeta sums in registers, written once per block and added up
// in a fixed order by a second kernel (no atomics: the same bits every run).
// Rows too wide for the registers take kernels that read them more than once.
#include <cuda_runtime.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "train_kernels.h"

namespace moe {

namespace {

template <typename T> struct NormCfg;
template <> struct NormCfg<bf16> { static constexpr int kVals = 16; };
template <> struct NormCfg<float> { static constexpr int kVals = 8; };

// Arithmetic is done on pairs: these kernels have as many instructions as the
// memory leaves time for.
__device__ __forceinline__ float sum_of(F2 v) {
  const float2 f = both(v);
  return f.x + f.y;
}

// A 16-byte piece as pairs.
__device__ __forceinline__ void piece_pairs(const uint4& w, F2* v, bf16) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = pair(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}
__device__ __forceinline__ void piece_pairs(const uint4& w, F2* v, float) {
  v[0] = pair(__uint_as_float(w.x), __uint_as_float(w.y));
  v[1] = pair(__uint_as_float(w.z), __uint_as_float(w.w));
}
__device__ __forceinline__ uint4 pairs_piece(const F2* v, bf16) {
  uint4 w;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = both(v[i]);
    h[i] = __floats2bfloat162_rn(f.x, f.y);
  }
  return w;
}
__device__ __forceinline__ uint4 pairs_piece(const F2* v, float) {
  const float2 a = both(v[0]), b = both(v[1]);
  return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                    __float_as_uint(b.y));
}

// A thread's kVals values of a row, as kVals / 2 pairs: 16-byte pieces t,
// t + TPR, ... (VEC) or single elements t, t + TPR, ...; those past the row
// are 0.
template <typename T, bool VEC>
struct RowSlice {
  static constexpr int V = NormCfg<T>::kVals;
  static constexpr int N = Vec16<T>::N;
  static constexpr int P = V / N;
  static constexpr int PP = N / 2;  // pairs of a piece

  // column of value i
  __device__ __forceinline__ static int col(int i, int t, int tpr) {
    return VEC ? (t + (i / N) * tpr) * N + i % N : t + i * tpr;
  }
  // fp32 parameters
  __device__ __forceinline__ static void load_f32(const float* p, int d, int t, int tpr, F2* v) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      float f[4] = {};
      const int c = col(i, t, tpr);
      if (VEC) {
        if (c < d) Vec16<float>::load(p + c, f);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c + j * tpr < d) f[j] = p[c + j * tpr];
      }
      v[i / 2] = pair(f[0], f[1]);
      v[i / 2 + 1] = pair(f[2], f[3]);
    }
  }
  __device__ __forceinline__ static void load(const T* p, int d, int t, int tpr, F2* v) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const int c = col(i, t, tpr), e = col(i + 1, t, tpr);
      v[i / 2] = pair(c < d ? to_f32(p[c]) : 0.0f, e < d ? to_f32(p[e]) : 0.0f);
    }
  }
  __device__ __forceinline__ static void store(T* p, int d, int t, int tpr, const F2* v) {
    if (VEC) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int c = (t + i * tpr) * N;
        if (c < d) *reinterpret_cast<uint4*>(p + c) = pairs_piece(v + i * PP, T());
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const int c = col(i, t, tpr), e = col(i + 1, t, tpr);
        const float2 f = both(v[i / 2]);
        if (c < d) p[c] = from_f32<T>(f.x);
        if (e < d) p[e] = from_f32<T>(f.y);
      }
    }
  }
  // zeroes the values past the row
  __device__ __forceinline__ static void clip(int d, int t, int tpr, F2* v) {
    if (VEC) {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if ((t + i * tpr) * N >= d) {
#pragma unroll
          for (int j = 0; j < PP; ++j) v[i * PP + j] = 0;
        }
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 f = both(v[i / 2]);
        v[i / 2] = pair(col(i, t, tpr) < d ? f.x : 0.0f, col(i + 1, t, tpr) < d ? f.y : 0.0f);
      }
    }
  }
  // how many values lie in the row
  __device__ __forceinline__ static int count(int d, int t, int tpr) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) n += col(i, t, tpr) < d;
    return n;
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the first W lanes (the others hold 0), in every lane.
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
  constexpr int P = W > 8 ? 16 : W > 4 ? 8 : W > 2 ? 4 : 2;
#pragma unroll
  for (int o = P / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return __shfl_sync(0xffffffffu, v, 0);
}

// Sum over a block of 512 threads (`red` is used by no other call until a
// block barrier).
__device__ __forceinline__ float block_sum512(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) v += red[i];
  return v;
}

constexpr int block_threads(int tpr) { return tpr > 256 ? tpr : 256 / tpr * tpr; }
template <int TPR> constexpr int block_of() { return block_threads(TPR); }
// Threads of a block: whole groups, about 256; and blocks per SM in the forward
// and the backward kernel: what the registers allow, or fewer where more were
// slower.  bf16 forward, 65536 x 1536: 87 us with four blocks, 78 with three;
// 32768 x 2048: 57 with three, 53 with two; x 4096: 88 with three, 101 with two.
// fp32, whose threads hold half the values: 32768 x 1000 forward 56 us with two
// blocks, 45 with three, backward 69 and 63.
constexpr int at_least_1(int v) { return v > 1 ? v : 1; }
template <typename T> constexpr int fwd_blocks(int tpr) {
  const bool few = sizeof(T) == 2 && tpr >= 64 && tpr <= 128;
  return at_least_1((!few ? 768 : tpr == 96 ? 576 : 512) / block_threads(tpr));
}
template <typename T> constexpr int bwd_blocks(int tpr) {
  return at_least_1((sizeof(T) == 2 ? 512 : tpr == 96 ? 576 : 768) / block_threads(tpr));
}
// Barrier of a row's group of TPR threads, whole warps, in its block.
template <int TPR>
__device__ __forceinline__ void group_sync() {
  if (block_of<TPR>() == TPR) __syncthreads();
  else {
    __syncwarp();  // the barrier takes whole warps
    asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.x / TPR), "n"(TPR) : "memory");
  }
}

// Rows on their way from memory: kRing rows per group, of each of the ARRAYS
// that a pass reads, in shared memory, fetched with cp.async.  A thread whose
// values are whole 16-byte pieces or fp32 copies exactly those, so that its own
// wait_group is all the waiting there is.  Rows of bf16 that start anywhere in a
// piece: the group copies the pieces that the row touches, up to the tensor's
// end, and a thread finds its values behind a barrier (kShared; 8192 x 4099
// forward 54 us, 71 with each thread loading its own as it needs them), except
// where a row is a warp's, whose many rows in flight do the same for less
// (kDirect; 65536 x 131 backward 35 us for 45).  With two or eight values of
// such a row per access and their realignment in registers it takes longer, as
// these kernels are bound by their instructions.
constexpr int kRing = 3;

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
// the first `bytes` of the 16, zeros behind them
__device__ __forceinline__ void copy_async_first(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T, bool VEC, int TPR, int ARRAYS>
struct RowRing {
  using S = RowSlice<T, VEC>;
  static constexpr int B = block_of<TPR>();
  static constexpr bool kAnywhere = !VEC && sizeof(T) == 2;
  static constexpr bool kShared = kAnywhere && TPR > 32, kDirect = kAnywhere && TPR == 32;
  static constexpr int kRow = S::V * TPR * static_cast<int>(sizeof(T)) + (kShared ? 32 : 0);
  static constexpr int kBytes = kDirect ? 0 : kRing * ARRAYS * (B / TPR) * kRow;

  // a thread's 16-byte pieces (VEC) or single values, those of all threads side by side
  __device__ __forceinline__ static T* own(uint8_t* base, int stage, int which, int i) {
    constexpr int N = VEC ? S::N : 1;
    return reinterpret_cast<T*>(base) +
           (((stage * ARRAYS + which) * (S::V / N) + i) * B + threadIdx.x) * N;
  }
  // kShared: this group's row
  __device__ __forceinline__ static uint8_t* row(uint8_t* base, int stage, int which) {
    return base + ((stage * ARRAYS + which) * (B / TPR) + threadIdx.x / TPR) * kRow;
  }
  // the row at p of a tensor that ends at `end`
  __device__ __forceinline__ static void fetch(uint8_t* base, int stage, int which, const T* p,
                                               const T* end, int d, int t) {
    if (kDirect) return;
    if (VEC) {
#pragma unroll
      for (int i = 0; i < S::P; ++i) {
        const int c = (t + i * TPR) * S::N;
        if (c < d) copy_async16(own(base, stage, which, i), p + c);
      }
    } else if (kShared) {
      const int skip = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
      const uint8_t* from = reinterpret_cast<const uint8_t*>(p) - skip;
      const int64_t left = reinterpret_cast<const uint8_t*>(end) - from;
      const int bytes = skip + d * static_cast<int>(sizeof(T));
      uint8_t* to = row(base, stage, which);
#pragma unroll
      for (int i = 0; i <= S::P; ++i) {
        const int at = (t + i * TPR) * 16;
        if (at < bytes)
          copy_async_first(to + at, from + at, left - at < 16 ? static_cast<int>(left - at) : 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < S::V; ++i) {
        const int c = t + i * TPR;
        if (c < d) copy_async4(own(base, stage, which, i), p + c);
      }
    }
  }
  // a row's copies have landed, for every thread that takes from them
  __device__ __forceinline__ static void landed() {
    if (!kDirect) copy_wait<kRing - 1>();
    if (kShared) group_sync<TPR>();
  }
  __device__ __forceinline__ static void take(uint8_t* base, int stage, int which, const T* p, int d,
                                              int t, F2* v) {
    if (VEC) {
#pragma unroll
      for (int i = 0; i < S::P; ++i) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if ((t + i * TPR) * S::N < d)
          w = *reinterpret_cast<const uint4*>(own(base, stage, which, i));
        piece_pairs(w, v + i * S::PP, T());
      }
    } else if (kDirect || kShared) {
      const T* s = kDirect ? p
                           : reinterpret_cast<const T*>(row(base, stage, which) +
                                                        (reinterpret_cast<uintptr_t>(p) & 15));
      S::load(s, d, t, TPR, v);
    } else {
#pragma unroll
      for (int i = 0; i < S::V; i += 2)
        v[i / 2] = pair(t + i * TPR < d ? to_f32(*own(base, stage, which, i)) : 0.0f,
                        t + (i + 1) * TPR < d ? to_f32(*own(base, stage, which, i + 1)) : 0.0f);
    }
  }
};

template <typename T, bool VEC, int TPR>
__global__ void __launch_bounds__(block_of<TPR>(), fwd_blocks<T>(TPR))
norm_fwd_kernel(const T* x, const float* __restrict__ gamma, const float* __restrict__ beta,
                int64_t rows, int d, float eps, T* y, float* __restrict__ mean,
                float* __restrict__ rstd) {
  using S = RowSlice<T, VEC>;
  using R = RowRing<T, VEC, TPR, 1>;
  constexpr int H = S::V / 2;
  constexpr int RG = block_of<TPR>() / TPR;
  constexpr int W = TPR / 32;  // warps per row
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 red[2][block_of<TPR>() / 32];
  pdl_wait();
  pdl_trigger();
  const int t = threadIdx.x % TPR;
  const int grp = threadIdx.x / TPR;
  const int warp = threadIdx.x >> 5, w0 = warp / W * W;
  const int64_t step = static_cast<int64_t>(gridDim.x) * RG;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * RG + grp;
  auto fetch = [&](int64_t row, int stage) {
    if (row < rows) R::fetch(ring, stage, 0, x + row * d, x + rows * d, d, t);
    copy_commit();
  };
#pragma unroll
  for (int s = 0; s < kRing - 1; ++s) fetch(first + s * step, s);
  F2 g[H], b[H];
  S::load_f32(gamma, d, t, TPR, g);
#pragma unroll
  for (int i = 0; i < H; ++i) b[i] = 0;
  if (beta != nullptr) S::load_f32(beta, d, t, TPR, b);
  const float inv_d = 1.0f / d;
  // values of a row in this warp, and what turns their sum into their mean
  const float n_w = warp_sum(static_cast<float>(S::count(d, t, TPR)));
  const float inv_n = n_w > 0.0f ? 1.0f / n_w : 0.0f;
  const int lane = threadIdx.x & 31;
  float n_lane = 0.0f;  // and in the row's warp number `lane`
  if (W > 1) {
    if (lane == 0) red[0][warp].x = n_w;
    __syncthreads();
    if (lane < W) n_lane = red[0][w0 + lane].x;
    __syncthreads();
  }
  int stage = 0, buf = 0;
  // every group of the block takes the same number of turns
  for (int64_t row = first; row - grp < rows; row += step, buf ^= 1) {
    const bool live = row < rows;
    fetch(row + (kRing - 1) * step, (stage + kRing - 1) % kRing);
    F2 v[H];
#pragma unroll
    for (int i = 0; i < H; ++i) v[i] = 0;
    R::landed();
    if (live) R::take(ring, stage, 0, x + row * d, d, t, v);
    stage = (stage + 1) % kRing;
    // each warp takes its values' mean and squares about it, and the warps of
    // a row then join theirs: M2 = sum M2_w + n_w (mean_w - mean)^2.  One
    // barrier, and no difference of large sums.
    F2 s = v[0];
#pragma unroll
    for (int i = 1; i < H; ++i) s = add2(s, v[i]);
    const float mu_w = warp_sum(sum_of(s)) * inv_n;
    float mu = mu_w;
    F2 m = pair(-mu, -mu);
#pragma unroll
    for (int i = 0; i < H; ++i) v[i] = add2(v[i], m);
    S::clip(d, t, TPR, v);
    F2 q = mul2(v[0], v[0]);
#pragma unroll
    for (int i = 1; i < H; ++i) q = fma2(v[i], v[i], q);
    float m2 = warp_sum(sum_of(q));
    if (W > 1) {
      // a lane for each warp of the row
      if (lane == 0) red[buf][warp] = make_float2(mu, m2);
      group_sync<TPR>();
      const float2 of = lane < W ? red[buf][w0 + lane] : make_float2(0.0f, 0.0f);
      const float x0 = __shfl_sync(0xffffffffu, of.x, 0);
      mu = x0 + lanes_sum<W>(n_lane * (of.x - x0)) * inv_d;  // of the row
      const float e = of.x - mu;
      m2 = lanes_sum<W>(of.y + n_lane * (e * e));
    }
    // Off by 2 steps at most.  1 / sqrtf, off by 1, stands in every row's way for
    // 5 to 7% of the time (32768 x 4096 bf16 99 us for 93, 16384 x 4096 fp32 106
    // for 99).
    const float rs = rsqrtf(m2 * inv_d + eps);
    if (!live) continue;
    m = pair(mu_w - mu, mu_w - mu);  // v is about the warp's mean already
    const F2 r2 = pair(rs, rs);
#pragma unroll
    for (int i = 0; i < H; ++i) v[i] = fma2(mul2(add2(v[i], m), r2), g[i], b[i]);
    S::store(y + row * d, d, t, TPR, v);
    if (t == 0) {
      if (mean != nullptr) mean[row] = mu;
      if (rstd != nullptr) rstd[row] = rs;
    }
  }
}

// `n` values from p (16-byte pieces where n is more than 1).
template <int n, typename T>
__device__ __forceinline__ void load_n(const T* p, float* v) {
  if (n == 1) {
    v[0] = to_f32(*p);
  } else {
#pragma unroll
    for (int i = 0; i < n; i += Vec16<T>::N) Vec16<T>::load(p + i, v + i);
  }
}

// Rows that the registers do not hold: three reads of x, the last two from L1
// and L2 (8192 x 16384 bf16 forward 131 us, 4.1 TB/s, backward 271; 4096 x 5120 and
// 8192 fp32 42 and 47 us, backward 93 and 127, 1.1 to 2.4 times the bytes').  N values
// per access: a 16-byte piece, or one where rows are not whole pieces.
template <typename T, int N>
__global__ void __launch_bounds__(512)
norm_fwd_wide_kernel(const T* x, const float* __restrict__ gamma,
                     const float* __restrict__ beta, int d, float eps, T* y,
                     float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float red[2][16];
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const T* p = x + row * d;
  float s = 0.0f, v[N];
#pragma unroll 4
  for (int c = threadIdx.x * N; c < d; c += 512 * N) {
    load_n<N>(p + c, v);
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) t += v[i];
    s += t;
  }
  const float mu = block_sum512(s, red[0]) / d;
  float q = 0.0f;
#pragma unroll 4
  for (int c = threadIdx.x * N; c < d; c += 512 * N) {
    load_n<N>(p + c, v);
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) t += (v[i] - mu) * (v[i] - mu);
    q += t;
  }
  const float rs = 1.0f / sqrtf(block_sum512(q, red[1]) / d + eps);
#pragma unroll(N > 1 ? 2 : 4)
  for (int c = threadIdx.x * N; c < d; c += 512 * N) {
    float g[N], b[N] = {};
    load_n<N>(p + c, v);
    load_n<N>(gamma + c, g);
    if (beta != nullptr) load_n<N>(beta + c, b);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (v[i] - mu) * rs * g[i] + b[i];
    if (N == 1) y[row * d + c] = from_f32<T>(v[0]);
    else Vec16<T>::store(y + row * d + c, v);
  }
  if (threadIdx.x == 0) {
    if (mean != nullptr) mean[row] = mu;
    if (rstd != nullptr) rstd[row] = rs;
  }
}

template <typename T, bool VEC, int TPR>
constexpr int bwd_smem() {
  constexpr int ring = RowRing<T, VEC, TPR, 2>::kBytes;
  constexpr int sums = block_of<TPR>() > TPR ? block_of<TPR>() * NormCfg<T>::kVals * 4 : 0;
  return ring > sums ? ring : sums;
}

template <typename T, bool VEC, int TPR>
__global__ void __launch_bounds__(block_of<TPR>(), bwd_blocks<T>(TPR))
norm_bwd_kernel(const T* dy, const T* __restrict__ x, const float* __restrict__ gamma,
                const float* __restrict__ mean, const float* __restrict__ rstd, int64_t rows,
                int d, T* dx, float* __restrict__ part) {
  using S = RowSlice<T, VEC>;
  using R = RowRing<T, VEC, TPR, 2>;
  constexpr int V = S::V, H = V / 2;
  constexpr int B = block_of<TPR>();
  constexpr int RG = B / TPR;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 red[2][B / 32];
  pdl_wait();
  pdl_trigger();
  const int t = threadIdx.x % TPR;
  const int grp = threadIdx.x / TPR;
  const int64_t step = static_cast<int64_t>(gridDim.x) * RG;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * RG + grp;
  auto fetch = [&](int64_t row, int stage) {
    if (row < rows) {
      R::fetch(ring, stage, 0, x + row * d, x + rows * d, d, t);
      R::fetch(ring, stage, 1, dy + row * d, dy + rows * d, d, t);
    }
    copy_commit();
  };
#pragma unroll
  for (int s = 0; s < kRing - 1; ++s) fetch(first + s * step, s);
  F2 g[H], dg[H], db[H];
  S::load_f32(gamma, d, t, TPR, g);
#pragma unroll
  for (int i = 0; i < H; ++i) dg[i] = db[i] = 0;
  const float inv_d = 1.0f / d;
  float mu = 0.0f, rs = 0.0f;
  if (first < rows) {
    mu = mean[first];
    rs = rstd[first];
  }
  int buf = 0, stage = 0;
  // every group of the block takes the same number of turns
  for (int64_t row = first; row - grp < rows; row += step, buf ^= 1) {
    const bool live = row < rows;
    fetch(row + (kRing - 1) * step, (stage + kRing - 1) % kRing);
    float mu_next = 0.0f, rs_next = 0.0f;
    if (row + step < rows) {
      mu_next = mean[row + step];
      rs_next = rstd[row + step];
    }
    F2 h[H], v[H];
#pragma unroll
    for (int i = 0; i < H; ++i) h[i] = v[i] = 0;
    R::landed();
    if (live) {
      R::take(ring, stage, 0, x + row * d, d, t, h);
      R::take(ring, stage, 1, dy + row * d, d, t, v);
    }
    stage = (stage + 1) % kRing;
    const F2 m = pair(-mu, -mu), r2 = pair(rs, rs);
    F2 a1 = 0, a2 = 0;
#pragma unroll
    for (int i = 0; i < H; ++i) {
      // past the row dy and gamma are 0, and h is not used
      h[i] = mul2(add2(h[i], m), r2);
      dg[i] = fma2(v[i], h[i], dg[i]);
      db[i] = add2(db[i], v[i]);
      v[i] = mul2(v[i], g[i]);
      a1 = add2(a1, v[i]);
      a2 = fma2(v[i], h[i], a2);
    }
    float s1 = sum_of(a1), s2 = sum_of(a2);
    // one barrier for both sums: the next row's use of this buffer is behind
    // the barrier of the row between
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (TPR > 32) {
      constexpr int W = TPR / 32;
      const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
      if (lane == 0) red[buf][warp] = make_float2(s1, s2);
      group_sync<TPR>();
      const float2 of = lane < W ? red[buf][warp / W * W + lane] : make_float2(0.0f, 0.0f);
      s1 = lanes_sum<W>(of.x);
      s2 = lanes_sum<W>(of.y);
    }
    if (live) {
      // s (v - s1 - h s2)
      const F2 c1 = pair(-s1 * inv_d, -s1 * inv_d), c2 = pair(-s2 * inv_d, -s2 * inv_d);
#pragma unroll
      for (int i = 0; i < H; ++i) v[i] = mul2(r2, fma2(h[i], c2, add2(v[i], c1)));
      S::store(dx + row * d, d, t, TPR, v);
    }
    mu = mu_next;
    rs = rs_next;
  }
  // this block's sums: part[0] dgamma, part[1] dbeta, [gridDim.x, d] each
  float* pg = part + static_cast<int64_t>(blockIdx.x) * d;
  float* pb = part + (static_cast<int64_t>(gridDim.x) + blockIdx.x) * d;
  float dgf[V], dbf[V];
#pragma unroll
  for (int i = 0; i < H; ++i) {
    const float2 p = both(dg[i]), o = both(db[i]);
    dgf[2 * i] = p.x;
    dgf[2 * i + 1] = p.y;
    dbf[2 * i] = o.x;
    dbf[2 * i + 1] = o.y;
  }
  if (RG == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = S::col(i, t, TPR);
      if (c < d) {
        pg[c] = dgf[i];
        pb[c] = dbf[i];
      }
    }
  } else {
    // the copies of rows past the last were never issued: the ring is free
    float* acc = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = S::col(i, t, TPR);
        if (c < d) acc[grp * TPR * V + c] = pass ? dbf[i] : dgf[i];
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
template <typename T, int N>
__global__ void __launch_bounds__(512)
norm_bwd_wide_kernel(const T* dy, const T* __restrict__ x,
                     const float* __restrict__ gamma, const float* __restrict__ mean,
                     const float* __restrict__ rstd, int d, T* dx) {
  __shared__ float red[2][16];
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const float mu = mean[row], rs = rstd[row];
  float s1 = 0.0f, s2 = 0.0f, h[N], v[N], g[N];
#pragma unroll(N > 1 ? 2 : 4)
  for (int c = threadIdx.x * N; c < d; c += 512 * N) {
    load_n<N>(x + row * d + c, h);
    load_n<N>(dy + row * d + c, v);
    load_n<N>(gamma + c, g);
    float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float w = v[i] * g[i];
      t1 += w;
      t2 += w * ((h[i] - mu) * rs);
    }
    s1 += t1;
    s2 += t2;
  }
  s1 = block_sum512(s1, red[0]) / d;
  s2 = block_sum512(s2, red[1]) / d;
#pragma unroll(N > 1 ? 2 : 4)
  for (int c = threadIdx.x * N; c < d; c += 512 * N) {
    load_n<N>(x + row * d + c, h);
    load_n<N>(dy + row * d + c, v);
    load_n<N>(gamma + c, g);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = rs * (v[i] * g[i] - s1 - (h[i] - mu) * rs * s2);
    if (N == 1) dx[row * d + c] = from_f32<T>(v[0]);
    else Vec16<T>::store(dx + row * d + c, v);
  }
}

// ... and the column sums in another, a thread per N columns and slice of rows.
template <typename T, int N>
__global__ void __launch_bounds__(256)
norm_bwd_cols_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                     const float* __restrict__ mean, const float* __restrict__ rstd, int64_t rows,
                     int d, float* __restrict__ part) {
  pdl_wait();
  pdl_trigger();
  const int c = (blockIdx.x * 256 + threadIdx.x) * N;
  if (c >= d) return;
  float g[N] = {}, b[N] = {};
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    float v[N], h[N];
    load_n<N>(dy + row * d + c, v);
    load_n<N>(x + row * d + c, h);
    const float mu = mean[row], rs = rstd[row];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      g[i] += v[i] * ((h[i] - mu) * rs);
      b[i] += v[i];
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    part[static_cast<int64_t>(blockIdx.y) * d + c + i] = g[i];
    part[(static_cast<int64_t>(gridDim.y) + blockIdx.y) * d + c + i] = b[i];
  }
}

// dgamma, dbeta = column sums of the blocks' partial rows, 32 columns by 32
// slices of the rows per block, added in a fixed order.
__global__ void __launch_bounds__(1024)
norm_bwd_reduce_kernel(const float* __restrict__ part, int part_rows, int d,
                       float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float red[32][33];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float* p = part + static_cast<int64_t>(blockIdx.y) * part_rows * d;
  float s = 0.0f;
  if (c < d) {
#pragma unroll 4
    for (int r = slice; r < part_rows; r += 32) s += p[static_cast<int64_t>(r) * d + c];
  }
  red[slice][lane] = s;
  __syncthreads();
  // a warp per column
  s = warp_sum(red[lane][slice]);
  const int col = blockIdx.x * 32 + slice;
  float* out = blockIdx.y ? dbeta : dgamma;
  if (lane == 0 && col < d && out != nullptr) out[col] = s;
}

// threads per row that hold d values, or 0 (too wide)
template <typename T>
int group_of(int d) {
  for (int tpr : {32, 64, 96, 128, 192, 256, 384, 512})
    if (d <= tpr * NormCfg<T>::kVals) return tpr;
  return 0;
}

template <typename T>
int part_rows_of(int64_t T_, int d, int sms) {
  const int tpr = group_of<T>(d);
  if (tpr == 0) return static_cast<int>(T_ < 64 ? T_ : 64);
  const int rg = block_threads(tpr) / tpr;
  const int64_t blocks = (T_ + rg - 1) / rg;
  const int64_t most = static_cast<int64_t>(sms) * bwd_blocks<T>(tpr);
  return static_cast<int>(blocks < most ? blocks : most);
}

template <typename T, bool VEC, int TPR>
int fwd_impl(const T* x, const float* gamma, const float* beta, int64_t rows, int d, float eps,
             T* y, float* mean, float* rstd, int sms, cudaStream_t st) {
  constexpr int RG = block_of<TPR>() / TPR;
  constexpr int smem = RowRing<T, VEC, TPR, 1>::kBytes;
  static std::atomic<uint64_t> optin{0};
  auto kern = norm_fwd_kernel<T, VEC, TPR>;
  if (int rc = ensure_smem_optin(reinterpret_cast<const void*>(kern), smem, optin)) return rc;
  const int64_t blocks = (rows + RG - 1) / RG, most = static_cast<int64_t>(sms) * fwd_blocks<T>(TPR);
  return launch_k(kern, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                  dim3(block_of<TPR>()), smem, st, 1, x, gamma, beta, rows, d, eps, y, mean, rstd);
}

template <typename T, bool VEC>
int fwd_group(const T* x, const float* gamma, const float* beta, int64_t rows, int d, float eps,
              T* y, float* mean, float* rstd, int sms, cudaStream_t st) {
  switch (group_of<T>(d)) {
    case 32: return fwd_impl<T, VEC, 32>(x, gamma, beta, rows, d, eps, y, mean, rstd, sms, st);
    case 64: return fwd_impl<T, VEC, 64>(x, gamma, beta, rows, d, eps, y, mean, rstd, sms, st);
    case 96: return fwd_impl<T, VEC, 96>(x, gamma, beta, rows, d, eps, y, mean, rstd, sms, st);
    case 128: return fwd_impl<T, VEC, 128>(x, gamma, beta, rows, d, eps, y, mean, rstd, sms, st);
    case 192: return fwd_impl<T, VEC, 192>(x, gamma, beta, rows, d, eps, y, mean, rstd, sms, st);
    case 256: return fwd_impl<T, VEC, 256>(x, gamma, beta, rows, d, eps, y, mean, rstd, sms, st);
    case 384: return fwd_impl<T, VEC, 384>(x, gamma, beta, rows, d, eps, y, mean, rstd, sms, st);
    case 512: return fwd_impl<T, VEC, 512>(x, gamma, beta, rows, d, eps, y, mean, rstd, sms, st);
  }
  return launch_k(norm_fwd_wide_kernel<T, VEC ? Vec16<T>::N : 1>, dim3(static_cast<unsigned>(rows)), dim3(512), 0, st, 1,
                  x, gamma, beta, d, eps, y, mean, rstd);
}

template <typename T>
int fwd_typed(const void* x, const float* gamma, const float* beta, int64_t rows, int d, float eps,
              void* y, float* mean, float* rstd, int sms, cudaStream_t st) {
  const T* xt = static_cast<const T*>(x);
  T* yt = static_cast<T*>(y);
  return d % Vec16<T>::N == 0 ? fwd_group<T, true>(xt, gamma, beta, rows, d, eps, yt, mean, rstd, sms, st)
                              : fwd_group<T, false>(xt, gamma, beta, rows, d, eps, yt, mean, rstd, sms, st);
}

template <typename T, bool VEC, int TPR>
int bwd_impl(const T* dy, const T* x, const float* gamma, const float* mean, const float* rstd,
             int64_t rows, int d, T* dx, float* part, int part_rows, cudaStream_t st) {
  static std::atomic<uint64_t> optin{0};
  auto kern = norm_bwd_kernel<T, VEC, TPR>;
  constexpr int smem = bwd_smem<T, VEC, TPR>();
  if (int rc = ensure_smem_optin(reinterpret_cast<const void*>(kern), smem, optin)) return rc;
  return launch_k(kern, dim3(part_rows), dim3(block_of<TPR>()), smem, st, 1, dy, x, gamma, mean, rstd, rows, d, dx, part);
}

template <typename T, bool VEC>
int bwd_group(const T* dy, const T* x, const float* gamma, const float* mean, const float* rstd,
              int64_t rows, int d, T* dx, float* part, int part_rows, cudaStream_t st) {
  switch (group_of<T>(d)) {
    case 32: return bwd_impl<T, VEC, 32>(dy, x, gamma, mean, rstd, rows, d, dx, part, part_rows, st);
    case 64: return bwd_impl<T, VEC, 64>(dy, x, gamma, mean, rstd, rows, d, dx, part, part_rows, st);
    case 96: return bwd_impl<T, VEC, 96>(dy, x, gamma, mean, rstd, rows, d, dx, part, part_rows, st);
    case 128: return bwd_impl<T, VEC, 128>(dy, x, gamma, mean, rstd, rows, d, dx, part, part_rows, st);
    case 192: return bwd_impl<T, VEC, 192>(dy, x, gamma, mean, rstd, rows, d, dx, part, part_rows, st);
    case 256: return bwd_impl<T, VEC, 256>(dy, x, gamma, mean, rstd, rows, d, dx, part, part_rows, st);
    case 384: return bwd_impl<T, VEC, 384>(dy, x, gamma, mean, rstd, rows, d, dx, part, part_rows, st);
    case 512: return bwd_impl<T, VEC, 512>(dy, x, gamma, mean, rstd, rows, d, dx, part, part_rows, st);
  }
  // the column sums first: dx may be dy
  constexpr int N = VEC ? Vec16<T>::N : 1;
  if (int rc = launch_k(norm_bwd_cols_kernel<T, N>, dim3((d + 256 * N - 1) / (256 * N), part_rows),
                        dim3(256), 0, st, 1, dy, x, mean, rstd, rows, d, part))
    return rc;
  return launch_k(norm_bwd_wide_kernel<T, N>, dim3(static_cast<unsigned>(rows)), dim3(512), 0, st, 1,
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
                      int d, float eps, void* y, float* mean, float* rstd, int sms,
                      cudaStream_t st) {
  return dtype == MOE_DTYPE_BF16
             ? fwd_typed<bf16>(x, gamma, beta, T, d, eps, y, mean, rstd, sms, st)
             : fwd_typed<float>(x, gamma, beta, T, d, eps, y, mean, rstd, sms, st);
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
  return launch_k(norm_bwd_reduce_kernel, dim3((d + 31) / 32, dbeta != nullptr ? 2 : 1), dim3(1024),
                  0, st, 1, static_cast<const float*>(part), part_rows, d, dgamma, dbeta);
}

}  // namespace moe
