// Newton-Schulz orthogonalisation of matrices whose short side is at most 128
// and whose long side at most 2048: all steps in one kernel, the matrix held
// on chip (the same numerics as ortho.cu: fp16 products beside X = hi + lo,
// the diagonals of A and B in fp32).
//
// One cluster of up to 8 CTAs per matrix.  X has the short side as its rows
// (128, the rest zero) and is cut along the long side, up to 256 columns per
// CTA in slices of 64.  A slice is 128 rows of 128 bytes, swizzled: read as a
// K-major tile it is an operand of X X^T, read as an MN-major one the operand
// X of B X, so that one copy in shared memory serves both products.  Per step
//
//   1. each CTA's part of A = X X^T (tcgen05), left as fp32 in shared memory
//   2. the cluster adds the parts up in a fixed order, each CTA its share of
//      the entries, and writes them to every CTA (fp16, the diagonal in fp32)
//   3. every CTA computes B = b A + c A A for itself, over A's place
//   4. and its columns of X <- a X + B X
//
// Bound by latency: some ten waits of one or two microseconds a step, against
// three kernel launches and their pipelines' filling and draining.  One matrix of
// 64 x 2048, five steps: 48 us, 8 a step.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "mm_ptx.cuh"
#include "train_kernels.h"

namespace moe {
namespace sm100 {

namespace {

constexpr int kSmThreads = 512;            // 16 warps: four per TMEM lane quarter
constexpr int kSmSide = 128;               // rows of X, padded
constexpr int kSmSlice = kSmSide * 128;    // bytes of 64 columns
constexpr int kSmMaxSlices = 4;
constexpr int kSmMaxCtas = 8;
constexpr int kSmSquare = 2 * kSmSlice;    // A or B: 128 x 128 fp16, two k-blocks
constexpr int kSmPart = kSmSide * kSmSide * 4;
// At least this much, so that an SM holds no other kernel's tensor memory beside
// a CTA's, which takes all of it: two clusters, each with a CTA that has its
// columns and one that waits for the other's, would wait for good.  The 67 KB
// left over are less than four stages of a 128-row pair's pipeline.  (With 200
// KB, L1 is short of M's second reading: five of 128 x 512 46.7 us for 44.8.)
constexpr int kSmLeast = 160 * 1024;

struct OrthoCoef {
  float v[3 * 16];
};

__device__ __forceinline__ uint32_t cluster_size_x() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}
// cluster_sync_all in two halves, for the work of one CTA between them
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u32x2(uint32_t addr, uint2 v) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y)
               : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}
// orders this thread's writes to any CTA's shared memory before the MMAs' reads
__device__ __forceinline__ void fence_async_cluster() {
  asm volatile("fence.proxy.async.shared::cluster;" ::: "memory");
}

// byte offset of 16-byte piece `ch` (0..7) of row i in a swizzled 128-row tile
__device__ __forceinline__ int tile_at(int i, int ch) { return i * 128 + ((ch ^ (i & 7)) << 4); }
// of piece `ch` (0..31) of row i in the fp32 part; swizzled against conflicts
__device__ __forceinline__ int part_at(int i, int ch) { return i * 512 + ((ch ^ (i & 31)) << 4); }

template <typename T>
__global__ void __launch_bounds__(kSmThreads, 1)
ortho_small_kernel(const T* __restrict__ M, bf16* __restrict__ O, int rows, int cols, int steps,
                   const OrthoCoef coef, float scale, int nsl, int32_t* status) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_mem;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ __align__(16) float da[kSmSide], db[kSmSide];
  __shared__ double sums[kSmMaxCtas];
  __shared__ double red[kSmThreads / 32];

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* hi = smem;
  uint8_t* lo = hi + nsl * kSmSlice;
  uint8_t* sq = lo + nsl * kSmSlice;  // A, then B, off the diagonal
  uint8_t* part = sq + kSmSquare;
  const uint32_t bar = smem_addr(&bar_mem);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int size = static_cast<int>(cluster_size_x());
  const int64_t mat = static_cast<int64_t>(cluster_id_x());
  const bool tall = rows > cols;
  const int m = tall ? cols : rows, n = tall ? rows : cols;
  const int width = nsl * 64, pieces = width / 8;  // this CTA's columns of X
  const int j0 = rank * width;
  const T* src = M + mat * rows * cols;
  volatile int* abort_p = &abort_flag;

  if (tid == 0) {
    mbar_init(bar, 1);
    abort_flag = 0;
    fence_mbar_init();
    fence_async_shared();
  }
  __syncwarp();  // here and below: what is .aligned wants the warp's lanes together
  if (warp == 0) {
    tmem_alloc(smem_addr(&tmem_slot), 512);
    tmem_relinquish();
  }
  // A CTA's shared memory may be written from the others only once it has
  // started: they wait for that behind the pass over M.
  cluster_arrive();
  pdl_wait();
  pdl_trigger();

  // X's pieces of 8 columns, those of its m real rows.  Neighbouring threads
  // follow M's rows: along a row of X, or for a tall M down a column.
  const int items = m * pieces;
  auto piece_of = [&](int item, int& i, int& ch) {
    if (tall) {
      ch = item / m;
      i = item - ch * m;
    } else {
      i = item / pieces;
      ch = item - i * pieces;
    }
  };
  const bool vec = !tall && cols % 8 == 0;
  auto load_piece = [&](int item, float* v) {
    int i, ch;
    piece_of(item, i, ch);
    const int j = j0 + ch * 8;
    if (vec) {
      if (item < items && j < n) {
#pragma unroll
        for (int e = 0; e < 8; e += Vec16<T>::N)
          Vec16<T>::load(src + static_cast<int64_t>(i) * cols + j + e, v + e);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
      }
      return;
    }
    const int64_t at = tall ? static_cast<int64_t>(j) * cols + i
                            : static_cast<int64_t>(i) * cols + j;
    const int64_t step = tall ? cols : 1;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = item < items && j + e < n ? to_f32(src[at + e * step]) : 0.0f;
  };
  constexpr int kBatch = 4;  // pieces whose loads are in flight together

  // ---- |M|_F, in fp64: squares of large finite entries overflow fp32 -------
  double s = 0.0;
  for (int t = tid; t < items; t += kBatch * kSmThreads) {
    float v[kBatch][8];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) load_piece(t + k * kSmThreads, v[k]);
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += static_cast<double>(v[k][e]) * v[k][e];
  }
  // meanwhile: zeros in X, A and B; their rows past m stay so
  for (int t = tid; t < (2 * nsl * kSmSlice + kSmSquare) / 16; t += kSmThreads)
    reinterpret_cast<uint4*>(hi)[t] = make_uint4(0, 0, 0, 0);
  if (tid < kSmSide) da[tid] = db[tid] = 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) red[warp] = s;
  __syncthreads();
  cluster_wait();  // every CTA has started
  if (tid < size) {
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < kSmThreads / 32; ++i) t += red[i];
    st_cluster_f64(map_to_cta(smem_addr(&sums[rank]), static_cast<uint32_t>(tid)), t);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  double sqsum = 0.0;
  for (int i = 0; i < size; ++i) sqsum += sums[i];
  const double f = scale / (sqrt(sqsum) + 1e-7);
  for (int t = tid; t < items; t += kBatch * kSmThreads) {
    float v[kBatch][8];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) load_piece(t + k * kSmThreads, v[k]);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (t + k * kSmThreads >= items) break;
      int i, ch;
      piece_of(t + k * kSmThreads, i, ch);
      __half h[8], l[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = static_cast<float>(v[k][e] * f);
        h[e] = __float2half_rn(x);
        l[e] = __float2half_rn(x - __half2float(h[e]));
      }
      const int at = (ch >> 3) * kSmSlice + tile_at(i, ch & 7);
      *reinterpret_cast<uint4*>(hi + at) = *reinterpret_cast<const uint4*>(h);
      *reinterpret_cast<uint4*>(lo + at) = *reinterpret_cast<const uint4*>(l);
    }
  }

  const float inv2 = 1.0f / (scale * scale);
  const int q = warp & 3, part4 = warp >> 2;  // TMEM lane quarter, quarter of the columns
  const int r = q * 32 + lane;               // this thread's row
  const bool idle = q * 32 >= m;             // no row of this warp is the matrix's
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16);
  constexpr uint32_t kUpd = 128;  // TMEM columns: A (or A A) at 0, B X at 128
  uint32_t phase = 0;
  // waits for the MMAs that thread 0 committed (every thread)
  auto wait_mma = [&] {
    wait_bounded(bar, phase, abort_p, status);
    phase ^= 1u;
    __syncwarp();
    tc_fence_after();
  };

  for (int step = 0; step < steps; ++step) {
    const float ca = coef.v[3 * step], cb = coef.v[3 * step + 1], cc = coef.v[3 * step + 2];
    // ---- 1. this CTA's part of X X^T ----------------------------------------
    fence_async_shared();  // hi was written by ordinary stores
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      constexpr uint32_t idesc = idesc_16bit_f32(128, 128, true, false, false);
      for (int sl = 0; sl < nsl; ++sl) {
        const uint64_t d = desc_kmajor_sw128(smem_addr(hi + sl * kSmSlice));
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_bf16(tmem, d + k * 2, d + k * 2, idesc, sl > 0 || k > 0);
      }
      mma_commit(bar);
    }
    __syncwarp();
    wait_mma();
    // ---- 2. A: the parts' sum, to every CTA ---------------------------------
    if (size == 1) {
      if (!idle) {
        float x[32];
        tmem_ld32(lane_base + part4 * 32, x);
        tmem_ld_wait_regs(x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = part4 * 32 + i * 8;
          uint4 w;
          __half2* h = reinterpret_cast<__half2*>(&w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[i * 8 + e] *= inv2;
            if (col + e == r) {
              da[r] = x[i * 8 + e];
              x[i * 8 + e] = 0.0f;
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            h[e] = __floats2half2_rn(x[i * 8 + 2 * e], x[i * 8 + 2 * e + 1]);
          *reinterpret_cast<uint4*>(sq + (col >> 6) * kSmSlice + tile_at(r, (col >> 3) & 7)) = w;
        }
      }
      fence_async_shared();
      tc_fence_before();
      __syncthreads();
    } else {
      if (!idle) {
        float x[32];
        tmem_ld32(lane_base + part4 * 32, x);
        tmem_ld_wait_regs(x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float4*>(part + part_at(r, part4 * 8 + i)) =
              make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      }
      tc_fence_before();
      cluster_sync_all();
      // groups of 4 columns of the m rows, spread over the cluster's threads
      const int per_row = (m + 3) >> 2;
      for (int t = rank * kSmThreads + tid; t < m * per_row; t += size * kSmThreads) {
        const int i = t / per_row, ch = t - i * per_row;
        const uint32_t at = smem_addr(part + part_at(i, ch));
        float4 v[kSmMaxCtas];
#pragma unroll
        for (int p = 0; p < kSmMaxCtas; ++p)
          v[p] = p < size ? ld_cluster_f32x4(map_to_cta(at, static_cast<uint32_t>(p)))
                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float y[4] = {};
#pragma unroll
        for (int p = 0; p < kSmMaxCtas; ++p) {
          y[0] += v[p].x;
          y[1] += v[p].y;
          y[2] += v[p].z;
          y[3] += v[p].w;
        }
        float diag = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] *= inv2;
          if (ch * 4 + e == i) {
            diag = y[e];
            y[e] = 0.0f;
          }
        }
        uint2 w;
        __half2* h = reinterpret_cast<__half2*>(&w);
        h[0] = __floats2half2_rn(y[0], y[1]);
        h[1] = __floats2half2_rn(y[2], y[3]);
        // columns 4 ch .. 4 ch + 3: half of 16-byte piece ch / 2
        const uint32_t to =
            smem_addr(sq + (ch >> 4) * kSmSlice + tile_at(i, (ch >> 1) & 7) + (ch & 1) * 8);
#pragma unroll
        for (int p = 0; p < kSmMaxCtas; ++p)
          if (p < size) st_cluster_u32x2(map_to_cta(to, static_cast<uint32_t>(p)), w);
        if ((i >> 2) == ch) {
#pragma unroll
          for (int p = 0; p < kSmMaxCtas; ++p)
            if (p < size)
              st_cluster_f32(map_to_cta(smem_addr(&da[i]), static_cast<uint32_t>(p)), diag);
        }
      }
      fence_async_cluster();
      __syncwarp();
      cluster_sync_all();
    }
    // ---- 3. B = b A + c A A -------------------------------------------------
    if (tid == 0) {
      fence_async_cluster();
      tc_fence_after();
      constexpr uint32_t idesc = idesc_16bit_f32(128, 128, true, false, false);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const uint64_t d = desc_kmajor_sw128(smem_addr(sq + kb * kSmSlice));
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_bf16(tmem, d + k * 2, d + k * 2, idesc, kb > 0 || k > 0);
      }
      mma_commit(bar);
    }
    __syncwarp();
    wait_mma();
    if (!idle) {
      const float di = da[r];
      float x[32];
      tmem_ld32(lane_base + part4 * 32, x);
      tmem_ld_wait_regs(x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = part4 * 32 + i * 8;
        uint4* at = reinterpret_cast<uint4*>(sq + (col >> 6) * kSmSlice + tile_at(r, (col >> 3) & 7));
        uint4 w = *at;
        __half2* h = reinterpret_cast<__half2*>(&w);
        float dj[8];
        Vec16<float>::load(da + col, dj);
        Vec16<float>::load(da + col + 4, dj + 4);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 a = __half22float2(h[e / 2]);
          float y0 = cb * a.x + cc * ((di + dj[e]) * a.x + x[i * 8 + e]);
          float y1 = cb * a.y + cc * ((di + dj[e + 1]) * a.y + x[i * 8 + e + 1]);
          // on the diagonal, where a = 0: b d + c (d^2 + the product's)
          if (col + e == r) {
            db[r] = y0 + di * (cb + cc * di);
            y0 = 0.0f;
          }
          if (col + e + 1 == r) {
            db[r] = y1 + di * (cb + cc * di);
            y1 = 0.0f;
          }
          h[e / 2] = __floats2half2_rn(y0, y1);
        }
        *at = w;
      }
    }
    fence_async_shared();
    tc_fence_before();
    __syncthreads();
    // ---- 4. X <- a X + B X --------------------------------------------------
    if (tid == 0) {
      tc_fence_after();
      const uint32_t idesc = idesc_16bit_f32(128, 0, true, false, true) |
                             (static_cast<uint32_t>(width >> 3) << 17);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint64_t d = desc_kmajor_sw128(smem_addr(sq + (k >> 2) * kSmSlice)) + (k & 3) * 2;
        const uint64_t x = desc_mnmajor_sw128(smem_addr(hi) + k * 2048, kSmSlice);
        mma_bf16(tmem + kUpd, d, x, idesc, k > 0);
      }
      mma_commit(bar);
    }
    __syncwarp();
    wait_mma();
    const float dr = idle ? 0.0f : db[r];
#pragma unroll 2
    for (int c = 0; !idle && c < nsl; ++c) {
      float x[16];
      const int col = part4 * (width / 4) + c * 16;  // of this CTA's columns
      tmem_ld16(lane_base + kUpd + col, x);
      tmem_ld_wait_regs16(x);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int ch = col / 8 + i;
        const int at = (ch >> 3) * kSmSlice + tile_at(r, ch & 7);
        uint4 hw = *reinterpret_cast<uint4*>(hi + at), lw = *reinterpret_cast<uint4*>(lo + at);
        __half2* h = reinterpret_cast<__half2*>(&hw);
        __half2* l = reinterpret_cast<__half2*>(&lw);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 hf = __half22float2(h[e]), lf = __half22float2(l[e]);
          const float y0 = ca * (hf.x + lf.x) + dr * hf.x + x[i * 8 + 2 * e];
          const float y1 = ca * (hf.y + lf.y) + dr * hf.y + x[i * 8 + 2 * e + 1];
          h[e] = __floats2half2_rn(y0, y1);
          const float2 nf = __half22float2(h[e]);
          l[e] = __floats2half2_rn(y0 - nf.x, y1 - nf.y);
        }
        *reinterpret_cast<uint4*>(hi + at) = hw;
        *reinterpret_cast<uint4*>(lo + at) = lw;
      }
    }
    tc_fence_before();
  }

  // ---- O = X / scale --------------------------------------------------------
  __syncthreads();
  bf16* dst = O + mat * rows * cols;
  const float inv = 1.0f / scale;
  for (int t = tid; t < items; t += kSmThreads) {
    int i, ch;
    piece_of(t, i, ch);
    const int j = j0 + ch * 8;
    if (j >= n) continue;
    const int at = (ch >> 3) * kSmSlice + tile_at(i, ch & 7);
    const __half* h = reinterpret_cast<const __half*>(hi + at);
    const __half* l = reinterpret_cast<const __half*>(lo + at);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (__half2float(h[e]) + __half2float(l[e])) * inv;
    if (vec) {
      Vec16<bf16>::store(dst + static_cast<int64_t>(i) * cols + j, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e < n)
          dst[tall ? static_cast<int64_t>(j + e) * cols + i
                   : static_cast<int64_t>(i) * cols + j + e] = __float2bfloat16_rn(v[e]);
    }
  }
  __syncwarp();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T>
int launch_small(const void* M, void* O, int mats, int rows, int cols, int steps,
                 const OrthoCoef& coef, float scale, int32_t* status, cudaStream_t st) {
  const int n = rows > cols ? rows : cols;
  // one slice per CTA up to 8 CTAs: a step's work on a slice takes longer than
  // the cluster's exchange
  int size = 1;
  while (size < kSmMaxCtas && size * 64 < n) size *= 2;
  const int nsl = (n + size * 64 - 1) / (size * 64);
  const int need = 2 * nsl * kSmSlice + kSmSquare + kSmPart + 1024;
  constexpr int most = 2 * kSmMaxSlices * kSmSlice + kSmSquare + kSmPart + 1024;
  static std::atomic<uint64_t> optin{0};
  auto kern = ortho_small_kernel<T>;
  if (int rc = ensure_smem_optin(reinterpret_cast<const void*>(kern), most, optin)) return rc;
  return launch_k(kern, dim3(static_cast<unsigned>(mats) * size), dim3(kSmThreads),
                  need > kSmLeast ? need : kSmLeast, st, size, static_cast<const T*>(M),
                  static_cast<bf16*>(O), rows, cols, steps, coef, scale, nsl, status);
}

}  // namespace

}  // namespace sm100

bool ortho_small_fits(int rows, int cols) {
  using namespace sm100;
  const int m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
  return m <= kSmSide && n <= kSmMaxCtas * kSmMaxSlices * 64;
}

int launch_ortho_small(int dtype, const void* M, void* O, int mats, int rows, int cols, int steps,
                       const float* coef, float scale, int32_t* status, cudaStream_t st) {
  using namespace sm100;
  OrthoCoef c{};
  for (int i = 0; i < 3 * steps; ++i) c.v[i] = coef[i];
  return dtype == MOE_DTYPE_BF16
             ? launch_small<bf16>(M, O, mats, rows, cols, steps, c, scale, status, st)
             : launch_small<float>(M, O, mats, rows, cols, steps, c, scale, status, st);
}

}  // namespace moe
