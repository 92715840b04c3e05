// fp32 products of ragged row groups with their group's matrix, on CUDA cores
// (tensor cores have no fp32 multiply): forward, input and weight gradient.
//
// 16 x 16 threads, MI x MI outputs each, 16-deep slices in two shared-memory
// buffers: the next slice is on its way from global memory while one is
// multiplied.  MI = 8 (128 x 128 tiles) reads 16 values from shared memory
// per 64 multiply-adds and is bound by the fp32 pipe; MI = 4 (64 x 64 tiles)
// is for shapes whose larger tiles would leave SMs idle or rows empty.
// Multiply-adds are issued in pairs (fma.rn.f32x2, each lane rounded as an
// fma.rn.f32).
//
// The weight gradient, whose reduction is a group's rows, sums 128 products at
// a time and adds these sums up apart, which keeps the rounding of long groups
// near sqrt(128) rather than sqrt(rows) half steps.  The other two sum a
// matrix's width in one chain, as two blocks per SM leave no registers for
// more (8 x 1024 x 2048 x 1024: 49 TFLOP/s, with apart sums 46).
#include <cuda_runtime.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "group_spans.cuh"
#include "sm100_ptx.cuh"
#include "train_kernels.h"

namespace moe {

namespace {

using namespace sm100;

constexpr int TK = 16;
constexpr int kFlush = 8;  // slices per inner sum
constexpr int kMaxG = 256;

__device__ __forceinline__ F2 ld_cluster_f2(uint32_t addr) {
  F2 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// Four neighbours p[0..3], those at or past `left` zero.
__device__ __forceinline__ float4 load4(const float* p, int left, bool vec) {
  if (left >= 4 && vec) return *reinterpret_cast<const float4*>(p);
  float4 v;
  v.x = left > 0 ? p[0] : 0.0f;
  v.y = left > 1 ? p[1] : 0.0f;
  v.z = left > 2 ? p[2] : 0.0f;
  v.w = left > 3 ? p[3] : 0.0f;
  return v;
}

// An operand's slices: T rows (of D's M or N) by 16 reduction steps.  ALONG_R:
// its memory rows run along the reduction, else along M (or N).
template <int T, bool ALONG_R>
struct Slice {
  static constexpr int V = T * TK / 4 / 256;  // float4s per thread
  float4 v[V];
  // base: the tile's first element; rows, left: what remains of the tile's
  // extent and of the reduction
  __device__ __forceinline__ void load(const float* base, int64_t ld, int rows, int left, bool vec,
                                       int tid) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = tid + i * 256;
      if (ALONG_R) {
        const int row = e >> 2, r = (e & 3) * 4;
        v[i] = load4(base + row * ld + r, row < rows ? left - r : 0, vec);
      } else {
        const int r = e / (T / 4), m = e % (T / 4) * 4;
        v[i] = load4(base + r * ld + m, r < left ? rows - m : 0, vec);
      }
    }
  }
  __device__ __forceinline__ void put(float (*s)[T + 4], int tid) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = tid + i * 256;
      if (ALONG_R) {
        const int row = e >> 2, r = (e & 3) * 4;
        s[r][row] = v[i].x;
        s[r + 1][row] = v[i].y;
        s[r + 2][row] = v[i].z;
        s[r + 3][row] = v[i].w;
      } else {
        const int r = e / (T / 4), m = e % (T / 4) * 4;
        *reinterpret_cast<float4*>(&s[r][m]) = v[i];
      }
    }
  }
};

template <int DIR, int MI, bool SPLIT>
__global__ void __launch_bounds__(256, MI == 8 && DIR == kGroupedDw ? 1 : 2)
grouped_f32_kernel(const float* __restrict__ a, const float* __restrict__ b,
                   const int32_t* __restrict__ offsets, int groups, int rows, int n, int k,
                   float* __restrict__ out, bool accumulate) {
  // D[M, N] = sum A(m, r) B(n, r):
  //   forward  M rows of X (ld k),  N rows of W_g (ld k),    r over k
  //   dX       M rows of dY (ld n), N columns of W_g (ld k), r over n
  //   dW       M columns of dY,     N columns of X,          r over the rows
  constexpr int T = 16 * MI;
  constexpr bool FWD = DIR == kGroupedFwd, DX = DIR == kGroupedDx, DW = DIR == kGroupedDw;
  static_assert(!SPLIT || MI * MI * 256 <= 4 * TK * (T + 4), "the sums take the slices' place");
  __shared__ __align__(16) float slices[4][TK][T + 4];  // A's two buffers, B's two
  float (*const As)[TK][T + 4] = slices, (*const Bs)[TK][T + 4] = slices + 2;
  __shared__ int32_t tile_start[kMaxG + 1];
  __shared__ int32_t row0s[kMaxG], rowsg[kMaxG];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  // The CTAs of a cluster take a tile's slices in turn.
  const int part = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
  const int parts = SPLIT ? static_cast<int>(gridDim.x / num_clusters_x()) : 1;
  const int N = FWD ? n : k;
  const int nt = (N + T - 1) / T;
  const int mt_dw = (n + T - 1) / T;
  group_spans(offsets, groups, rows, tile_start, tid, 256);
  for (int g = tid; g < groups; g += 256) {
    row0s[g] = tile_start[g];
    rowsg[g] = tile_start[g + 1] - tile_start[g];
  }
  __syncthreads();
  for (int g = tid; g < groups; g += 256)
    tile_start[g + 1] = (DW ? mt_dw : (rowsg[g] + T - 1) / T) * nt;
  __syncthreads();
  if (tid < 32) {
    // inclusive scan, a run of groups per lane
    const int per = (groups + 31) / 32, beg = min(tid * per, groups), end = min(beg + per, groups);
    int sum = 0;
    for (int i = beg; i < end; ++i) sum += tile_start[i + 1];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (tid >= o) incl += v;
    }
    int run = incl - sum;
    for (int i = beg; i < end; ++i) {
      run += tile_start[i + 1];
      tile_start[i + 1] = run;
    }
    if (tid == 0) tile_start[0] = 0;
  }
  __syncthreads();
  const int total = tile_start[groups];
  const int tx = tid & 15, ty = tid >> 4;
  const int64_t lda = FWD ? k : n, ldb = k;
  const bool vec_a = lda % 4 == 0, vec_b = ldb % 4 == 0;
  for (int tile = blockIdx.x / parts; tile < total; tile += gridDim.x / parts) {
    int lo = 0, hi = groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tile_start[mid] <= tile) lo = mid; else hi = mid - 1;
    }
    const int g = lo;
    const int local = tile - tile_start[g];
    const int m0 = (local / nt) * T, n0 = (local % nt) * T;
    const int64_t r0 = row0s[g];
    const int M = DW ? n : rowsg[g];
    const int R = FWD ? k : (DX ? n : rowsg[g]);
    const float* wg = DW ? nullptr : b + static_cast<int64_t>(g) * n * k;
    const float* pa = DW ? a + r0 * n + m0 : a + (r0 + m0) * lda;
    const float* pb = FWD ? wg + static_cast<int64_t>(n0) * k : (DX ? wg + n0 : b + r0 * k + n0);
    const int64_t step_a = DW ? lda * TK : TK, step_b = FWD ? TK : ldb * TK;
    Slice<T, !DW> sa;
    Slice<T, FWD> sb;
    uint64_t acc[MI][MI / 2], sum[MI][MI / 2];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < MI / 2; ++j) acc[i][j] = sum[i][j] = 0;
    const int first = part * TK, stride = parts * TK;
    if (first < R) {
      pa += step_a * part;
      pb += step_b * part;
      sa.load(pa, lda, M - m0, R - first, vec_a, tid);
      sb.load(pb, ldb, N - n0, R - first, vec_b, tid);
    }
    int buf = 0, cnt = 0;
    for (int rb = first; rb < R; rb += stride, buf ^= 1) {
      sa.put(As[buf], tid);
      sb.put(Bs[buf], tid);
      // the slice before last is behind this barrier, and its buffer free
      __syncthreads();
      if (rb + stride < R) {
        pa += step_a * parts;
        pb += step_b * parts;
        sa.load(pa, lda, M - m0, R - rb - stride, vec_a, tid);
        sb.load(pb, ldb, N - n0, R - rb - stride, vec_b, tid);
      }
#pragma unroll
      for (int r = 0; r < TK; ++r) {
        // outputs ty*4 + i (+ 64), tx*4 + j (+ 64)
        float x[MI];
        uint64_t y[MI / 2];
#pragma unroll
        for (int h = 0; h < MI / 4; ++h) {
          const float4 xv = *reinterpret_cast<const float4*>(&As[buf][r][h * 64 + ty * 4]);
          x[h * 4] = xv.x; x[h * 4 + 1] = xv.y; x[h * 4 + 2] = xv.z; x[h * 4 + 3] = xv.w;
          const ulonglong2 yv = *reinterpret_cast<const ulonglong2*>(&Bs[buf][r][h * 64 + tx * 4]);
          y[h * 2] = yv.x;
          y[h * 2 + 1] = yv.y;
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const uint64_t xx = pair(x[i], x[i]);
#pragma unroll
          for (int j = 0; j < MI / 2; ++j) acc[i][j] = fma2(xx, y[j], acc[i][j]);
        }
      }
      if (DW && ++cnt == kFlush) {
        cnt = 0;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < MI / 2; ++j) {
            sum[i][j] = add2(sum[i][j], acc[i][j]);
            acc[i][j] = 0;
          }
      }
    }
    __syncthreads();  // the next tile writes buffer 0 again
    auto store = [&](int i, int j, F2 value) {
      const int m = m0 + (i >> 2) * 64 + ty * 4 + (i & 3);
      if (m >= M) return;
      float* row = DW ? out + (static_cast<int64_t>(g) * n + m) * k : out + (r0 + m) * N;
      const int c = n0 + (j >> 1) * 64 + tx * 4 + (j & 1) * 2;
      const float2 v = both(value);
      if (c < N) row[c] = accumulate ? row[c] + v.x : v.x;
      if (c + 1 < N) row[c + 1] = accumulate ? row[c + 1] + v.y : v.y;
    };
    if (!SPLIT) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < MI / 2; ++j)
          store(i, j, DW ? add2(sum[i][j], acc[i][j]) : acc[i][j]);
    } else {
      // the CTAs' sums are added up in order, each CTA its share of the tile
      F2* mine = reinterpret_cast<F2*>(&slices[0][0][0]);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < MI / 2; ++j)
          mine[(i * (MI / 2) + j) * 256 + tid] = DW ? add2(sum[i][j], acc[i][j]) : acc[i][j];
      cluster_sync_all();
      const int share = MI * (MI / 2) / parts;
      for (int e = part * share; e < (part + 1) * share; ++e) {
        const uint32_t at = smem_addr(mine + e * 256 + tid);
        F2 v = 0;
        for (int p = 0; p < parts; ++p) v = add2(v, ld_cluster_f2(map_to_cta(at, p)));
        store(e / (MI / 2), e % (MI / 2), v);
      }
      cluster_sync_all();
    }
  }
}

template <int MI, bool SPLIT>
int launch_tiles(int dir, const float* a, const float* b, const int32_t* offsets, int groups,
                 int64_t rows, int n, int k, float* out, bool accumulate, int64_t tiles, int most,
                 int parts, cudaStream_t st) {
  const int grid = static_cast<int>(tiles < most ? tiles : most) * parts;
  if (grid <= 0) return MOE_OK;
  auto kern = dir == kGroupedFwd ? grouped_f32_kernel<kGroupedFwd, MI, SPLIT>
              : dir == kGroupedDx ? grouped_f32_kernel<kGroupedDx, MI, SPLIT>
                                  : grouped_f32_kernel<kGroupedDw, MI, SPLIT>;
  return launch_k(kern, dim3(grid), dim3(256), 0, st, parts, a, b, offsets, groups,
                  static_cast<int>(rows), n, k, out, accumulate);
}

}  // namespace

int launch_grouped_f32(int dir, const float* a, const float* b, const int32_t* offsets, int groups,
                       int64_t rows, int n, int k, float* out, bool accumulate, int sms,
                       cudaStream_t st) {
  const int64_t N = dir == kGroupedFwd ? n : k;
  const int64_t some = rows < groups ? rows : groups;  // groups with rows, at most
  auto tiles = [&](int T) {
    const int64_t nt = (N + T - 1) / T;
    return nt * (dir == kGroupedDw ? static_cast<int64_t>(groups) * ((n + T - 1) / T)
                                   : (rows + T - 1) / T + some);
  };
  // The tile size whose most loaded SM is done first: a 128 x 128 tile is four
  // 64 x 64 ones, which take 1.45 times as long for the same work (8 x 1024 x
  // 2048 x 1024: 49 against 34 TFLOP/s; 16 x 300 x 512 x 512: 105 against 93 us).
  auto rounds = [&](int T) { return (tiles(T) + sms - 1) / sms; };
  const bool fill = dir == kGroupedDw || rows >= 96 * some;  // groups fill the large ones
  if (fill && 4.0 * rounds(128) <= 1.45 * rounds(64))
    return launch_tiles<8, false>(dir, a, b, offsets, groups, rows, n, k, out, accumulate,
                                  tiles(128), dir == kGroupedDw ? sms : 2 * sms, 1, st);
  // Few tiles: clusters of up to 8 CTAs share a tile's reduction, four slices
  // each at least (6 x 357 rows of 248 x 656: 46 us without).
  const int64_t length = dir == kGroupedFwd ? k : dir == kGroupedDx ? n : rows / groups;
  int parts = 1;
  while (parts < 8 && tiles(64) * parts * 2 <= 4ll * sms && length >= 4ll * TK * parts * 2) parts *= 2;
  if (parts > 1)
    return launch_tiles<4, true>(dir, a, b, offsets, groups, rows, n, k, out, accumulate, tiles(64),
                                 4 * sms / parts, parts, st);
  return launch_tiles<4, false>(dir, a, b, offsets, groups, rows, n, k, out, accumulate, tiles(64),
                                3 * sms, 1, st);
}

}  // namespace moe
