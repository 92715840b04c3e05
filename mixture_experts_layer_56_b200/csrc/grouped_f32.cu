// fp32 products of ragged row groups with their group's matrix, on CUDA cores
// (tensor cores have no fp32 multiply): forward, input and weight gradient.
//
// 64 x 64 tiles, 256 threads of 4 x 4 outputs, 16-deep slices in shared
// memory.  Products are summed over 128 values at a time and these sums added
// up apart, which keeps the rounding of long reductions near sqrt(128) rather
// than sqrt(length) half steps.
#include <cuda_runtime.h>

#include "common.cuh"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr int TM = 64, TN = 64, TK = 16;
constexpr int kFlush = 8;  // slices per inner sum
constexpr int kMaxG = 256;

template <int DIR>
__global__ void __launch_bounds__(256)
grouped_f32_kernel(const float* __restrict__ a, const float* __restrict__ b,
                   const int32_t* __restrict__ offsets, int groups, int rows, int n, int k,
                   float* __restrict__ out, bool accumulate) {
  // D[M, N] = sum A(m, r) B(n, r):
  //   forward  M rows of X (ld k),  N rows of W_g (ld k),    r over k
  //   dX       M rows of dY (ld n), N columns of W_g (ld k), r over n
  //   dW       M columns of dY,     N columns of X,          r over the rows
  __shared__ float As[TK][TM + 4];
  __shared__ float Bs[TK][TN + 4];
  __shared__ int32_t tile_start[kMaxG + 1];
  __shared__ int32_t row0s[kMaxG], rowsg[kMaxG];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int N = DIR == kGroupedFwd ? n : k;
  const int nt = (N + TN - 1) / TN;
  const int mt_dw = (n + TM - 1) / TM;
  for (int g = tid; g < groups; g += 256) {
    const int p = min(max(offsets[g], 0), rows);
    const int e = min(max(offsets[g + 1], p), rows);
    row0s[g] = p;
    rowsg[g] = e - p;
    tile_start[g + 1] = (DIR == kGroupedDw ? mt_dw : (e - p + TM - 1) / TM) * nt;
  }
  __syncthreads();
  if (tid == 0) {
    tile_start[0] = 0;
    for (int g = 0; g < groups; ++g) tile_start[g + 1] += tile_start[g];
  }
  __syncthreads();
  const int total = tile_start[groups];
  const int tx = tid & 15, ty = tid >> 4;
  for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
    int lo = 0, hi = groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tile_start[mid] <= tile) lo = mid; else hi = mid - 1;
    }
    const int g = lo;
    const int local = tile - tile_start[g];
    const int m0 = (local / nt) * TM, n0 = (local % nt) * TN;
    const int64_t r0 = row0s[g];
    const int M = DIR == kGroupedDw ? n : rowsg[g];
    const int R = DIR == kGroupedFwd ? k : (DIR == kGroupedDx ? n : rowsg[g]);
    const float* wg = DIR == kGroupedDw ? nullptr : b + static_cast<int64_t>(g) * n * k;
    float acc[4][4] = {}, sum[4][4] = {};
    for (int rb = 0, cnt = 0; rb < R; rb += TK) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = tid + i * 256;  // 1024 values of each operand
        {
          // consecutive threads follow the operand's memory rows
          const int mm = DIR == kGroupedDw ? (e & 63) : (e >> 4);
          const int rr = DIR == kGroupedDw ? (e >> 6) : (e & 15);
          float v = 0.0f;
          if (m0 + mm < M && rb + rr < R) {
            if (DIR == kGroupedDw) v = a[(r0 + rb + rr) * n + m0 + mm];
            else v = a[(r0 + m0 + mm) * (DIR == kGroupedFwd ? k : n) + rb + rr];
          }
          As[rr][mm] = v;
        }
        {
          const int nn = DIR == kGroupedFwd ? (e >> 4) : (e & 63);
          const int rr = DIR == kGroupedFwd ? (e & 15) : (e >> 6);
          float v = 0.0f;
          if (n0 + nn < N && rb + rr < R) {
            if (DIR == kGroupedFwd) v = wg[static_cast<int64_t>(n0 + nn) * k + rb + rr];
            else if (DIR == kGroupedDx) v = wg[static_cast<int64_t>(rb + rr) * k + n0 + nn];
            else v = b[(r0 + rb + rr) * k + n0 + nn];
          }
          Bs[rr][nn] = v;
        }
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < TK; ++r) {
        const float4 x = *reinterpret_cast<const float4*>(&As[r][ty * 4]);
        const float4 y = *reinterpret_cast<const float4*>(&Bs[r][tx * 4]);
        const float xv[4] = {x.x, x.y, x.z, x.w}, yv[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xv[i], yv[j], acc[i][j]);
      }
      if (++cnt == kFlush) {
        cnt = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sum[i][j] += acc[i][j];
            acc[i][j] = 0.0f;
          }
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + ty * 4 + i;
      if (m >= M) continue;
      float* row = DIR == kGroupedDw ? out + (static_cast<int64_t>(g) * n + m) * k
                                     : out + (r0 + m) * N;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = n0 + tx * 4 + j;
        if (c >= N) continue;
        const float v = sum[i][j] + acc[i][j];
        row[c] = accumulate ? row[c] + v : v;
      }
    }
  }
}

}  // namespace

int launch_grouped_f32(int dir, const float* a, const float* b, const int32_t* offsets, int groups,
                       int64_t rows, int n, int k, float* out, bool accumulate, int sms,
                       cudaStream_t st) {
  const int N = dir == kGroupedFwd ? n : k;
  const int64_t nt = (N + TN - 1) / TN;
  const int64_t mt = dir == kGroupedDw ? static_cast<int64_t>(groups) * ((n + TM - 1) / TM)
                                       : (rows + TM - 1) / TM + (rows < groups ? rows : groups);
  const int64_t tiles = mt * nt, most = 4ll * sms;
  const int grid = static_cast<int>(tiles < most ? tiles : most);
  if (grid <= 0) return MOE_OK;
  auto kern = dir == kGroupedFwd ? grouped_f32_kernel<kGroupedFwd>
              : dir == kGroupedDx ? grouped_f32_kernel<kGroupedDx>
                                  : grouped_f32_kernel<kGroupedDw>;
  return launch_k(kern, dim3(grid), dim3(256), 0, st, 1, a, b, offsets, groups,
                  static_cast<int>(rows), n, k, out, accumulate);
}

}  // namespace moe
