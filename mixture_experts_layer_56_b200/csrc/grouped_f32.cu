// fp32 products of ragged row groups with their group's matrix, on CUDA cores
// (tensor cores have no fp32 multiply): forward, input and weight gradient.
//
// 16 x 16 threads, MI x MI outputs each, 16-deep slices in two shared-memory
// buffers: the next slice is on its way from global memory while one is
// multiplied.  MI = 8 (128 x 128 tiles) reads 16 values from shared memory
// per 64 multiply-adds and is bound by the fp32 pipe; MI = 4 (64 x 64 tiles)
// is for shapes whose larger tiles would leave SMs idle or rows empty.  Groups of
// few rows have kernels of their own, which stream the matrices.
// Multiply-adds are issued in pairs (fma.rn.f32x2, each lane rounded as an
// fma.rn.f32).
//
// The weight gradient, whose reduction is a group's rows, sums 128 products at
// a time and adds these sums up apart, which keeps the rounding of long groups
// near sqrt(128) rather than sqrt(rows) half steps (its kernel for few rows adds 8
// at a time to what lies in memory).  The other two sum a
// matrix's width in one chain, as two blocks per SM leave no registers for
// more (8 x 1024 x 2048 x 1024: 54 TFLOP/s; with apart sums 6% less).
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

// tile_start[g + 1], the tiles of group g, become the number up to and with
// group g.  Every thread of the block calls it, behind a barrier; it ends with
// one.
__device__ __forceinline__ void scan_tiles(int32_t* tile_start, int groups, int tid) {
  if (tid < 32) {
    // a run of groups per lane
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
}
__device__ __forceinline__ int group_of_tile(const int32_t* tile_start, int groups, int tile) {
  int lo = 0, hi = groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tile_start[mid] <= tile) lo = mid; else hi = mid - 1;
  }
  return lo;
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
  scan_tiles(tile_start, groups, tid);
  const int total = tile_start[groups];
  const int tx = tid & 15, ty = tid >> 4;
  const int64_t lda = FWD ? k : n, ldb = k;
  const bool vec_a = lda % 4 == 0, vec_b = ldb % 4 == 0;
  for (int tile = blockIdx.x / parts; tile < total; tile += gridDim.x / parts) {
    const int g = group_of_tile(tile_start, groups, tile);
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
    // dW: four neighbours in one store where rows are whole 16-byte pieces (the
    // other two, whose outputs are few beside their reductions, lose registers)
    auto store4 = [&](int i, int j, F2 lo, F2 hi) {
      if (N % 4 != 0 || accumulate) {
        store(i, j, lo);
        store(i, j + 1, hi);
        return;
      }
      const int m = m0 + (i >> 2) * 64 + ty * 4 + (i & 3), c = n0 + (j >> 1) * 64 + tx * 4;
      if (m >= M || c >= N) return;
      const float2 v = both(lo), w = both(hi);
      *reinterpret_cast<float4*>(out + (static_cast<int64_t>(g) * n + m) * k + c) =
          make_float4(v.x, v.y, w.x, w.y);
    };
    if (!SPLIT) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < MI / 2; ++j) {
          if (!DW) {
            store(i, j, acc[i][j]);
          } else {
            acc[i][j] = add2(sum[i][j], acc[i][j]);
            if (j & 1) store4(i, j - 1, acc[i][j - 1], acc[i][j]);
          }
        }
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
      __syncwarp();
      cluster_sync_all();
    }
  }
}

// Few rows per group: a matrix is streamed once for every kFewR rows of its
// group, and one pass is bound by memory (40 groups of one row of 2392 x 1528:
// forward 109 us, 5.4 TB/s, input gradient 121; in 64 x 64 tiles, almost all of
// each of them empty, 594 and 694).  More passes than one are not: 16 groups of 16
// rows of 2048 x 1024 68 and 59 us, of 30 rows 146 (in tiles) and 102, where the
// bytes take 21.
constexpr int kFewR = 8;
constexpr int kFewK = 1024;  // reduction steps of the rows in shared memory at a time

// The tiles of kFewR rows by `blocks` of every group, and the groups' rows.
__device__ __forceinline__ void few_tiles(const int32_t* offsets, int groups, int rows, int blocks,
                                          int32_t* tile_start, int32_t* row0s, int32_t* rowsg,
                                          int tid) {
  group_spans(offsets, groups, rows, tile_start, tid, 256);
  for (int g = tid; g < groups; g += 256) {
    row0s[g] = tile_start[g];
    rowsg[g] = tile_start[g + 1] - tile_start[g];
  }
  __syncthreads();
  for (int g = tid; g < groups; g += 256)
    tile_start[g + 1] = (rowsg[g] + kFewR - 1) / kFewR * blocks;
  __syncthreads();
  scan_tiles(tile_start, groups, tid);
}

// Forward: a warp takes four rows of W_g, its lanes along k, and R rows of the
// group.  VEC: rows of whole 16-byte pieces, loaded without conditions, so that
// they go out together.
template <int R, bool VEC, typename Fill>
__device__ __forceinline__ void few_dot(const float* w, int n, int k, int n0,
                                        const float (*xs)[kFewK], Fill fill, int here, int lane,
                                        float* y) {
  const float* wr[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)  // past the last row: the last one, not stored
    wr[i] = w + static_cast<int64_t>(min(n0 + i, n - 1)) * k;
  F2 acc[4][R];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < R; ++r) acc[i][r] = 0;
  for (int k0 = 0; k0 < k; k0 += kFewK) {
    const int len = min(kFewK, k - k0);
    fill(k0, len);
#pragma unroll(R > 2 ? 2 : 4)
    for (int c = lane * 4; c < len; c += 128) {
      F2 v[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* from = wr[i] + k0 + c;
        const float4 f = VEC ? *reinterpret_cast<const float4*>(from) : load4(from, len - c, false);
        v[i][0] = pair(f.x, f.y);
        v[i][1] = pair(f.z, f.w);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&xs[r][c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][r] = fma2(v[i][1], x.y, fma2(v[i][0], x.x, acc[i][r]));
      }
    }
  }
  // 4 R sums over the lanes, of which lane l ends with number l % (4 R)
  float v[4 * R];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float2 f = both(acc[i][r]);
      v[i * R + r] = f.x + f.y;
    }
#pragma unroll
  for (int o = 2 * R; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
#pragma unroll
  for (int o = 4 * R; o < 32; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  const int r = lane % R, c = n0 + lane / R;
  if (lane < 4 * R && r < here && c < n) y[static_cast<int64_t>(r) * n + c] = v[0];
}

template <bool VEC>
__global__ void __launch_bounds__(256, 2)
grouped_f32_few_fwd_kernel(const float* __restrict__ x, const float* __restrict__ w,
                           const int32_t* __restrict__ offsets, int groups, int rows, int n, int k,
                           float* __restrict__ y) {
  __shared__ __align__(16) float xs[kFewR][kFewK];
  __shared__ int32_t tile_start[kMaxG + 1], row0s[kMaxG], rowsg[kMaxG];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nb = (n + 31) / 32;
  few_tiles(offsets, groups, rows, nb, tile_start, row0s, rowsg, tid);
  const int64_t total = tile_start[groups];
  // a run of tiles, so that most of them find their rows in place
  const int end = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
  int64_t in_place = -1;  // first row of what xs holds
  for (int tile = static_cast<int>(total * blockIdx.x / gridDim.x); tile < end; ++tile) {
    const int g = group_of_tile(tile_start, groups, tile);
    const int local = tile - tile_start[g], chunk = local / nb;
    const int n0 = (local - chunk * nb) * 32 + warp * 4;
    const int64_t r0 = static_cast<int64_t>(row0s[g]) + chunk * kFewR;
    const int here = min(kFewR, rowsg[g] - chunk * kFewR);
    auto fill = [&](int k0, int len) {
      if (k <= kFewK && in_place == r0) return;
      __syncthreads();  // what xs held has been used
      for (int e = tid; e < here * (kFewK / 4); e += 256) {
        const int r = e / (kFewK / 4), c = e % (kFewK / 4) * 4;
        if (c < len)
          *reinterpret_cast<float4*>(&xs[r][c]) = load4(x + (r0 + r) * k + k0 + c, len - c, VEC);
      }
      __syncthreads();
      in_place = r0;
    };
    const float* wg = w + static_cast<int64_t>(g) * n * k;
    float* to = y + r0 * n;
    if (here == 1) few_dot<1, VEC>(wg, n, k, n0, xs, fill, here, lane, to);
    else if (here == 2) few_dot<2, VEC>(wg, n, k, n0, xs, fill, here, lane, to);
    else if (here <= 4) few_dot<4, VEC>(wg, n, k, n0, xs, fill, here, lane, to);
    else few_dot<kFewR, VEC>(wg, n, k, n0, xs, fill, here, lane, to);
  }
}

// Input gradient: a lane takes four columns of W_g, the block's warps its rows
// in turn.  The CTAs of a cluster take a part of the rows each.
template <int R, bool VEC>
__device__ __forceinline__ void few_axpy(const float* wc, int64_t ld, int left,
                                         const float (*ds)[kFewR], int len, int warp,
                                         F2 (&acc)[kFewR][2]) {
#pragma unroll 8
  for (int j = warp; j < len; j += 8) {
    const float4 v = VEC ? *reinterpret_cast<const float4*>(wc + j * ld) : load4(wc + j * ld, left, false);
    const F2 w0 = pair(v.x, v.y), w1 = pair(v.z, v.w);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const F2 d = pair(ds[j][r], ds[j][r]);
      acc[r][0] = fma2(d, w0, acc[r][0]);
      acc[r][1] = fma2(d, w1, acc[r][1]);
    }
  }
}

template <bool VEC>
__global__ void __launch_bounds__(256, 2)
grouped_f32_few_dx_kernel(const float* __restrict__ dy, const float* __restrict__ w,
                          const int32_t* __restrict__ offsets, int groups, int rows, int n, int k,
                          float* __restrict__ dx) {
  // the rows' slice, then the warps' sums, then in warp 0's place the block's
  __shared__ __align__(16) float buf[8][kFewR][128];
  static_assert(sizeof(buf) >= kFewK * kFewR * 4, "the slice takes the sums' place");
  float (*const ds)[kFewR] = reinterpret_cast<float (*)[kFewR]>(&buf[0][0][0]);
  __shared__ int32_t tile_start[kMaxG + 1], row0s[kMaxG], rowsg[kMaxG];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = static_cast<int>(cluster_ctarank());
  const int parts = static_cast<int>(gridDim.x / num_clusters_x());
  const int per = (n + parts - 1) / parts;
  const int nbeg = min(part * per, n), nend = min(nbeg + per, n);
  const int kb = (k + 127) / 128;
  few_tiles(offsets, groups, rows, kb, tile_start, row0s, rowsg, tid);
  const int total = tile_start[groups];
  for (int tile = blockIdx.x / parts; tile < total; tile += gridDim.x / parts) {
    const int g = group_of_tile(tile_start, groups, tile);
    const int local = tile - tile_start[g], chunk = local / kb;
    const int c0 = (local - chunk * kb) * 128 + lane * 4;
    const int64_t r0 = static_cast<int64_t>(row0s[g]) + chunk * kFewR;
    const int here = min(kFewR, rowsg[g] - chunk * kFewR);
    // VEC: lanes past the row take its first columns, which they do not store
    const float* wg = w + static_cast<int64_t>(g) * n * k + (VEC && c0 >= k ? 0 : c0);
    F2 acc[kFewR][2];
#pragma unroll
    for (int r = 0; r < kFewR; ++r) acc[r][0] = acc[r][1] = 0;
    for (int j0 = nbeg; j0 < nend; j0 += kFewK) {
      const int len = min(kFewK, nend - j0);
      __syncthreads();  // what was in the buffer has been used
      for (int e = tid; e < here * kFewK; e += 256) {
        const int r = e / kFewK, j = e % kFewK;
        if (j < len) ds[j][r] = dy[(r0 + r) * n + j0 + j];
      }
      __syncthreads();
      const float* wc = wg + static_cast<int64_t>(j0) * k;
      if (here == 1) few_axpy<1, VEC>(wc, k, k - c0, ds, len, warp, acc);
      else if (here == 2) few_axpy<2, VEC>(wc, k, k - c0, ds, len, warp, acc);
      else if (here <= 4) few_axpy<4, VEC>(wc, k, k - c0, ds, len, warp, acc);
      else few_axpy<kFewR, VEC>(wc, k, k - c0, ds, len, warp, acc);
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kFewR; ++r)
      *reinterpret_cast<ulonglong2*>(&buf[warp][r][lane * 4]) = make_ulonglong2(acc[r][0], acc[r][1]);
    __syncthreads();
    // warp r adds row r up, over the warps and then over the cluster, in order
    float4 s = *reinterpret_cast<const float4*>(&buf[0][warp][lane * 4]);
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(&buf[i][warp][lane * 4]);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    if (parts > 1) {
      *reinterpret_cast<float4*>(&buf[0][warp][lane * 4]) = s;
      cluster_sync_all();
      const uint32_t at = smem_addr(&buf[0][warp][lane * 4]);
      if (warp % parts == part) {
        F2 a = 0, b = 0;
        for (int p = 0; p < parts; ++p) {
          const uint32_t from = map_to_cta(at, static_cast<uint32_t>(p));
          a = add2(a, ld_cluster_f2(from));
          b = add2(b, ld_cluster_f2(from + 8));
        }
        const float2 lo = both(a), hi = both(b);
        s = make_float4(lo.x, lo.y, hi.x, hi.y);
      }
    }
    if (warp < here && warp % parts == part) {
      float* to = dx + (r0 + warp) * k + c0;
      if (VEC) {
        if (c0 < k) *reinterpret_cast<float4*>(to) = s;
      } else {
        if (c0 < k) to[0] = s.x;
        if (c0 + 1 < k) to[1] = s.y;
        if (c0 + 2 < k) to[2] = s.z;
        if (c0 + 3 < k) to[3] = s.w;
      }
    }
    __syncwarp();
    if (parts > 1) cluster_sync_all();  // the sums have been read
  }
}

// Weight gradient: a lane takes four columns of dW_g, the block's warps its rows
// in turn, kFewN of them a tile; bound by the writes (40 groups of one row of
// 2392 x 1528: 95 us, 6.1 TB/s; in 64 x 64 tiles 308).
constexpr int kFewN = 128;

template <bool VEC>
__global__ void __launch_bounds__(256, 3)
grouped_f32_few_dw_kernel(const float* __restrict__ dy, const float* __restrict__ x,
                          const int32_t* __restrict__ offsets, int groups, int rows, int n, int k,
                          float* __restrict__ dw, bool accumulate) {
  __shared__ __align__(16) float ds[kFewN][kFewR];
  __shared__ int32_t span[kMaxG + 1];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  group_spans(offsets, groups, rows, span, tid, 256);
  const int kb = (k + 127) / 128, nb = (n + kFewN - 1) / kFewN;
  const int64_t total = static_cast<int64_t>(groups) * kb * nb;
  for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
    const int g = static_cast<int>(tile / (kb * nb)), local = static_cast<int>(tile % (kb * nb));
    const int n0 = local / kb * kFewN, c0 = local % kb * 128 + lane * 4;
    const int left = min(kFewN, n - n0);
    const int64_t r0 = span[g];
    const int len = span[g + 1] - span[g];
    float* to = dw + (static_cast<int64_t>(g) * n + n0) * k + c0;
    // more rows than kFewR are added in turn to what lies there
    bool add = accumulate;
    for (int c = 0; c < max(len, add ? 0 : 1); c += kFewR, add = true) {
      const int here = min(kFewR, len - c);
      __syncthreads();  // the slice before has been used
      for (int e = tid; e < kFewR * kFewN; e += 256) {
        const int r = e / kFewN, j = e % kFewN;
        ds[j][r] = r < here && j < left ? dy[(r0 + c + r) * n + n0 + j] : 0.0f;
      }
      F2 v[kFewR][2];
#pragma unroll
      for (int r = 0; r < kFewR; ++r) {
        float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < here) f = load4(x + (r0 + c + r) * k + c0, k - c0, VEC);
        v[r][0] = pair(f.x, f.y);
        v[r][1] = pair(f.z, f.w);
      }
      __syncthreads();
#pragma unroll 2
      for (int j = warp; j < left; j += 8) {
        float* at = to + static_cast<int64_t>(j) * k;
        F2 s0 = 0, s1 = 0;
#pragma unroll
        for (int r = 0; r < kFewR; ++r) {
          const F2 d = pair(ds[j][r], ds[j][r]);
          s0 = fma2(d, v[r][0], s0);
          s1 = fma2(d, v[r][1], s1);
        }
        if (add) {
          const float4 f = load4(at, k - c0, VEC);
          s0 = add2(s0, pair(f.x, f.y));
          s1 = add2(s1, pair(f.z, f.w));
        }
        const float2 lo = both(s0), hi = both(s1);
        if (VEC) {
          if (c0 < k) *reinterpret_cast<float4*>(at) = make_float4(lo.x, lo.y, hi.x, hi.y);
        } else {
          if (c0 < k) at[0] = lo.x;
          if (c0 + 1 < k) at[1] = lo.y;
          if (c0 + 2 < k) at[2] = hi.x;
          if (c0 + 3 < k) at[3] = hi.y;
        }
      }
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
  // Few rows per group, on average, which is all that the host knows.  A group far
  // above it is the same work in passes of 8 rows: 64 groups of 1024 x 1024, all
  // of 1500 rows in one, forward 131 us (142 for that group alone), input gradient
  // 106 (150), weight gradient 191 (104).  (16 groups of 2048 x 1024 forward, 24 rows: 95
  // us for 145 in tiles, 40 rows: 154 for 147; input gradient, 24: 88 for 143, 40:
  // 145 for 145).
  if (dir != kGroupedDw && rows <= (dir == kGroupedFwd ? 24ll : 32ll) * groups) {
    const int64_t blocks = (N + (dir == kGroupedFwd ? 31 : 127)) / (dir == kGroupedFwd ? 32 : 128);
    const int64_t most = blocks * (rows / kFewR + some);
    int parts = 1;
    if (dir == kGroupedDx)
      while (parts < 8 && most * parts < 2ll * sms && n >= 128 * parts) parts *= 2;
    const int64_t fit = 2ll * sms / parts;
    const int grid = static_cast<int>(most < fit ? most : fit) * parts;
    auto kern = dir == kGroupedFwd ? (k % 4 == 0 ? grouped_f32_few_fwd_kernel<true>
                                                 : grouped_f32_few_fwd_kernel<false>)
                                   : (k % 4 == 0 ? grouped_f32_few_dx_kernel<true>
                                                 : grouped_f32_few_dx_kernel<false>);
    return launch_k(kern, dim3(grid), dim3(256), 0, st, parts, a, b, offsets, groups,
                    static_cast<int>(rows), n, k, out);
  }
  // (the same, 8 rows: 33 us for 56; 16 rows: 66 for 57)
  if (dir == kGroupedDw && rows <= 8ll * groups) {
    const int64_t most = static_cast<int64_t>(groups) * ((k + 127) / 128) * ((n + kFewN - 1) / kFewN);
    auto kern = k % 4 == 0 ? grouped_f32_few_dw_kernel<true> : grouped_f32_few_dw_kernel<false>;
    return launch_k(kern, dim3(static_cast<unsigned>(most < 3ll * sms ? most : 3ll * sms)), dim3(256),
                    0, st, 1, a, b, offsets, groups, static_cast<int>(rows), n, k, out, accumulate);
  }
  auto tiles = [&](int T) {
    const int64_t nt = (N + T - 1) / T;
    return nt * (dir == kGroupedDw ? static_cast<int64_t>(groups) * ((n + T - 1) / T)
                                   : (rows + T - 1) / T + some);
  };
  // The tile size whose most loaded SM is done first: a 128 x 128 tile is four
  // 64 x 64 ones, which take some 1.45 times as long for the same work (8 x 1024 x
  // 2048 x 1024: forward 633 against 1015 us, dX 758 and 976, dW 689 and 968; 16 x
  // 300 x 512 x 512, part empty in the large ones: 96 against 93, 100 and 91, 64
  // and 86).
  auto rounds = [&](int T) { return (tiles(T) + sms - 1) / sms; };
  const bool fill = dir == kGroupedDw || rows >= 96 * some;  // groups fill the large ones
  if (fill && 4.0 * rounds(128) <= 1.45 * rounds(64))
    return launch_tiles<8, false>(dir, a, b, offsets, groups, rows, n, k, out, accumulate,
                                  tiles(128), dir == kGroupedDw ? sms : 2 * sms, 1, st);
  // Few tiles: clusters of up to 8 CTAs share a tile's reduction, four slices
  // each at least (6 x 357 rows of 248 x 656 forward: 30 us, without 46).
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
