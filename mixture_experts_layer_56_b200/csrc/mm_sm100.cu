// Matrix products of the training operators on CTA pairs (tcgen05
// cta_group::2): D[m, n] = sum_k A(m, k) B(n, k), fp32 accumulation in TMEM.
//
//   forward          Y[r]  = X[r] W_g^T      NT, ragged rows
//   input gradient   dX[r] = dY[r] W_g       NN, ragged rows
//   (few rows)       the same, transposed    NT and TT, ragged columns
//   weight gradient  dW_g  = dY_g^T X_g      TN, ragged reduction
//   Newton-Schulz    X X^T, A A, B X         any, a batch of equal matrices
//
// No operand is transposed in memory.  A TMA box is 64 elements (128 bytes,
// swizzled) of the memory rows; where those run along m or n instead of k the
// box holds 64 k rows of one 64-wide slice, and the MMA's descriptor and the
// instruction's major bit say so.
//
// A tile is 256 x 256 at most, its rows split over the two SMs of a cluster: each CTA
// loads its 128 rows of A and its half of B's 256 rows, and the leader issues
// M = 256, N = 256 MMAs for both.  Five 32 KB stages per CTA; the accumulator
// is double-buffered in TMEM (2 x 256 columns), so that the epilogue of one
// tile runs under the MMAs of the next.  Warps: 0 TMA, 1 MMA, 2 TMEM, 3 the
// ragged reduction's zeroing, 4-11 epilogue.
//
// Ragged rows need no masking: a tile may run past its group's last row, and
// the rows it computes there are not stored.  A ragged reduction does: the
// last k-block of a group holds the first rows of the next one (or rows that
// nobody owns, which may hold NaN).  MMA steps of 16 that hold none of the
// group's rows are not issued, and warp 3 of each CTA zeroes the rest of the
// last one in both operands in shared memory before the MMAs may read it.
//
// Bound by the tensor cores (full groups), whose rate under long loads is the
// power cap's: 16 groups of 4096 rows of 2048 x 2048 forward 444 us in a loop,
// 1240 TFLOP/s, and 375 rested (the library's best single product of 8192 cubed:
// 1369 and 1643 TFLOP/s); 63 groups of some 910 rows of 1792 x 1280 270 us, 975
// TFLOP/s, a last tile per group being part empty; the weight gradient at 1784 x
// 1288 362 us, whose row pitches are no multiple of 128 bytes and cost the TMA
// loads and L2 a third.  A float32 weight gradient costs its stores (64 groups of
// 12 rows of 2816 x 2048: 253 us, 148 in bf16, of 227 and 113 for the bytes); one
// that is added to reads the old values a piece at a time behind the accumulator
// and takes 1744 there, 1801 for 1044 with 1536 rows per group.  Its reduction is
// not split: one group of 16384 rows of 256 x 256 is four tiles, 72 us.  Bound by memory (few rows per group): 8 tokens x 6 of 64
// experts of 2816 x 2048 63 us, 0.98 of the rate of a copy.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <mutex>

#include "common.cuh"
#include "f32x2.cuh"
#include "group_spans.cuh"
#include "mm_sm100.h"
#include "mm_ptx.cuh"

namespace moe {
namespace sm100 {

namespace {

constexpr int kTile = 256;      // rows, and most columns, of a pair's tile
constexpr int kHalf = 128;      // rows of a tile per CTA
constexpr int kKB = 64;         // k-block
constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kStagePitch = 128 + 16;  // staging row: 128 bytes, padded off the bank period
constexpr int kWarpStage = 32 * kStagePitch;
constexpr int kWarpDiag = 128 * 4;  // a diagonal's values over an epilogue warp's columns
constexpr uint32_t kSliceBytes = 64 * kKB * 2;  // an MN-major 64-wide slice
constexpr uint64_t kLandNs = 1000000;  // copies in flight after an expired wait: 1 ms
constexpr int kColChunk = 8;  // N tiles that a group's row blocks sweep together

// Shared memory with BR rows of B per CTA in a stage.
template <int BR>
struct Stage {
  static constexpr uint32_t kA = kHalf * kKB * 2;
  static constexpr uint32_t kB = BR * kKB * 2;
  static constexpr uint32_t kBytes = kA + kB;
  // what 227 KB hold beside the epilogue's staging and 5 KB of barriers,
  // group tables and alignment
  static constexpr int kCount = (227 * 1024 - 5120 - kEpiWarps * (kWarpStage + kWarpDiag)) / kBytes;
  static constexpr int kSmem = kCount * kBytes + kEpiWarps * (kWarpStage + kWarpDiag) + 1024;
  static_assert(kCount >= 4 && kCount <= 16, "the issued-stage masks hold 32");
};

// 32 rows (lane r holds row r, NV 16-byte pieces) written to global memory as
// whole row segments through the warp's staging area: `dst` is where row 0
// goes, `pitch` the bytes between rows; of the rows `rows` are written, and of
// the pieces those below `pieces` (the others lie outside the matrix).
template <int NV, typename Put>
__device__ __forceinline__ void store_rows(uint8_t* stage, const uint4* v, void* dst, int64_t pitch,
                                           int rows, int pieces, int lane, Put put) {
  constexpr int RPI = 32 / NV;
#pragma unroll
  for (int c = 0; c < NV; ++c)
    *reinterpret_cast<uint4*>(stage + lane * kStagePitch + c * 16) = v[c];
  __syncwarp();
  const int c = lane % NV, r0 = lane / NV;
  uint8_t* at = static_cast<uint8_t*>(dst) + r0 * pitch + c * 16;
  if (c >= pieces) rows = 0;
#pragma unroll
  for (int it = 0; it < NV; ++it) {
    const uint4 x = *reinterpret_cast<const uint4*>(stage + (it * RPI + r0) * kStagePitch + c * 16);
    if (it * RPI + r0 < rows) put(reinterpret_cast<uint4*>(at), x);
    at += RPI * pitch;
  }
  __syncwarp();
}

// A warp's 32 rows of 32 fp16 values as whole row segments: piece `it` of a
// lane is row it * 8 + lane / 4, columns 8 (lane % 4) .. + 7.  Rows at or past
// `rows` and pieces past the matrix give zeros.
struct RowFetch {
  uint4 v[4];
  __device__ __forceinline__ void fetch(const __half* base, int64_t ld, int rows, int pieces,
                                        int lane) {
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int row = it * 8 + lane / 4, c = lane % 4;
      v[it] = row < rows && c < pieces
                  ? *reinterpret_cast<const uint4*>(base + row * ld + c * 8)
                  : make_uint4(0, 0, 0, 0);
    }
  }
};

struct PutPlain {
  __device__ __forceinline__ void operator()(uint4* p, uint4 x) const { *p = x; }
};
struct PutAddF32 {
  __device__ __forceinline__ void operator()(uint4* p, uint4 x) const {
    float4 o = *reinterpret_cast<float4*>(p);
    o.x += __uint_as_float(x.x);
    o.y += __uint_as_float(x.y);
    o.z += __uint_as_float(x.z);
    o.w += __uint_as_float(x.w);
    *reinterpret_cast<float4*>(p) = o;
  }
};

__device__ __forceinline__ uint4 pack_half8(const float* x) {
  uint4 v;
  __half2* h = reinterpret_cast<__half2*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
  return v;
}
// eight fp16 values and four pairs
__device__ __forceinline__ void half_pairs(const uint4& v, F2* x) {
  const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    x[i] = pair(f.x, f.y);
  }
}
__device__ __forceinline__ uint4 pairs_half(const F2* x) {
  uint4 v;
  __half2* h = reinterpret_cast<__half2*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = both(x[i]);
    h[i] = __floats2half2_rn(f.x, f.y);
  }
  return v;
}

struct Tile {
  int g, m_blk, n_blk;
  int row0;  // ragged: the group's first row
  int rows;  // rows of D of the group (ragged rows, or m), or the ragged reduction's length
  int len;   // of the reduction
  int nkb;   // k-blocks
  int col0;  // first column of D
  int ncols; // of the MMA
};

template <int LAYOUT, int SCHED, int EPI, bool FP16, int BR>
__global__ void __launch_bounds__(kThreads, 1)
mm_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmTail, const MmArgs args) {
  constexpr bool A_MN = LAYOUT == kMmTN || LAYOUT == kMmTT;
  constexpr bool B_MN = LAYOUT == kMmNN || LAYOUT == kMmTN;
  constexpr bool RAG_M = SCHED == kMmRaggedM;
  constexpr bool RAG_K = SCHED == kMmRaggedK;
  constexpr bool RAG_N = SCHED == kMmRaggedN;
  constexpr bool SYM = SCHED == kMmBatchSym;
  constexpr uint32_t A_BYTES = Stage<BR>::kA;
  constexpr uint32_t B_BYTES = Stage<BR>::kB;
  constexpr uint32_t STAGE_BYTES = Stage<BR>::kBytes;
  constexpr int STAGES = Stage<BR>::kCount;
  constexpr uint32_t TMEM_COLS = 2 * kTile;
  static_assert(!B_MN || BR == 128, "an MN-major B comes in up to two slices");
  constexpr uint16_t kBoth = 0x3;

  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[3 * STAGES + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int32_t tile_start[kMmMaxGroups + 1];
  __shared__ int32_t grp_row0[kMmMaxGroups];
  __shared__ int32_t grp_rows[kMmMaxGroups];
  __shared__ int16_t grp_order[kMmMaxGroups];  // ragged reductions: longest first

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t smem_base = smem_addr(smem);
  const uint32_t bar_base = smem_addr(bars);
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
  auto land_bar = [&](int s) { return bar_base + 8u * (2 * STAGES + s); };
  auto tfull_bar = [&](int a) { return bar_base + 8u * (3 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar_base + 8u * (3 * STAGES + 2 + a); };
  const uint32_t drain_bar = bar_base + 8u * (3 * STAGES + 4);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster = static_cast<int>(cluster_id_x());
  const int nclusters = static_cast<int>(num_clusters_x());
  const int G = args.groups;
  const int tn = args.tn;  // columns of a tile
  const int nt = (args.n + tn - 1) / tn;
  volatile int* abort_p = &abort_flag;

  // ---- setup --------------------------------------------------------------
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      // the leader's arrive (+ both CTAs' bytes); with a ragged reduction
      // either CTA arrives, its rows zeroed where the k-block is a group's last
      mbar_init(full_bar(s), RAG_K ? 2 : 1);
      mbar_init(empty_bar(s), 1);  // one multicast commit
      mbar_init(land_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 2 * kEpiWarps);  // epilogue warps of both CTAs (leader's copy)
    }
    mbar_init(drain_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
    fence_async_shared();
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_addr(&tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();  // barrier inits and TMEM allocations visible to the pair
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  // all of the above runs while the kernel before this one ends
  pdl_wait();
  pdl_trigger();
  if (RAG_M || RAG_K || RAG_N) {
    group_spans(args.offsets, G, args.rows, tile_start, tid, kThreads);
    for (int g = tid; g < G; g += kThreads) {
      grp_row0[g] = tile_start[g];
      grp_rows[g] = tile_start[g + 1] - tile_start[g];
    }
    __syncthreads();
    for (int g = tid; g < G; g += kThreads)
      tile_start[g + 1] = RAG_N ? ((grp_rows[g] + tn - 1) / tn) * ((args.m + kTile - 1) / kTile)
                                : ((grp_rows[g] + kTile - 1) / kTile) * nt;
    __syncthreads();
    if (RAG_K) {
      // tiles of equal length run side by side, the longest first
      for (int g = tid; g < G; g += kThreads) {
        int before = 0;
        for (int i = 0; i < G; ++i)
          before += grp_rows[i] > grp_rows[g] || (grp_rows[i] == grp_rows[g] && i < g);
        grp_order[before] = static_cast<int16_t>(g);
      }
    }
    if ((RAG_M || RAG_N) && warp == 0) {
      const int per = (G + 31) / 32;
      const int beg = min(lane * per, G);
      const int end = min(beg + per, G);
      int sum = 0;
      for (int i = beg; i < end; ++i) sum += tile_start[i + 1];
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      int run = incl - sum;
      for (int i = beg; i < end; ++i) {
        run += tile_start[i + 1];
        tile_start[i + 1] = run;
      }
      if (lane == 0) tile_start[0] = 0;
    }
    __syncthreads();
  }
  const int mt_fixed = RAG_M ? 0 : (args.m + kTile - 1) / kTile;
  // a symmetric product's block of rows mb has the column tiles from its
  // diagonal block on, each 1 / per_blk of a block wide (above the diagonal,
  // as columns come in steps of 32 where a block of few rows costs a whole one)
  const int per_blk = kTile / tn;
  const int per_group = mt_fixed * nt - (SYM ? per_blk * (mt_fixed * (mt_fixed - 1) / 2) : 0);
  const int total_tiles = RAG_M || RAG_N ? tile_start[G] : G * per_group;

  // position v of this pair's sequence cluster, cluster + nclusters, ...
  auto tile_of = [&](int v) {
    Tile ti;
    int t = v;
    if (RAG_K) {
      // Every other round backwards: a round's tiles get shorter from first
      // to last, and so no pair has the longer one of every round.
      const int round = v / nclusters;
      const int first = round * nclusters;
      const int here = min(nclusters, total_tiles - first);
      if (round & 1) t = first + here - 1 - (v - first);
    }
    if (RAG_M || RAG_N) {
      int lo = 0, hi = G - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tile_start[mid] <= t) lo = mid; else hi = mid - 1;
      }
      ti.g = lo;
      const int local = t - tile_start[lo];
      ti.row0 = grp_row0[lo];
      ti.rows = grp_rows[lo];
      // the row blocks sweep kColChunk tiles along the matrix together, so that
      // the pairs in flight share a slice of the group's matrix in L2
      const int along = RAG_N ? (args.m + kTile - 1) / kTile : nt;
      const int blocks = (tile_start[lo + 1] - tile_start[lo]) / along;
      const int cw = min(kColChunk, along);
      const int c = local / (cw * blocks);
      const int rem = local - c * cw * blocks;
      const int wc = min(cw, along - c * cw);
      const int block = rem / wc;
      const int at = c * cw + (rem - block * wc);
      ti.m_blk = RAG_N ? at : block;
      ti.n_blk = RAG_N ? block : at;
    } else {
      ti.g = t / per_group;
      const int local = t - ti.g * per_group;
      if (RAG_K) ti.g = grp_order[ti.g];
      if (SYM) {
        // the tiles before block row mb
        auto before = [&](int mb) { return mb * nt - per_blk * (mb * (mb - 1) / 2); };
        const float h = nt + 0.5f * per_blk;
        int mb = static_cast<int>((h - sqrtf(fmaxf(h * h - 2.0f * per_blk * local, 0.0f))) / per_blk);
        mb = min(max(mb, 0), mt_fixed - 1);
        while (mb > 0 && before(mb) > local) --mb;
        while (mb + 1 < mt_fixed && before(mb + 1) <= local) ++mb;
        ti.m_blk = mb;
        ti.n_blk = per_blk * mb + local - before(mb);
      } else {
        ti.m_blk = local / nt;
        ti.n_blk = local - ti.m_blk * nt;
      }
      ti.row0 = RAG_K ? grp_row0[ti.g] : 0;
      ti.rows = RAG_K ? grp_rows[ti.g] : args.m;
    }
    ti.len = RAG_K ? ti.rows : args.k;
    ti.nkb = (ti.len + kKB - 1) / kKB;
    ti.col0 = ti.n_blk * tn;
    // the MMA's width: the last column tile's, in steps of 32 (what makes a
    // group's last rows cheaper as columns than in a tile of 256 rows)
    ti.ncols = min(tn, ((RAG_N ? ti.rows : args.n) - ti.col0 + 31) & ~31);
    return ti;
  };
  // whether CTA `r` of the pair has rows in the tile
  auto has_rows = [&](const Tile& ti, int r) {
    return ti.m_blk * kTile + r * kHalf < (RAG_K || RAG_N ? args.m : ti.rows);
  };

  // the same with every field known to be uniform across the warp
  auto uniform_tile = [&](int v) {
    Tile ti = tile_of(v);
    ti.g = uniform(ti.g);
    ti.m_blk = uniform(ti.m_blk);
    ti.n_blk = uniform(ti.n_blk);
    ti.row0 = uniform(ti.row0);
    ti.rows = uniform(ti.rows);
    ti.len = uniform(ti.len);
    ti.nkb = uniform(ti.nkb);
    ti.col0 = uniform(ti.col0);
    ti.ncols = uniform(ti.ncols);
    return ti;
  };

  if (warp == 0) {
    // ---------------------------------------------------- TMA producer ----
    int stage = 0;
    uint32_t phase = 0, issued = 0, issued_parity = 0;
    bool ok = true;
    for (int tile = cluster; tile < total_tiles && ok; tile += nclusters) {
      const Tile ti = uniform_tile(tile);
      const int m0 = ti.m_blk * kTile + static_cast<int>(rank) * kHalf + (RAG_M ? ti.row0 : 0);
      const int n0 = ti.col0 + static_cast<int>(rank) * (ti.ncols / 2) + (RAG_N ? ti.row0 : 0);
      // a CTA without rows leaves its part of A as it is: what the MMA makes
      // of it is not stored
      const bool mine = has_rows(ti, static_cast<int>(rank));
      // of an MN-major B the slices that the tile's width takes
      const bool two = !B_MN || ti.ncols > 128;
      // of a ragged group's last rows boxes of 32
      const bool tail = RAG_N && BR == 128 && ti.ncols < tn;
      const int boxes = tail ? (ti.ncols + 63) / 64 : 0;
      const uint32_t b_bytes = B_MN   ? (two ? B_BYTES : kSliceBytes)
                               : tail ? static_cast<uint32_t>(boxes) * (32 * kKB * 2)
                                      : static_cast<uint32_t>(tn / 2) * (kKB * 2);
      const uint32_t bytes = (mine ? A_BYTES : 0) + b_bytes;
      const uint32_t pair_bytes = 2 * b_bytes + A_BYTES + (has_rows(ti, 1) ? A_BYTES : 0);
      const int za = RAG_M || RAG_K ? 0 : ti.g;
      const int zb = RAG_K || RAG_N ? 0 : ti.g;
      int k0 = RAG_K ? ti.row0 : 0;
      for (int kb = 0; kb < ti.nkb; ++kb, k0 += kKB) {
        ok = __all_sync(0xffffffffu,
                        wait_bounded(empty_bar(stage), phase ^ 1u, abort_p, args.status));
        if (!ok) break;
        const uint32_t sa = smem_base + stage * STAGE_BYTES;
        const uint32_t sb = sa + A_BYTES;
        // a ragged group's last, partial k-block lands on this CTA's own
        // barrier, where warp 3 takes it over
        const bool partial = RAG_K && kb == ti.nkb - 1 && (ti.rows & 15) != 0;
        const uint32_t fb = partial || leader ? (partial ? land_bar(stage) : full_bar(stage))
                                              : map_to_cta(full_bar(stage), 0);
        if (elect_lane()) {
          if (partial) mbar_arrive_expect_tx(fb, bytes);
          else if (leader) mbar_arrive_expect_tx(fb, pair_bytes);
          else if (RAG_K) mbar_arrive_cluster(fb);
          if (mine) {
            if (A_MN) {
              tma_load_3d_pair(sa, &tmA, fb, m0, k0, za);
              tma_load_3d_pair(sa + kSliceBytes, &tmA, fb, m0 + 64, k0, za);
            } else {
              tma_load_3d_pair(sa, &tmA, fb, k0, m0, za);
            }
          }
          if (B_MN) {
            tma_load_3d_pair(sb, &tmB, fb, n0, k0, zb);
            if (two) tma_load_3d_pair(sb + kSliceBytes, &tmB, fb, n0 + 64, k0, zb);
          } else if (tail) {
            for (int i = 0; i < boxes; ++i)
              tma_load_3d_pair(sb + i * (32 * kKB * 2), &tmTail, fb, k0, n0 + i * 32, zb);
          } else {
            tma_load_3d_pair(sb, &tmB, fb, k0, n0, zb);
          }
        }
        __syncwarp();
        issued |= 1u << stage;
        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    if (ok) {
      // the last round's "empty" arrivals land in this CTA's shared memory:
      // wait for them so that none is still in flight when the CTA exits
      for (int s = 0; s < STAGES; ++s)
        if (issued & (1u << s)) {
          int dummy = 0;
          wait_bounded(empty_bar(s), (issued_parity >> s) & 1u, &dummy, nullptr);
        }
    } else {
      // A wait ran out.  Copies that were issued land in microseconds, on
      // barriers that may be the other CTA's; this CTA's memory stays until then.
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < kLandNs) {
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------- MMA issuer (leader only) ----
    if (leader) {
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      bool ok = true;
      for (int tile = cluster; tile < total_tiles && ok; tile += nclusters) {
        const Tile ti = uniform_tile(tile);
        if (RAG_K && ti.nkb == 0) continue;  // an empty group: the epilogue writes zeros
        const int acc = it & 1;
        const uint32_t ap = (it >> 1) & 1;
        ++it;
        ok = __all_sync(0xffffffffu,
                        wait_bounded(tempty_bar(acc), ap ^ 1u, abort_p, args.status));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kTile);
        const uint32_t idesc = idesc_16bit_f32(kTile, 0, FP16, A_MN, B_MN) |
                               (static_cast<uint32_t>(ti.ncols >> 3) << 17);
        for (int kb = 0; kb < ti.nkb; ++kb) {
          ok = __all_sync(0xffffffffu, wait_bounded(full_bar(stage), phase, abort_p, args.status));
          if (!ok) break;
          tc_fence_after();
          // 16 k values further: 32 bytes along a K-major row, 16 rows of 128
          // bytes of an MN-major slice
          const uint32_t sa = smem_base + stage * STAGE_BYTES;
          const uint64_t da = A_MN ? desc_mnmajor_sw128(sa, kSliceBytes) : desc_kmajor_sw128(sa);
          const uint64_t db = B_MN ? desc_mnmajor_sw128(sa + A_BYTES, kSliceBytes)
                                   : desc_kmajor_sw128(sa + A_BYTES);
          constexpr uint32_t a_step = (A_MN ? 2048 : 32) >> 4, b_step = (B_MN ? 2048 : 32) >> 4;
          // steps of 16 that hold anything of the reduction
          const int steps = min(kKB, ti.len - kb * kKB + 15) >> 4;
          if (elect_lane()) {
            if (steps == 4) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_bf16_pair(d_tmem, da + k * a_step, db + k * b_step, idesc,
                              (kb > 0 || k > 0) ? 1u : 0u);
            } else {
              for (int k = 0; k < steps; ++k)
                mma_bf16_pair(d_tmem, da + k * a_step, db + k * b_step, idesc,
                              (kb > 0 || k > 0) ? 1u : 0u);
            }
            mma_commit_pair(empty_bar(stage), kBoth);
            if (kb == ti.nkb - 1) mma_commit_pair(tfull_bar(acc), kBoth);
          }
          __syncwarp();
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {
        // wait for every MMA already issued before TMEM is released
        if (elect_lane()) mma_commit_pair(drain_bar, 0x1);
        __syncwarp();
        int dummy = 0;
        wait_bounded(drain_bar, 0, &dummy, nullptr);
      }
    }
    __syncwarp();
  } else if (RAG_K && warp == 3) {
    // ------------------------- the last k-block's rows behind the group ----
    uint32_t parity = 0;  // of each stage's landing barrier
    int done = 0;         // stage of the next tile's first k-block
    for (int tile = cluster; tile < total_tiles; tile += nclusters) {
      const Tile ti = tile_of(tile);
      if ((ti.rows & 15) != 0) {
        const int rem = ti.rows & (kKB - 1);
        const int s = (done + ti.nkb - 1) % STAGES;
        if (!__all_sync(0xffffffffu,
                        wait_bounded(land_bar(s), (parity >> s) & 1u, abort_p, args.status)))
          break;
        parity ^= 1u << s;
        uint8_t* base = smem + s * STAGE_BYTES;
        // the rows from rem to the end of their step of 16 (the steps behind it
        // are not issued), in each of the four 64-wide slices
        for (int o = rem * 128 + lane * 16; o < ((rem + 15) & ~15) * 128; o += 512) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(base + c * kSliceBytes + o) = make_uint4(0, 0, 0, 0);
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_release(map_to_cta(full_bar(s), 0));
      }
      done = (done + ti.nkb) % STAGES;
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------- epilogue -----
    const int q = warp & 3;            // TMEM lane quarter of this warp
    const int hcol = (warp - 4) >> 2;  // which half of the tile's columns it drains
    constexpr int CW = EPI == kMmStoreBf16 ? 64 : 32;  // columns of a chunk
    const int hw = (tn / 2 + CW - 1) / CW * CW;        // columns of a half
    const int r = q * 32 + lane;
    const uint32_t tempty_leader0 = map_to_cta(tempty_bar(0), 0);
    const uint32_t tempty_leader1 = map_to_cta(tempty_bar(1), 0);
    uint8_t* stage = smem + STAGES * STAGE_BYTES + (warp - 4) * kWarpStage;
    int it = 0;
    // Newton-Schulz: the values of src beside the accumulator, read two chunks
    // of 32 columns ahead, across tiles
    constexpr bool SRC = EPI == kMmPoly || EPI == kMmUpdate;
    RowFetch src_hi[2], src_lo[2];
    auto fetch_src = [&](const Tile& t, int c) {
      const int col = t.col0 + hcol * hw + c * 32;
      const int row0 = t.m_blk * kTile + static_cast<int>(rank) * kHalf + q * 32;
      const int64_t at = t.g * (static_cast<int64_t>(args.m) * args.ld) + row0 * args.ld + col;
      const int rows = c * 32 < hw && col < t.col0 + tn ? args.m - row0 : 0;
      const int pieces = (static_cast<int>(args.ld) - col) / 8;
      src_hi[c & 1].fetch(static_cast<const __half*>(args.src) + at, args.ld, rows, pieces, lane);
      if (EPI == kMmUpdate)
        src_lo[c & 1].fetch(static_cast<const __half*>(args.src_lo) + at, args.ld, rows, pieces,
                            lane);
    };
    // and of the diagonal beside them: a value per row, or per column, which
    // go to this warp's columns in shared memory
    float* diag_cols =
        reinterpret_cast<float*>(smem + STAGES * STAGE_BYTES + kEpiWarps * kWarpStage) +
        (warp - 4) * (kWarpDiag / 4);
    const bool by_row = EPI == kMmPoly || !args.diag_cols, by_col = EPI == kMmPoly || args.diag_cols;
    float next_row[4] = {};
    float4 next_col = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto fetch_diag = [&](const Tile& t) {
      const float* diag = args.diag + static_cast<int64_t>(t.g) * args.diag_ld;
      const int row0 = t.m_blk * kTile + static_cast<int>(rank) * kHalf + q * 32;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int pr = row0 + i * 8 + lane / 4;
        next_row[i] = by_row && pr < args.m ? diag[pr] : 0.0f;
      }
      const int col = t.col0 + hcol * hw + lane * 4;
      next_col = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (by_col && col < args.diag_ld) next_col = *reinterpret_cast<const float4*>(diag + col);
    };
    Tile following{};
    if (SRC && cluster < total_tiles) {
      following = tile_of(cluster);
      fetch_diag(following);
      fetch_src(following, 0);
      fetch_src(following, 1);
    }
    for (int tile = cluster; tile < total_tiles; tile += nclusters) {
      const Tile ti = SRC ? following : tile_of(tile);
      const bool more = tile + nclusters < total_tiles;
      float drow[4] = {};
      if (SRC) {
        __syncwarp();
        *reinterpret_cast<float4*>(diag_cols + lane * 4) = next_col;
#pragma unroll
        for (int i = 0; i < 4; ++i) drow[i] = next_row[i];
        __syncwarp();
        if (more) {
          following = tile_of(tile + nclusters);
          fetch_diag(following);
        }
      }
      auto fetch_ahead = [&](int c) {
        if (c < 2) fetch_src(ti, c + 2);
        else if (more) fetch_src(following, c - 2);
      };
      // 32 accumulator columns through the staging area, from a row per lane to
      // RowFetch's pieces: the one crossing that this epilogue makes, since
      // shared memory also feeds the MMAs and is what they contend for (src
      // and results crossing instead cost 5 x 0.2 ms more at 64 x 2048 x 1408)
      auto stage_acc = [&](uint32_t addr) {
        float x[32];
        __syncwarp();  // lanes leave the chunk before this one at different points
        tmem_ld32(addr, x);
        tmem_ld_wait_regs(x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float4*>(stage + lane * kStagePitch + i * 16) =
              make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        __syncwarp();
      };
      auto take_acc = [&](int it4, F2* y) {
        const ulonglong2* p = reinterpret_cast<const ulonglong2*>(
            stage + (it4 * 8 + lane / 4) * kStagePitch + (lane % 4) * 32);
        const ulonglong2 u = p[0], v = p[1];
        y[0] = u.x;
        y[1] = u.y;
        y[2] = v.x;
        y[3] = v.y;
      };
      // the diagonal's values at the columns of this lane's pieces of chunk c
      auto take_diag = [&](int c, F2* d) {
        const ulonglong2* p =
            reinterpret_cast<const ulonglong2*>(diag_cols + c * 32 + (lane % 4) * 8);
        const ulonglong2 u = p[0], v = p[1];
        d[0] = u.x;
        d[1] = u.y;
        d[2] = v.x;
        d[3] = v.y;
      };
      const bool empty = RAG_K && ti.nkb == 0;
      const int acc = it & 1;
      const uint32_t ap = (it >> 1) & 1;
      if (!empty) {
        ++it;
        if (!__all_sync(0xffffffffu, wait_bounded(tfull_bar(acc), ap, abort_p, args.status)))
          break;
        tc_fence_after();
      }
      const int row = ti.m_blk * kTile + static_cast<int>(rank) * kHalf + r;
      const bool live = row < (RAG_K ? args.m : ti.rows);
      const int col0 = ti.col0 + hcol * hw;
      const int col_end = min(min(col0 + hw, ti.col0 + tn), args.n);
      const int ld_end = col_end < args.n ? col_end : static_cast<int>(args.ld);
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                             static_cast<uint32_t>(acc * kTile + hcol * hw);
      const int64_t orow = RAG_M ? static_cast<int64_t>(ti.row0) + row : row;
      // of this warp's 32 rows: where the first goes, and how many there are
      const int64_t obase = (RAG_M ? 0 : ti.g * args.out_stride) + (orow - lane) * args.ld;
      const int warp_rows = (RAG_K ? args.m : ti.rows) - (row - lane);
      if (EPI == kMmStoreTBf16) {
        // D's columns are the output's rows: 32 lanes hold 32 neighbours of
        // each.  The halves of the warps take halves of the columns.
        const int width = max(32, tn / 2);
#pragma unroll 1
        for (int c = hcol * width; c < min((hcol + 1) * width, tn); c += 32) {
          const int left = ti.rows - ti.col0 - c;  // rows of the group from here
          if (left <= 0) break;
          float x[32];
          tmem_ld32(tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                        static_cast<uint32_t>(acc * kTile + c),
                    x);
          tmem_ld_wait_regs(x);
          bf16* out = static_cast<bf16*>(args.out) +
                      (static_cast<int64_t>(ti.row0) + ti.col0 + c) * args.ld + (row - lane);
          if (left < 8) {
            if (row < args.m) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (j < left) out[static_cast<int64_t>(j) * args.ld + lane] = __float2bfloat16_rn(x[j]);
            }
          } else {
            // through the staging area, to 16-byte pieces of the output's rows
#pragma unroll
            for (int j = 0; j < 32; ++j)
              reinterpret_cast<bf16*>(stage + j * kStagePitch)[lane] = __float2bfloat16_rn(x[j]);
            __syncwarp();
#pragma unroll
            for (int it4 = 0; it4 < 4; ++it4) {
              const int j = it4 * 8 + lane / 4, piece = lane % 4;
              const uint4 v = *reinterpret_cast<const uint4*>(stage + j * kStagePitch + piece * 16);
              if (j < left && row - lane + piece * 8 < args.m)
                *reinterpret_cast<uint4*>(out + static_cast<int64_t>(j) * args.ld + piece * 8) = v;
            }
            __syncwarp();
          }
        }
      } else if (EPI == kMmStoreBf16) {
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {  // a half is at most 128 wide
          const int col = col0 + c * 64;
          if (col >= col_end) break;
          float x[64];
          if (!empty) {
            tmem_ld32(taddr + c * 64, x);
            tmem_ld32(taddr + c * 64 + 32, x + 32);
            tmem_ld_wait_regs(x);
            tmem_ld_wait_regs(x + 32);
          } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) x[i] = 0.0f;
          }
          uint4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            Vec16<bf16>::store(reinterpret_cast<bf16*>(&v[i]), x + i * 8);
          bf16* out = static_cast<bf16*>(args.out) + obase + col;
          store_rows<8>(stage, v, out, args.ld * 2, warp_rows, (col_end - col) / 8, lane, PutPlain{});
        }
      } else if (EPI == kMmStoreF32 || EPI == kMmAddF32) {
        if (!(EPI == kMmAddF32 && empty)) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const int col = col0 + c * 32;
            if (col >= col_end) break;
            float x[32];
            if (!empty) {
              tmem_ld32(taddr + c * 32, x);
              tmem_ld_wait_regs(x);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = 0.0f;
            }
            float* out = static_cast<float*>(args.out) + obase + col;
            const uint4* v = reinterpret_cast<const uint4*>(x);
            if (EPI == kMmAddF32)
              store_rows<8>(stage, v, out, args.ld * 4, warp_rows, (col_end - col) / 4, lane, PutAddF32{});
            else
              store_rows<8>(stage, v, out, args.ld * 4, warp_rows, (col_end - col) / 4, lane, PutPlain{});
          }
        }
      } else if (EPI == kMmGram) {
        // fp16 off the diagonal, the diagonal itself in fp32 apart
        float* dout = args.diag_out + static_cast<int64_t>(ti.g) * args.diag_ld;
        __half* omat = static_cast<__half*>(args.out) + ti.g * args.out_stride;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const int col = col0 + c * 32;
          if (col >= col_end) break;
          float x[32];
          tmem_ld32(taddr + c * 32, x);
          tmem_ld_wait_regs(x);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] *= args.inv_scale2;
          if (live && row >= col && row < col + 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (col + i == row) {
                dout[row] = x[i];
                x[i] = 0.0f;
              }
          }
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = pack_half8(x + i * 8);
          __half* out = omat + static_cast<int64_t>(row - lane) * args.ld + col;
          store_rows<4>(stage, v, out, args.ld * 2, warp_rows, (ld_end - col) / 8, lane, PutPlain{});
          if (SYM && ti.m_blk != ti.n_blk / per_blk) {
            // the mirrored tile: lane r writes column r of the staging area,
            // whose rows go out in 16-byte pieces
#pragma unroll
            for (int i = 0; i < 32; ++i)
              reinterpret_cast<__half*>(stage + i * kStagePitch)[lane] = __float2half_rn(x[i]);
            __syncwarp();
            const int mrow0 = row - lane;  // the mirrored rows' first column
#pragma unroll
            for (int it4 = 0; it4 < 4; ++it4) {
              const int j = it4 * 8 + lane / 4, piece = lane % 4;
              const uint4 v4 = *reinterpret_cast<const uint4*>(stage + j * kStagePitch + piece * 16);
              if (col + j < col_end && mrow0 + piece * 8 < args.ld)
                *reinterpret_cast<uint4*>(omat + static_cast<int64_t>(col + j) * args.ld + mrow0 +
                                          piece * 8) = v4;
            }
            __syncwarp();
          }
        }
      } else if (EPI == kMmPoly) {
        // off the diagonal b a + c ((d_i + d_j) a + o), o the product of A's
        // off-diagonal parts; on it, where a = 0, (b + c d) d + c o
        float* dout = args.diag_out + static_cast<int64_t>(ti.g) * args.diag_ld;
        __half* omat = static_cast<__half*>(args.out) + ti.g * args.out_stride;
        const int row0 = row - lane;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int col = col0 + c * 32;
          const int pc = col + (lane % 4) * 8;  // first column of this lane's pieces
          uint4 out[4];
          if (col < col_end) {
            stage_acc(taddr + c * 32);
            F2 dj[4];
            take_diag(c, dj);
            const F2 cc = pair(args.cc, args.cc);
            const bool on = col < row0 + 32 && row0 < col + 32;  // the diagonal passes here
#pragma unroll
            for (int it4 = 0; it4 < 4; ++it4) {
              const int pr = row0 + it4 * 8 + lane / 4;
              F2 a[4], y[4];
              half_pairs(src_hi[c & 1].v[it4], a);
              take_acc(it4, y);
              const float e = args.cb + args.cc * drow[it4];  // (b + c d_i + c d_j) a + c o
              const F2 e2 = pair(e, e);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                y[j] = fma2(fma2(cc, dj[j], e2), a[j], mul2(cc, y[j]));
              if (on) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float2 f = both(y[j]);
                  const int at = pr - pc - 2 * j;  // which of the pair is on it
                  if (at == 0 || at == 1) {
                    if (pr < args.m) dout[pr] = (at ? f.y : f.x) + drow[it4] * e;
                    y[j] = pair(at ? f.x : 0.0f, at ? 0.0f : f.y);
                  }
                }
              }
              out[it4] = pairs_half(y);
              if (pr < args.m && pc < ld_end)
                *reinterpret_cast<uint4*>(omat + static_cast<int64_t>(pr) * args.ld + pc) = out[it4];
            }
          }
          fetch_ahead(c);
          if (col < col_end && ti.m_blk != ti.n_blk / per_blk) {
            // the mirrored tile, transposed through the staging area in rows of
            // 72 bytes
            constexpr int pitch = 72;
            __syncwarp();
#pragma unroll
            for (int it4 = 0; it4 < 4; ++it4) {
              const __half* h = reinterpret_cast<const __half*>(&out[it4]);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                reinterpret_cast<__half*>(stage + ((lane % 4) * 8 + j) * pitch)[it4 * 8 + lane / 4] =
                    h[j];
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int j = k * 4 + lane / 8, piece = lane % 8;
              const uint2 v2 = *reinterpret_cast<const uint2*>(stage + j * pitch + piece * 8);
              if (col + j < col_end && row0 + piece * 4 < args.ld)
                *reinterpret_cast<uint2*>(omat + static_cast<int64_t>(col + j) * args.ld + row0 +
                                          piece * 4) = v2;
            }
            __syncwarp();
          }
        }
      } else {
        // X' = a (hi + lo) + d hi + (B off its diagonal) hi, all times `scale`;
        // d is B's diagonal, of the row where B stands on the left
        const int64_t src_base = ti.g * (static_cast<int64_t>(args.m) * args.ld);
        const bool last = args.out_lo == nullptr;
        const float inv = 1.0f / args.scale;
        const int row0 = row - lane;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int col = col0 + c * 32;
          const int pc = col + (lane % 4) * 8;
          if (col < col_end) {
            stage_acc(taddr + c * 32);
            F2 dc[4];
            take_diag(c, dc);
            const F2 ca = pair(args.ca, args.ca), minus = pair(-1.0f, -1.0f);
#pragma unroll
            for (int it4 = 0; it4 < 4; ++it4) {
              const int pr = row0 + it4 * 8 + lane / 4;
              F2 h[4], l[4], y[4];
              half_pairs(src_hi[c & 1].v[it4], h);
              half_pairs(src_lo[c & 1].v[it4], l);
              take_acc(it4, y);
              const float e = args.ca + drow[it4];  // (a + d) hi + a lo + the product
              const F2 e2 = pair(e, e);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                y[j] = fma2(add2(e2, dc[j]), h[j], fma2(ca, l[j], y[j]));
              if (pr >= args.m || pc >= ld_end) continue;
              if (!last) {
                const int64_t at = src_base + static_cast<int64_t>(pr) * args.ld + pc;
                const uint4 hv = pairs_half(y);
                *reinterpret_cast<uint4*>(static_cast<__half*>(args.out) + at) = hv;
                half_pairs(hv, h);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = fma2(h[j], minus, y[j]);
                *reinterpret_cast<uint4*>(static_cast<__half*>(args.out_lo) + at) = pairs_half(y);
              } else {
                // the last step: bf16 in the caller's dense layout
                bf16* out = static_cast<bf16*>(args.out) + ti.g * args.out_stride +
                            static_cast<int64_t>(pr) * args.n + pc;
                float f[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float2 v = both(y[j]);
                  f[2 * j] = v.x * inv;
                  f[2 * j + 1] = v.y * inv;
                }
                if (args.vec_ok) {
                  Vec16<bf16>::store(out, f);
                } else if (args.n % 2 == 0) {
#pragma unroll
                  for (int j = 0; j < 8; j += 2)
                    if (pc + j < col_end)
                      *reinterpret_cast<__nv_bfloat162*>(out + j) =
                          __floats2bfloat162_rn(f[j], f[j + 1]);
                } else {
#pragma unroll
                  for (int j = 0; j < 8; ++j)
                    if (pc + j < col_end) out[j] = __float2bfloat16_rn(f[j]);
                }
              }
            }
          }
          fetch_ahead(c);
        }
      }
      if (!empty) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc ? tempty_leader1 : tempty_leader0);
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync_all();  // no CTA of the pair leaves while the other still works
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

template <int LAYOUT, int SCHED, int EPI, bool FP16, int BR = 128>
int launch_impl(const CUtensorMap& a, const CUtensorMap& b, const MmArgs& args, int pairs,
                cudaStream_t st, const CUtensorMap* tail = nullptr) {
  static std::atomic<uint64_t> optin{0};
  auto kern = mm_pair_kernel<LAYOUT, SCHED, EPI, FP16, BR>;
  constexpr int smem = Stage<BR>::kSmem;
  if (int rc = ensure_smem_optin(reinterpret_cast<const void*>(kern), smem, optin)) return rc;
  return launch_k(kern, dim3(2 * pairs), kThreads, smem, st, 2, a, b, tail ? *tail : b, args);
}

}  // namespace

bool make_map_16bit(CUtensorMap* map, bool fp16, const void* base, uint64_t inner, uint64_t rows,
                    uint64_t depth, uint64_t ld, uint64_t stride, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn || !base || inner == 0 || rows == 0 || depth == 0) return false;
  cuuint64_t dims[3] = {inner, rows, depth};
  cuuint64_t strides[2] = {ld * 2, stride * 2};
  cuuint32_t box[3] = {64, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int launch_mm(int layout, int sched, int epi, const CUtensorMap& a, const CUtensorMap& b,
              const MmArgs& args, int pairs, cudaStream_t st, const CUtensorMap* tail) {
  if (pairs <= 0) return MOE_OK;
  if (sched == kMmRaggedM && epi == kMmStoreBf16) {
    if (layout == kMmNT) return launch_impl<kMmNT, kMmRaggedM, kMmStoreBf16, false>(a, b, args, pairs, st);
    if (layout == kMmNN) return launch_impl<kMmNN, kMmRaggedM, kMmStoreBf16, false>(a, b, args, pairs, st);
  }
  if (sched == kMmRaggedN && epi == kMmStoreTBf16) {
    if (args.tn > 128) {
      if (!tail) return MOE_ERR_SHAPE;
      if (layout == kMmNT) return launch_impl<kMmNT, kMmRaggedN, kMmStoreTBf16, false>(a, b, args, pairs, st, tail);
      if (layout == kMmTT) return launch_impl<kMmTT, kMmRaggedN, kMmStoreTBf16, false>(a, b, args, pairs, st, tail);
    }
    if (args.tn > 64) {
      if (layout == kMmNT) return launch_impl<kMmNT, kMmRaggedN, kMmStoreTBf16, false, 64>(a, b, args, pairs, st);
      if (layout == kMmTT) return launch_impl<kMmTT, kMmRaggedN, kMmStoreTBf16, false, 64>(a, b, args, pairs, st);
    }
    if (layout == kMmNT) return launch_impl<kMmNT, kMmRaggedN, kMmStoreTBf16, false, 32>(a, b, args, pairs, st);
    if (layout == kMmTT) return launch_impl<kMmTT, kMmRaggedN, kMmStoreTBf16, false, 32>(a, b, args, pairs, st);
  }
  if (sched == kMmRaggedK && layout == kMmTN) {
    if (epi == kMmStoreBf16) return launch_impl<kMmTN, kMmRaggedK, kMmStoreBf16, false>(a, b, args, pairs, st);
    if (epi == kMmStoreF32) return launch_impl<kMmTN, kMmRaggedK, kMmStoreF32, false>(a, b, args, pairs, st);
    if (epi == kMmAddF32) return launch_impl<kMmTN, kMmRaggedK, kMmAddF32, false>(a, b, args, pairs, st);
  }
  if (sched == kMmBatchSym && epi == kMmGram) {
    if (layout == kMmNT) return launch_impl<kMmNT, kMmBatchSym, kMmGram, true>(a, b, args, pairs, st);
    if (layout == kMmTN) return launch_impl<kMmTN, kMmBatchSym, kMmGram, true>(a, b, args, pairs, st);
  }
  if (sched == kMmBatchSym && epi == kMmPoly && layout == kMmNT)
    return launch_impl<kMmNT, kMmBatchSym, kMmPoly, true>(a, b, args, pairs, st);
  if (sched == kMmBatch && epi == kMmUpdate) {
    if (layout == kMmNT) return launch_impl<kMmNT, kMmBatch, kMmUpdate, true>(a, b, args, pairs, st);
    if (layout == kMmNN) return launch_impl<kMmNN, kMmBatch, kMmUpdate, true>(a, b, args, pairs, st);
  }
  return MOE_ERR_SHAPE;
}

}  // namespace sm100
}  // namespace moe
