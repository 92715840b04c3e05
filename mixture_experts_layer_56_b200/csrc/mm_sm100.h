// Host interface of the tcgen05 matrix products of the training operators
// (mm_sm100.cu): products of ragged row groups with their group's matrix, and
// the products of the Newton-Schulz iteration over a stack of matrices.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {
namespace sm100 {

// Operand layouts of D[M, N] = sum_k A(m, k) B(n, k).  K-major: k runs along
// the memory rows; MN-major: m (or n) does.
enum MmLayout {
  kMmNT = 0,  // A [M, K], B [N, K]: both K-major
  kMmNN = 1,  // A [M, K] K-major, B [K, N] MN-major
  kMmTN = 2,  // A [K, M], B [K, N]: both MN-major
  kMmTT = 3,  // A [K, M] MN-major, B [N, K] K-major
};

// What a tile's rows, columns and reduction come from.
enum MmSched {
  kMmRaggedM = 0,  // rows offsets[g] .. offsets[g+1]-1 against matrix g
  kMmRaggedN = 4,  // the same with the matrix as A and the rows as B: D is the
                   // output's transpose
  kMmRaggedK = 1,  // the reduction runs over those rows; one output per group
  kMmBatch = 2,    // `groups` equal products
  kMmBatchSym = 3, // the same, D symmetric: the tiles on and above the diagonal
};

enum MmEpi {
  kMmStoreBf16 = 0,
  kMmStoreF32 = 1,
  kMmAddF32 = 2,   // out += D
  kMmGram = 3,     // Newton-Schulz: A = X X^T, diagonal apart
  kMmPoly = 4,     // Newton-Schulz: B = b A + c A A, diagonal apart
  kMmUpdate = 5,   // Newton-Schulz: X <- a X + B X
  kMmStoreTBf16 = 6,  // D^T as bf16
};

constexpr int kMmMaxGroups = 256;

struct MmArgs {
  const int32_t* offsets;  // ragged schedules: device, [groups + 1]
  int32_t rows;            // ragged schedules: bound of the offsets
  int32_t groups;
  int32_t m;               // rows of D of one group (not kMmRaggedM)
  int32_t n;               // columns of D (not kMmRaggedN)
  int32_t tn;              // columns of a tile (mm_tile_width)
  int32_t k;               // reduction length (not kMmRaggedK)
  void* out;
  int64_t ld;              // elements between rows of out
  int64_t out_stride;      // elements between groups of out (not kMmRaggedM)
  int32_t* status;
  // Newton-Schulz only; see ortho.cu for what each holds
  const void* src;         // kMmPoly: A off the diagonal; kMmUpdate: X, high part
  const void* src_lo;      // kMmUpdate: X, low part
  void* out_lo;            // kMmUpdate: X', low part (NULL: the last step)
  const float* diag;       // kMmPoly: diagonal of A; kMmUpdate: diagonal of B
  float* diag_out;         // kMmGram, kMmPoly
  int32_t diag_ld;         // elements between matrices of diag
  int32_t diag_cols;       // kMmUpdate: B stands on the right (its diagonal scales columns)
  int32_t vec_ok;          // kMmUpdate, last step: rows of out are 16-byte aligned
  float ca, cb, cc;        // coefficients of the step
  float scale, inv_scale2; // X is held times `scale`; 1 / scale^2
};

// Rank-3 map {inner, rows, depth} with 128-byte swizzle and box {64, box_rows, 1}
// of a 16-bit type; strides in elements.
bool make_map_16bit(CUtensorMap* map, bool fp16, const void* base, uint64_t inner, uint64_t rows,
                    uint64_t depth, uint64_t ld, uint64_t stride, uint32_t box_rows);

// Columns of a tile: n cut into equal tiles of at most 256, in the MMA's steps
// of 32 (n = 1288: six tiles of 224, not five of 256 and one of 8).  Where
// `bands` such rows of tiles leave pairs of CTAs idle, tiles are 128 or 64
// wide.
inline int32_t mm_tile_width(int32_t n, int64_t bands, int pairs) {
  int32_t most = 256;
  while (most > 64 && bands * ((n + most / 2 - 1) / (most / 2)) <= pairs) most /= 2;
  const int32_t tiles = (n + most - 1) / most;
  return ((n + tiles - 1) / tiles + 31) / 32 * 32;
}
// The same for a symmetric product (kMmBatchSym) of `mats` matrices of side n,
// whose tiles divide a block of 256; *tiles gets their number.
inline int32_t mm_tile_width_sym(int32_t n, int64_t mats, int pairs, int64_t* tiles) {
  const int64_t blocks = (n + 255) / 256;
  auto count = [&](int32_t w) {
    return mats * (blocks * ((n + w - 1) / w) - 256 / w * (blocks * (blocks - 1) / 2));
  };
  int32_t w = 256;
  while (w > 64 && count(w / 2) <= pairs) w /= 2;
  *tiles = count(w);
  return w;
}

// Box rows of the A (or B) map of a layout: MN-major operands come in slices
// of 64 k rows, K-major ones in a CTA's 128 rows of A or its half of the
// tile's columns.
inline uint32_t mm_box_a(int layout) { return layout == kMmTN || layout == kMmTT ? 64u : 128u; }
inline uint32_t mm_box_b(int layout, int32_t tn) {
  return layout == kMmNT || layout == kMmTT ? static_cast<uint32_t>(tn / 2) : 64u;
}

// `pairs` CTA pairs compute the product.  kMmRaggedN with tn = 256 takes a
// second map of B, with a box of 32 rows, for the groups' last ones.
int launch_mm(int layout, int sched, int epi, const CUtensorMap& a, const CUtensorMap& b,
              const MmArgs& args, int pairs, cudaStream_t st, const CUtensorMap* tail = nullptr);

}  // namespace sm100
}  // namespace moe
