// Newton-Schulz orthogonalisation of a stack of matrices (the update rule of
// the Muon optimiser): X = M / (|M|_F + 1e-7), then per step
//
//   A = X X^T (X^T X for tall matrices),  B = b A + c A A,  X <- a X + B X.
//
// The products run on the tensor cores in fp16 (fp32 accumulation): every
// entry of X, A and B is at most a few units, so fp16's 11 bits beat bf16's 8
// at the same rate.  What a rounding does to the result depends on where it
// enters.  A step multiplies directions with singular value 0 by a = 3.4, so
// noise that reaches X itself outside M's row and column space grows by 3.4
// per step (with a rounded X, 10% of the result for a matrix of rank 1).  So
// X is kept as a sum hi + lo of two fp16 numbers (22 bits), and only the
// products read hi alone: B hi has M's column space on the left, A has it on
// both sides, and the noise that they add does not grow.  The diagonals of A
// and B, their largest entries by far as X nears orthogonality, are kept in
// fp32 and left out of the fp16 matrices:
//
//   (D + O)(D + O) = D D + D O + O D + O O,   B X = diag(B) hi + B_off hi.
//
// X is held times a power of two near sqrt(max side), which centres its
// entries in fp16's range.  A and B are symmetric: only the tiles on and above
// the diagonal are computed, and written twice.
//
// Bound by the tensor cores and the power cap: 64 matrices of 2048 x 1408, five
// steps, 4.79 TFLOP (symmetric halves counted once), 6.4 ms call after call, the
// cap holding the clock near 1.2 GHz, and 5.4 rested at 1.9 GHz; per step, rested,
// A takes 235 us, B 197 and the update 510 (it reads hi, lo and writes both beside
// its product, 1.5 GB).
// Matrices of few hundred rows are bound by three launches a step of about 10 us
// each: one of 256 x 256 108 us, five of 640 x 560 167.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "mm_sm100.h"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr int kOrthoThreads = 256;
constexpr int kMaxParts = 64;
constexpr int64_t kPartElems = 16384;

template <typename T>
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[kOrthoThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kOrthoThreads / 32; ++i) s += red[i];
  return s;
}

// partial[mat][part] = sum of squares of a slice of the matrix.  fp64: the
// squares of large finite entries overflow fp32.
template <typename T>
__global__ void __launch_bounds__(kOrthoThreads)
ortho_sumsq_kernel(const T* __restrict__ M, int64_t elems, double* __restrict__ partial) {
  pdl_wait();
  pdl_trigger();
  const int parts = gridDim.x;
  const T* m = M + blockIdx.y * elems;
  // slices start on multiples of 8 elements
  const int64_t per = ((elems + parts - 1) / parts + 7) / 8 * 8;
  const int64_t beg = blockIdx.x * per;
  const int64_t end = beg + per < elems ? beg + per : elems;
  constexpr int N = Vec16<T>::N;
  double s = 0.0;
  if (elems % N == 0) {
    for (int64_t i = beg + static_cast<int64_t>(threadIdx.x) * N; i < end;
         i += kOrthoThreads * N) {
      float v[N];
      Vec16<T>::load(m + i, v);
#pragma unroll
      for (int j = 0; j < N; ++j) s += static_cast<double>(v[j]) * v[j];
    }
  } else {
    for (int64_t i = beg + threadIdx.x; i < end; i += kOrthoThreads) {
      const double v = to_f32(m[i]);
      s += v * v;
    }
  }
  s = block_sum<T>(s);
  if (threadIdx.x == 0) partial[blockIdx.y * parts + blockIdx.x] = s;
}

// hi + lo = scale * M / (|M|_F + 1e-7), rows of pitch ld
template <typename T>
__global__ void __launch_bounds__(kOrthoThreads)
ortho_split_kernel(const T* __restrict__ M, int rows, int cols, int64_t ld,
                   const double* __restrict__ partial, int parts, float scale,
                   __half* __restrict__ hi, __half* __restrict__ lo) {
  pdl_wait();
  pdl_trigger();
  const double* p = partial + static_cast<int64_t>(blockIdx.y) * parts;
  const double sq = block_sum<T>(threadIdx.x < parts ? p[threadIdx.x] : 0.0);
  const double f = scale / (sqrt(sq) + 1e-7);
  const int64_t mat = blockIdx.y;
  const T* m = M + mat * rows * cols;
  const int per_row = static_cast<int>(ld / 8);
  const int64_t pieces = static_cast<int64_t>(rows) * per_row;
  const bool vec = cols % 8 == 0;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kOrthoThreads + threadIdx.x; i < pieces;
       i += static_cast<int64_t>(gridDim.x) * kOrthoThreads) {
    const int64_t r = i / per_row;
    const int c = static_cast<int>(i - r * per_row) * 8;
    float v[8];
    if (vec) {
#pragma unroll
      for (int j = 0; j < 8; j += Vec16<T>::N) Vec16<T>::load(m + r * cols + c + j, v + j);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = c + j < cols ? to_f32(m[r * cols + c + j]) : 0.0f;
    }
    __half h[8], l[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = static_cast<float>(v[j] * f);
      h[j] = __float2half_rn(x);
      l[j] = __float2half_rn(x - __half2float(h[j]));
    }
    const int64_t at = mat * rows * ld + r * ld + c;
    *reinterpret_cast<uint4*>(hi + at) = *reinterpret_cast<const uint4*>(h);
    *reinterpret_cast<uint4*>(lo + at) = *reinterpret_cast<const uint4*>(l);
  }
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <typename T>
int launch_prepare(const void* M, int mats, int rows, int cols, const OrthoLayout& L, float scale,
                   uint8_t* ws, cudaStream_t st) {
  double* partial = reinterpret_cast<double*>(ws + L.partial);
  const int64_t elems = static_cast<int64_t>(rows) * cols;
  if (int rc = launch_k(ortho_sumsq_kernel<T>, dim3(L.parts, mats), dim3(kOrthoThreads), 0, st, 1,
                        static_cast<const T*>(M), elems, partial))
    return rc;
  const int64_t pieces = static_cast<int64_t>(rows) * (L.ldx / 8);
  const int64_t want = (pieces + kOrthoThreads * 4 - 1) / (kOrthoThreads * 4);
  const int gx = static_cast<int>(want < 1024 ? want : 1024);
  return launch_k(ortho_split_kernel<T>, dim3(gx, mats), dim3(kOrthoThreads), 0, st, 1,
                  static_cast<const T*>(M), rows, cols, L.ldx,
                  static_cast<const double*>(partial), L.parts, scale,
                  reinterpret_cast<__half*>(ws + L.hi0), reinterpret_cast<__half*>(ws + L.lo));
}

}  // namespace

OrthoLayout ortho_layout(int mats, int rows, int cols) {
  OrthoLayout L{};
  L.m = rows < cols ? rows : cols;
  L.ldx = (cols + 7) / 8 * 8;
  L.ldm = (L.m + 7) / 8 * 8;
  const int64_t elems = static_cast<int64_t>(rows) * cols;
  const int64_t parts = (elems + kPartElems - 1) / kPartElems;
  L.parts = static_cast<int>(parts < kMaxParts ? parts : kMaxParts);
  const size_t n = static_cast<size_t>(mats);
  const size_t x = n * static_cast<size_t>(rows) * L.ldx * 2, g = n * static_cast<size_t>(L.m) * L.ldm * 2,
               dg = n * static_cast<size_t>(L.ldm) * 4;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += up256(bytes);
    return at;
  };
  L.status = take(256);
  if (ortho_small_fits(rows, cols)) {
    L.total = o;
    return L;
  }
  L.partial = take(n * L.parts * 8);
  L.hi0 = take(x);
  L.hi1 = take(x);
  L.lo = take(x);
  L.gram = take(g);
  L.poly = take(g);
  L.dgram = take(dg);
  L.dpoly = take(dg);
  L.total = o;
  return L;
}

int launch_orthogonalize(int dtype, const void* M, void* O, int mats, int rows, int cols, int steps,
                         const float* coef, void* wsp, int sms, cudaStream_t st) {
  using namespace sm100;
  const OrthoLayout L = ortho_layout(mats, rows, cols);
  uint8_t* ws = static_cast<uint8_t*>(wsp);
  const int longest = rows > cols ? rows : cols;
  float scale = 1.0f;
  while (scale * scale * 4.0f <= static_cast<float>(longest)) scale *= 2.0f;
  if (ortho_small_fits(rows, cols))
    return launch_ortho_small(dtype, M, O, mats, rows, cols, steps, coef, scale,
                              reinterpret_cast<int32_t*>(ws + L.status), st);
  const int rc = dtype == MOE_DTYPE_BF16
                     ? launch_prepare<bf16>(M, mats, rows, cols, L, scale, ws, st)
                     : launch_prepare<float>(M, mats, rows, cols, L, scale, ws, st);
  if (rc) return rc;
  const bool tall = rows > cols;
  const uint64_t r64 = rows, c64 = cols, m64 = L.m, n64 = mats;
  const uint64_t xs = r64 * L.ldx, gs = m64 * L.ldm;
  // operands of the three products (see mm_sm100.h)
  const int gram_layout = tall ? kMmTN : kMmNT;
  const int upd_layout = tall ? kMmNT : kMmNN;
  const int most = sms / 2;
  int64_t sym_tiles = 0;
  const int32_t sym_tn = mm_tile_width_sym(L.m, mats, most, &sym_tiles);
  const int64_t bands = static_cast<int64_t>(mats) * ((rows + 255) / 256);
  const int32_t upd_tn = mm_tile_width(cols, bands, most);
  const int64_t upd_tiles = bands * ((cols + upd_tn - 1) / upd_tn);
  const int sym_pairs = static_cast<int>(sym_tiles < most ? sym_tiles : most);
  const int upd_pairs = static_cast<int>(upd_tiles < most ? upd_tiles : most);
  // each matrix as the A and as the B operand of what it enters; X twice, for
  // the steps read and write it in turn
  CUtensorMap xa[2], xb[2], xu[2], ga, gb, bu;
  bool ok = make_map_16bit(&ga, true, ws + L.gram, m64, m64, n64, L.ldm, gs, mm_box_a(kMmNT)) &&
            make_map_16bit(&gb, true, ws + L.gram, m64, m64, n64, L.ldm, gs,
                           mm_box_b(kMmNT, sym_tn)) &&
            make_map_16bit(&bu, true, ws + L.poly, m64, m64, n64, L.ldm, gs,
                           tall ? mm_box_b(upd_layout, upd_tn) : mm_box_a(upd_layout));
  for (int i = 0; i < 2; ++i) {
    void* x = ws + (i ? L.hi1 : L.hi0);
    ok = ok && make_map_16bit(&xa[i], true, x, c64, r64, n64, L.ldx, xs, mm_box_a(gram_layout)) &&
         make_map_16bit(&xb[i], true, x, c64, r64, n64, L.ldx, xs, mm_box_b(gram_layout, sym_tn)) &&
         make_map_16bit(&xu[i], true, x, c64, r64, n64, L.ldx, xs,
                        tall ? mm_box_a(upd_layout) : mm_box_b(upd_layout, upd_tn));
  }
  if (!ok) return MOE_ERR_CUDA;
  for (int s = 0; s < steps; ++s) {
    const int cur = s & 1;
    MmArgs a{};
    a.groups = mats;
    a.status = reinterpret_cast<int32_t*>(ws + L.status);
    a.ca = coef[3 * s];
    a.cb = coef[3 * s + 1];
    a.cc = coef[3 * s + 2];
    a.scale = scale;
    a.inv_scale2 = 1.0f / (scale * scale);
    a.diag_ld = static_cast<int32_t>(L.ldm);
    // A = X X^T
    a.m = a.n = L.m;
    a.tn = sym_tn;
    a.k = tall ? rows : cols;
    a.out = ws + L.gram;
    a.ld = L.ldm;
    a.out_stride = static_cast<int64_t>(gs);
    a.diag_out = reinterpret_cast<float*>(ws + L.dgram);
    if (int e = launch_mm(gram_layout, kMmBatchSym, kMmGram, xa[cur], xb[cur], a, sym_pairs, st))
      return e;
    // B = b A + c A A
    a.k = L.m;
    a.src = ws + L.gram;
    a.diag = reinterpret_cast<const float*>(ws + L.dgram);
    a.out = ws + L.poly;
    a.diag_out = reinterpret_cast<float*>(ws + L.dpoly);
    if (int e = launch_mm(kMmNT, kMmBatchSym, kMmPoly, ga, gb, a, sym_pairs, st)) return e;
    // X <- a X + B X, the last time as bf16 into O
    const bool last = s == steps - 1;
    a.m = rows;
    a.n = cols;
    a.tn = upd_tn;
    a.src = ws + (cur ? L.hi1 : L.hi0);
    a.src_lo = ws + L.lo;
    a.diag = reinterpret_cast<const float*>(ws + L.dpoly);
    a.diag_cols = tall;
    a.ld = L.ldx;
    if (last) {
      a.out = O;
      a.out_stride = static_cast<int64_t>(rows) * cols;
      a.out_lo = nullptr;
      a.vec_ok = cols % 8 == 0;
    } else {
      a.out = ws + (cur ? L.hi0 : L.hi1);
      a.out_stride = static_cast<int64_t>(xs);
      a.out_lo = ws + L.lo;  // each element is read and then written by one warp
    }
    if (int e = launch_mm(upd_layout, kMmBatch, kMmUpdate, tall ? xu[cur] : bu, tall ? bu : xu[cur],
                          a, upd_pairs, st))
      return e;
  }
  return MOE_OK;
}

}  // namespace moe
