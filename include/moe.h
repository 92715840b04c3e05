/*
 * moe.h -- C ABI of libmoe: the DeepSeekMoE layer forward on NVIDIA B200
 * (sm_100a).
 *
 * The layer (from "DeepSeekMoE: Towards Ultimate Expert Specialization in
 * Mixture-of-Experts Language Models", §3.2 Shared Expert Isolation,
 * eqs. (9)-(11)):
 *
 *   h_t  = u_t + sum_{s < K_s} FFN_s(u_t) + sum_{k < K} g_{t,k} FFN_{idx[t,k]}(u_t)
 *   s_t  = Softmax_i(u_t^T e_i (+ b_i))   over the N_r routed experts
 *   idx  = the K largest s_{t,i} (lower expert index wins ties),
 *   g    = s at those experts, not renormalised
 *   FFN(x) = W2 (SiLU(W1 x) * (W3 x))    (SwiGLU, no biases)
 *
 * with N_r = mN - K_s fine-grained routed experts (§3.1) and K = mK - K_s.
 * Layer normalisation is not part of the layer (the pages omit it, §2).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Pointers are DEVICE pointers owned by the caller unless a parameter says
 *   HOST.  The library never allocates device memory; scratch space comes
 *   from the caller's workspace `ws` (size from moe_workspace_size).
 * - All tensors are dense row-major.  Element types: `dtype` MOE_DTYPE_BF16
 *   means activations and weights are bfloat16 (raw 16-bit); MOE_DTYPE_F32
 *   means float32.  Router bias, gates and fp32 intermediates are float32;
 *   indices are int32.
 * - Base pointers must be 16-byte aligned (MOE_ERR_ALIGN otherwise).
 * - The bf16 path runs the expert GEMMs on tcgen05 tensor cores and needs
 *   d % 64 == 0 and inter % 64 == 0; the fp32 path runs them on CUDA cores.
 * - Every call is asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *   default stream) and never synchronises the host, except where stated.
 * - Return value: MOE_OK (0) or a negative MOE_ERR_* code.  Nothing is
 *   launched after a validation error.  MOE_ERR_CUDA reports a launch error.
 *   A kernel that gives up on a bounded wait records MOE_ERR_DEVICE_CHECK in
 *   the workspace's status word, read with moe_read_status.
 * - Results are bitwise reproducible from run to run (no atomics decide any
 *   value or order).
 * - Kernels are launched with programmatic dependent launch: one may start
 *   its set-up while the previous kernel on the stream finishes, but it reads
 *   and writes no global memory before that kernel has completed, so the
 *   usual stream order holds for the caller's own work too.
 * - moe_layer_forward only enqueues kernels on `stream` (no allocation, no
 *   host synchronisation), so a caller may capture it into a CUDA graph and
 *   replay it; replays give the eager result bit for bit.
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef void* moe_stream_t; /* a cudaStream_t */

enum {
  MOE_DTYPE_F32 = 0,
  MOE_DTYPE_BF16 = 1,
};

enum {
  MOE_OK = 0,
  MOE_ERR_NULLPTR = -1,      /* a required pointer is NULL */
  MOE_ERR_SHAPE = -2,        /* sizes out of range or inconsistent */
  MOE_ERR_ALIGN = -3,        /* a pointer is not 16-byte aligned */
  MOE_ERR_WORKSPACE = -4,    /* workspace smaller than moe_workspace_size */
  MOE_ERR_DTYPE = -5,        /* unknown dtype */
  MOE_ERR_CUDA = -6,         /* CUDA runtime / launch error */
  MOE_ERR_DEVICE_CHECK = -7, /* a kernel gave up waiting (see moe_read_status) */
  MOE_ERR_UNSUPPORTED = -8,  /* no device of compute capability 10.0 */
  MOE_ERR_SCRATCH_LIMIT = -9, /* shape too large for moe_dispatch_static_scratch */
};

/* Router flags (moe_shape_t.flags). */
enum {
  /* The router bias b_i shifts only the top-K selection; the gates are the
     softmax of the unbiased logits (the per-expert load-balancing bias the
     csdn.net DeepSeekMoE article describes in words, §2.3).  Default (0):
     the bias is part of the logit for both selection and softmax. */
  MOE_FLAG_BIAS_SELECT_ONLY = 1,
  /* Tile shape of the bf16 expert GEMMs (default: chosen from the average
     rows per routed expert).  SINGLE_CTA: 128-row tiles, one SM each.
     CTA_PAIR: 256-row tiles computed by the two SMs of a 2-CTA cluster
     (tcgen05 cta_group::2).  Setting both is MOE_ERR_SHAPE.  Results are the
     same up to fp32 summation order inside the tensor cores. */
  MOE_FLAG_GEMM_SINGLE_CTA = 2,
  MOE_FLAG_GEMM_CTA_PAIR = 4,
  /* bf16 router on the CUDA cores: each logit is two fp32 FMA chains over
     the halves of d in increasing j, added once.  Default (0): the logits
     are one tcgen05 MMA tile per 128 tokens (bf16 products are exact in
     fp32; fp32 accumulation in the tensor cores' own order).  The two agree
     up to fp32 summation order.  The fp32 dtype always uses the CUDA
     cores. */
  MOE_FLAG_ROUTER_SIMT = 8,
  /* Failure injection, for tests of the error path: the TMA producer of each
     bf16 expert GEMM waits, before its first load, for a shared-memory slot
     that nothing releases.  That wait gives up after 1 ms like any bounded
     wait: the kernel records MOE_ERR_DEVICE_CHECK in the workspace status
     word, lets its in-flight work finish, frees its tensor memory and
     returns.  The call's outputs are then not valid; the context stays
     usable.  Never set in production. */
  MOE_FLAG_INJECT_WAIT_TIMEOUT = 16,
  /* CTA-pair tiles at most 256 columns wide.  Default (0): where every
     group's output width is a multiple of 512 (2*inter and 2*inter*n_shared
     for the gate/up GEMM, d for the down GEMM), a CTA pair computes
     256 x 512 tiles (two N = 256 MMAs per k-block, 48 rather than 64 bytes
     of operand tiles per clock of tensor work).  Same results up to fp32
     summation order inside the tensor cores. */
  MOE_FLAG_GEMM_NARROW = 32,
};

/* Layer shape.  Limits: 1 <= n_routed <= 256, 1 <= top_k <= min(n_routed, 32),
   0 <= n_shared <= 64, T >= 0 (T = 0 is a no-op), d >= 1, inter >= 1.  */
typedef struct {
  int64_t T;        /* tokens */
  int32_t d;        /* hidden size */
  int32_t n_routed; /* N_r = mN - K_s routed experts */
  int32_t n_shared; /* K_s shared experts */
  int32_t inter;    /* I, intermediate width of one fine-grained expert */
  int32_t top_k;    /* K = mK - K_s routed experts per token */
  int32_t dtype;    /* MOE_DTYPE_* */
  int32_t flags;    /* MOE_FLAG_* */
} moe_shape_t;

/* Human-readable name of a status code (static string). */
const char* moe_strerror(int status);

/* Bytes of workspace that moe_layer_forward, moe_dispatch and
   moe_expert_ffn need for `shape` (a multiple of 256). */
int moe_workspace_size(const moe_shape_t* shape, size_t* bytes);

/* W13 packing used by the tensor-core gate/up GEMM.
   W1, W3: [n_experts, inter, d]; W13 out: [n_experts, 2*inter, d] where, for
   every block b of 64 intermediate rows, packed rows 128b..128b+63 are W1
   rows 64b..64b+63 and packed rows 128b+64..128b+127 are W3 rows 64b..64b+63.
   (For dtype F32 the packed layout is the same.)  inter % 64 must be 0.
   Weight preparation, done once per model, not per forward. */
int moe_pack_w13(const moe_shape_t* shape, int32_t n_experts, const void* W1,
                 const void* W3, void* W13, moe_stream_t stream);

/* a1-a2, router (eqs. (10)-(11)): logits u_t.e_i (+ b_i) accumulated in fp32
   (tensor cores for bf16, see MOE_FLAG_ROUTER_SIMT), softmax over the
   n_routed experts, top-K.
   u: [T, d]; E: [n_routed, d]; bias: [n_routed] float32 or NULL.
   Outputs idx: [T, top_k] int32 in descending score order (ties: lower
   index first); w: [T, top_k] float32 gates (not renormalised). */
int moe_route(const moe_shape_t* shape, const void* u, const void* E,
              const float* bias, int32_t* idx, float* w, moe_stream_t stream);

/* a3, dispatch ("each token is computed only by its K experts", §2):
   counts[e] = #{(t,k): idx[t,k] = e}; offsets = exclusive scan (n_routed+1);
   perm[p] = slot t*top_k+k of position p, expert e's slots filling
   offsets[e]..offsets[e+1]-1 in increasing t; inv[t*top_k+k] = its position.
   idx must hold distinct experts per token in [0, n_routed).
   All outputs int32; bit-exact.  Uses workspace `ws`. */
int moe_dispatch(const moe_shape_t* shape, const int32_t* idx, int32_t* counts,
                 int32_t* offsets, int32_t* perm, int32_t* inv, void* ws,
                 size_t ws_bytes, moe_stream_t stream);

/* The same dispatch as moe_dispatch, same outputs bit for bit, for callers
   that cannot supply device memory per call: the paper has no counterpart;
   it is an interface for embedders.  Allocation may synchronise the device
   or fail once a caching pool holds the GPU's memory, so a latency-bound
   serving loop, or a host library without an allocator of its own, may not
   be able to provide `ws`.  This call allocates nothing: its scratch is one
   fixed array of MOE_DISPATCH_STATIC_SCRATCH_BYTES inside libmoe.
   Limit: 2 * round_up_256(ceil(T/128) * n_routed * 4) bytes must fit in
   that array (T <= 32768 at 256 routed experts, T <= 131072 at 64);
   larger shapes return MOE_ERR_SCRATCH_LIMIT before any launch.
   Set-up: the first call on each device (current device at the call)
   looks up the array's device address; make that first call before any
   stream capture begins on the device.  If that lookup fails the call
   returns MOE_ERR_CUDA and clears the calling thread's last CUDA error
   (cudaGetLastError), including an earlier one the caller had not read.
   Tracing (moe_profile_enable) brackets its kernels as MOE_KERNEL_DISPATCH.
   Sharing: every call in the process, on any stream, uses the same array.
   Calls whose kernels may overlap on a device race on it and corrupt each
   other's perm/inv/offsets; order them (one stream, or events).  Nothing in
   the array has to start at zero: each call writes every entry it reads. */
#define MOE_DISPATCH_STATIC_SCRATCH_BYTES (512u * 1024u)
int moe_dispatch_static_scratch(const moe_shape_t* shape, const int32_t* idx,
                                int32_t* counts, int32_t* offsets, int32_t* perm,
                                int32_t* inv, moe_stream_t stream);

/* a4-a6, expert FFNs: for every position p of expert e's segment,
   y[p] = FFN_e(u_{perm[p]/top_k}); and ysh[t] = sum_s FFN_s(u_t) over the
   shared experts (computed as one SwiGLU FFN of width n_shared*inter, the
   segmentation identity of §3.1).
   W13: [n_routed, 2*inter, d] packed by moe_pack_w13; W2: [n_routed, d, inter];
   W13_s: [n_shared, 2*inter, d] packed; W2_s: [n_shared, d, inter].
   y: [T*top_k, d] in dtype; ysh: [T, d] float32.  fp32 accumulation; for bf16
   the SwiGLU activation is rounded to bf16 before the down projection.
   perm/offsets as produced by moe_dispatch.  Uses workspace `ws`. */
int moe_expert_ffn(const moe_shape_t* shape, const void* u, const int32_t* perm,
                   const int32_t* offsets, const void* W13, const void* W2,
                   const void* W13_s, const void* W2_s, void* y, float* ysh,
                   void* ws, size_t ws_bytes, moe_stream_t stream);

/* a7, combine + residual (eq. (9)): h_t = u_t + ysh_t + sum_{k<K} w[t,k] *
   y[inv[t*K+k]], accumulated in fp32 in exactly that order, rounded once to
   dtype.  h: [T, d] dtype. */
int moe_combine(const moe_shape_t* shape, const void* u, const float* ysh,
                const void* y, const float* w, const int32_t* inv, void* h,
                moe_stream_t stream);

/* The whole layer: route, dispatch, expert FFNs and combine, on `stream`,
   with every intermediate in `ws`.  Arguments as above; h: [T, d] dtype.
   Decode-sized batches (see moe_forward_path) run as one kernel that
   streams each activated expert's weights once in units of 64 intermediate
   rows, with fp32 partial down projections summed in a fixed order, and
   other batches of up to 128 tokens route, dispatch and gather in one
   kernel (each after a one-warp kernel that zeroes its grid-wide counters
   in ws); their h matches the oracle within the same bars but is not the
   stage-wise result bit for bit.  All other batches give exactly the result
   of moe_route, moe_dispatch, moe_expert_ffn and moe_combine. */
int moe_layer_forward(const moe_shape_t* shape, const void* u, const void* E,
                      const float* bias, const void* W13, const void* W2,
                      const void* W13_s, const void* W2_s, void* h, void* ws,
                      size_t ws_bytes, moe_stream_t stream);

/* moe_layer_forward with the activations in HOST memory: u_host [T, d] is
   copied to the device, the layer runs, and h is copied back into h_host;
   the call returns when h_host is written.  Page-locked host buffers make
   the copies asynchronous DMA.  Weights stay on the device.  Batches of at
   least 4352 tokens run in up to 4 chunks: the uploads and downloads go
   through two streams of the library's own, overlapping the forward of
   other chunks on `stream`, and start after the work already on `stream`.
   h equals moe_layer_forward's bit for bit.  Calls on one device run one
   at a time.  Workspace: moe_workspace_size plus 2*T*d*elem bytes. */
int moe_layer_forward_host(const moe_shape_t* shape, const void* u_host,
                           const void* E, const float* bias, const void* W13,
                           const void* W2, const void* W13_s, const void* W2_s,
                           void* h_host, void* ws, size_t ws_bytes,
                           moe_stream_t stream);

/* How moe_layer_forward runs `shape`:
   MOE_PATH_DECODE_LAYER: one kernel for the whole layer (bf16, 1 <= T <= 8,
     d in {256, 512, 1024, 2048}, inter % 64 == 0, and neither a GEMM tile
     shape nor failure injection forced in flags);
   MOE_PATH_SMALL_BATCH: router, dispatch and gather in one kernel with fp32
     CUDA-core logits, then the grouped GEMMs and the combine (other bf16
     batches of at most 128 tokens with d in {256, 512, 1024, 2048}, without
     MOE_FLAG_ROUTER_SIMT);
   MOE_PATH_STAGES: router, dispatch, grouped GEMMs, combine, each as
     moe_route / moe_dispatch / moe_expert_ffn / moe_combine compute them
     (h is their result bit for bit).
   The first two match the oracle within the same bars; their gates follow
   their own fp32 logits, so h is not the stage-wise result bit for bit. */
enum { MOE_PATH_STAGES = 0, MOE_PATH_DECODE_LAYER = 1, MOE_PATH_SMALL_BATCH = 2 };
int moe_forward_path(const moe_shape_t* shape, int32_t* path);

/* Bytes moe_layer_forward_host needs. */
int moe_workspace_size_host(const moe_shape_t* shape, size_t* bytes);

/* Expert load statistics of §3.3, eqs. (12)-(14), for the routing in idx
   and the scores of the router: f[e] = N'/(K'T) * counts[e] and P[e] =
   (1/T) sum_t s_{t,e}, with s recomputed from u, E, bias as in moe_route.
   f, P: [n_routed] float32.  (Training statistic; not on the forward path.)
   Uses workspace `ws`. */
int moe_expert_balance(const moe_shape_t* shape, const void* u, const void* E,
                       const float* bias, const int32_t* counts, float* f,
                       float* P, void* ws, size_t ws_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------------------
 * Training operators: what a training step of the experts is made of.
 *
 *   x = moe_layer_norm(u)                        the norm in front of the layer
 *   moe_route, moe_dispatch, rows gathered by perm
 *   gu = moe_grouped_matmul(x_rows, W13)         packed gate/up columns
 *   a  = moe_swiglu(gu)
 *   y  = moe_grouped_matmul(a, W2)               -> moe_combine
 *   da = moe_grouped_matmul_dx(dy, W2)           dW2  = moe_grouped_matmul_dw(dy, a)
 *   dgu = moe_swiglu_backward(gu, da)
 *   dx = moe_grouped_matmul_dx(dgu, W13)         dW13 = moe_grouped_matmul_dw(dgu, x_rows)
 *   du = moe_layer_norm_backward(...)
 *   update = moe_orthogonalize(momentum of dW)
 *
 * The conventions at the top of this file hold: device pointers, dense
 * row-major tensors, 16-byte aligned, asynchronous on `stream`, no
 * allocation, bitwise reproducible, capturable.  An output overlaps no input
 * unless its function says so.  A call that takes `ws` writes there: calls
 * that may run at the same time, replays of captured ones among them, need a
 * workspace each.  Nothing in it has to be set before a call; but a workspace
 * that moe_read_status is to be asked about (those of the grouped products and
 * of moe_orthogonalize) has its first 4 bytes zeroed once.
 * ------------------------------------------------------------------------- */

/* Ragged groups of rows, each with its own matrix: group g owns the rows
   offsets[g] .. offsets[g+1]-1 (device int32 [n_groups + 1], as moe_dispatch
   writes them) and W_g, row-major [n, k] in W [n_groups, n, k].  Groups may be
   empty.  Offsets outside [0, rows] count as the nearer bound, and one below
   an offset before it as that one: no offsets reach outside the tensors or
   give a row to two groups.  Rows that no group owns are not written, and
   nothing depends on them.
   Limits: 1 <= n_groups <= 256, 0 <= rows <= 2^31 - 512, 1 <= n, k <= 2^24;
   bf16: n and k multiples of 8; fp32 runs on the CUDA cores.  The products'
   64 x 64 output tiles must number fewer than 2^31, and the tensors be smaller
   than 2^40 bytes. */
typedef struct {
  int64_t rows;     /* rows of X, Y, dY and dX */
  int32_t n_groups;
  int32_t n;        /* columns of Y and dY, rows of one W */
  int32_t k;        /* columns of X and dX, columns of one W */
  int32_t dtype;    /* MOE_DTYPE_* of X, Y, dY, dX and W */
  int32_t flags;    /* MOE_GROUPED_* */
} moe_grouped_shape_t;

enum {
  /* dW is float32 instead of `dtype`. */
  MOE_GROUPED_DW_F32 = 1,
  /* dW += the gradient; dW must be float32 (dtype F32 or the flag above). */
  MOE_GROUPED_DW_ACCUMULATE = 2,
};

int moe_grouped_workspace_size(const moe_grouped_shape_t* shape, size_t* bytes);

/* Y[r] = W_g X[r] for every row r of group g.  X [rows, k], Y [rows, n]. */
int moe_grouped_matmul(const moe_grouped_shape_t* shape, const void* X, const int32_t* offsets,
                       const void* W, void* Y, void* ws, size_t ws_bytes, moe_stream_t stream);

/* Input gradient: dX[r] = W_g^T dY[r].  dY [rows, n], dX [rows, k]. */
int moe_grouped_matmul_dx(const moe_grouped_shape_t* shape, const void* dY, const int32_t* offsets,
                          const void* W, void* dX, void* ws, size_t ws_bytes,
                          moe_stream_t stream);

/* Weight gradient: dW_g = sum over the group's rows of dY[r] X[r]^T, zero for
   an empty group (left as it is with MOE_GROUPED_DW_ACCUMULATE).
   dW [n_groups, n, k], every element written.  fp32 accumulation; for bf16
   inputs it is the tensor cores' own, which truncates: relative to its norm, a
   float32 dW is off by about 1e-9 times the group's rows where the products'
   signs are mixed, and by up to 6e-9 times, downwards, where they are all the
   same (5.5e-4 for 98304 rows).  So are the sums of the two products above, of
   k and n terms, beside their own rounding to bf16. */
int moe_grouped_matmul_dw(const moe_grouped_shape_t* shape, const void* dY, const void* X,
                          const int32_t* offsets, void* dW, void* ws, size_t ws_bytes,
                          moe_stream_t stream);

/* SwiGLU on packed gate/up columns: a row of gu [rows, 2*inter] holds, for
   each block of 64 intermediate columns, 64 gate values g and then the 64 up
   values u (the product of a row with moe_pack_w13's W13).
   0 <= rows < 2^31, inter a positive multiple of 64, at most 2^24. */
typedef struct {
  int64_t rows;
  int32_t inter;
  int32_t dtype;
} moe_swiglu_shape_t;

/* a = SiLU(g) * u.  a [rows, inter]. */
int moe_swiglu(const moe_swiglu_shape_t* shape, const void* gu, void* a, moe_stream_t stream);

/* With s = 1 / (1 + e^-g): dg = da * u * s * (1 + g (1 - s)), du = da * g * s,
   packed like gu into dgu [rows, 2*inter], which may be gu itself. */
int moe_swiglu_backward(const moe_swiglu_shape_t* shape, const void* gu, const void* da, void* dgu,
                        moe_stream_t stream);

/* Layer norm of each row of x [T, d]: y = (x - mean) * rstd * gamma + beta,
   rstd = 1 / sqrt(var + eps), var = mean (x - mean)^2, all in fp32.
   0 <= T < 2^31, 1 <= d <= 2^24, eps finite and >= 0. */
typedef struct {
  int64_t T;
  int32_t d;
  int32_t dtype;  /* of x, y, dy and dx */
  float eps;
} moe_norm_shape_t;

/* gamma [d] and beta [d] (NULL: none) are float32.  mean and rstd [T] float32
   are kept for the backward pass; either may be NULL.  y may be x. */
int moe_layer_norm(const moe_norm_shape_t* shape, const void* x, const float* gamma,
                   const float* beta, void* y, float* mean, float* rstd, moe_stream_t stream);

int moe_layer_norm_workspace_size(const moe_norm_shape_t* shape, size_t* bytes);

/* The gradients of moe_layer_norm from its input x and its mean and rstd:
   dx [T, d], dgamma [d] and dbeta [d] (NULL: not wanted) float32.  dx may be
   dy.  For T = 0 dgamma and dbeta are zero. */
int moe_layer_norm_backward(const moe_norm_shape_t* shape, const void* dy, const void* x,
                            const float* gamma, const float* mean, const float* rstd, void* dx,
                            float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                            moe_stream_t stream);

/* Newton-Schulz orthogonalisation of n_mats matrices M [n_mats, rows, cols]
   (the Muon optimiser's update): X = M / (|M|_F + 1e-7), then `steps` times
   A = X X^T (for rows > cols the transpose's), X <- a X + (b A + c A A) X.
   `coef` is HOST memory, (a, b, c) for each step, read before the call
   returns; NULL means 3.4445, -4.7750, 2.0315 in each.  O [n_mats, rows,
   cols] is bfloat16, whatever the dtype of M.  The products run on the tensor
   cores with fp16 operands beside a 22-bit X, whatever the dtype of M, which
   needs the coefficients to keep the singular values of every step's X below
   about 10 (the defaults keep them below 1.25).  O's error relative to its norm
   is about 2e-3 for random matrices and up to 2.6e-3 where all singular values
   are alike, bf16's own rounding of 1.7e-3 among it (which for a matrix of one
   value can be 2^-8 by itself).  Entries of X below about 2^-24 /
   sqrt(max(rows, cols)) are lost, as in matrices whose norm is far below the
   1e-7.  A matrix of
   zeros gives zeros; one with an infinity or NaN gives NaN, the others of the
   stack are untouched by it.  M's tensor may have any 1 <= rows, cols <=
   65536; n_mats <= 65535; 1 <= steps <= 16. */
typedef struct {
  int32_t n_mats;
  int32_t rows;
  int32_t cols;
  int32_t steps;
  int32_t dtype;  /* of M */
} moe_ortho_shape_t;

int moe_orthogonalize_workspace_size(const moe_ortho_shape_t* shape, size_t* bytes);
int moe_orthogonalize(const moe_ortho_shape_t* shape, const float* coef, const void* M, void* O,
                      void* ws, size_t ws_bytes, moe_stream_t stream);

/* Copies the workspace status word (0 or MOE_ERR_DEVICE_CHECK) to *status
   and clears it; synchronises `stream`. */
int moe_read_status(const void* ws, int32_t* status, moe_stream_t stream);

/* Tracing: device time of each stage.  While enabled, every kernel (the
   dispatch kernels count as one stage) that libmoe launches is
   bracketed by CUDA events recorded on its stream.  moe_profile_read waits
   for those events and returns, oldest first, the stage kind (MOE_KERNEL_*)
   and elapsed milliseconds of each bracketed launch since the last read:
   at most `max` entries are written and *count receives the number
   written; up to 4096 are kept, later ones are dropped.  `on`: 0 = off,
   1 = every stage, otherwise a mask of (1 << MOE_KERNEL_*) bits naming the
   stages to bracket (each bracket adds two event records to the stream, so
   a mask keeps the timing of the other stages undisturbed).  Tracing never
   changes any result. */
enum {
  MOE_KERNEL_ROUTER = 1,
  MOE_KERNEL_DISPATCH = 2,
  MOE_KERNEL_GATHER = 3,
  MOE_KERNEL_GEMM_GATE_UP = 4, /* grouped gate/up GEMM + SwiGLU (tcgen05) */
  MOE_KERNEL_GEMM_DOWN = 5,    /* grouped down GEMM (tcgen05) */
  MOE_KERNEL_COMBINE = 6,
  MOE_KERNEL_FFN_F32 = 7,      /* the fp32 expert FFN (both GEMMs) */
  MOE_KERNEL_MEMSET = 8,
  MOE_KERNEL_PACK = 9,
  MOE_KERNEL_BALANCE = 10,
  MOE_KERNEL_DECODE_LAYER = 11, /* the whole layer for decode-sized batches */
  MOE_KERNEL_GROUPED_FWD = 12,
  MOE_KERNEL_GROUPED_DX = 13,
  MOE_KERNEL_GROUPED_DW = 14,
  MOE_KERNEL_SWIGLU = 15,
  MOE_KERNEL_SWIGLU_BACKWARD = 16,
  MOE_KERNEL_LAYER_NORM = 17,
  MOE_KERNEL_LAYER_NORM_BACKWARD = 18,
  MOE_KERNEL_ORTHOGONALIZE = 19,
};
int moe_profile_enable(int on);
int moe_profile_read(int32_t* kinds, float* ms, int32_t max, int32_t* count);
const char* moe_kernel_name(int32_t kind);

/* Number of kernels this library has launched since load (all threads). */
uint64_t moe_launch_count(void);

/* Library version string. */
const char* moe_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H_ */
