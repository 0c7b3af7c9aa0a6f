/*
 * gemm_gb300.h -- C ABI of the GB300 (sm_103a) dense GEMM with fused epilogue.
 *
 * Operation (one call):
 *
 *     z[i][j] = alpha * sum_k A[i][k] * B[k][j]  +  beta * C[i][j]  +  bias[j]
 *     C[i][j] = cast_out( epilogue(z[i][j]) )        for 0 <= i < M, 0 <= j < N
 *
 * with fp32 accumulation whatever the input type, the epilogue applied to the
 * accumulators in registers and the result stored once.  Defined on the pages
 * by: "Case Study: Steel's BlockMMA" (the paragraph on the ending where fusion
 * plugs in -- store_result applies the Epilogue to every accumulator, and
 * apply_epilogue reads an input C for alpha*AB + beta*C; AccumType = float;
 * transposition by the A_str_m / A_str_k stride constants), "Case Study: The
 * Tiled GEMM" (the fused alpha*AB + beta*C store), "X3: Metal GEMM" sections
 * 2, 4 and 5 (out-of-range operand elements read as zero; the masked,
 * casting write-back that never touches elements outside M x N) and Rigel
 * (abstract and section 1: GEMM + bias + GELU fused into one kernel).
 *
 * Conventions shared by every entry point
 *   - All pointers except those documented as host pointers are DEVICE
 *     pointers on the current CUDA device.  The caller owns every buffer;
 *     the library allocates nothing per call and keeps no pointer after a
 *     call returns.
 *   - Strides and leading dimensions are in ELEMENTS, not bytes.
 *   - Calls are asynchronous on `stream` (NULL = the legacy default stream).
 *     A returned GEMM_OK means the work was enqueued; device-side failures
 *     are reported later by gemm_device_status().
 *   - No entry point prints, aborts or traps.  Argument errors return a
 *     status code before anything is enqueued.
 */
#ifndef GEMM_GB300_H
#define GEMM_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream. */
typedef struct CUstream_st *gemm_stream_t;

/* Element types.  E4M3 is OCP FP8 E4M3 ("fn": finite, saturating, NaN = S.1111.111). */
typedef enum {
    GEMM_F32 = 0,
    GEMM_F16 = 1,
    GEMM_BF16 = 2,
    GEMM_E4M3 = 3
} gemm_dtype_t;

/* Epilogues, applied to z before the cast: none, or bias[j] added and then
 * an activation.  GELU is the exact erf form 0.5*z*(1 + erf(z/sqrt(2))) (the
 * pages' bias+GELU fusion, Rigel section 1); the others use the same
 * pluggable place ("Case Study: Steel's BlockMMA", the Epilogue functor):
 * GELU's tanh form 0.5*z*(1 + tanh(sqrt(2/pi)*(z + 0.044715*z^3))), SiLU
 * z/(1 + exp(-z)) and ReLU max(z, 0).  Every one needs a bias. */
typedef enum {
    GEMM_EPI_NONE = 0,
    GEMM_EPI_BIAS = 1,
    GEMM_EPI_BIAS_GELU = 2,
    GEMM_EPI_BIAS_GELU_TANH = 3,
    GEMM_EPI_BIAS_SILU = 4,
    GEMM_EPI_BIAS_RELU = 5
} gemm_epilogue_t;

typedef enum {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_ARG = 1,   /* negative size, ldc < N, bad enum, NULL where a buffer is needed */
    GEMM_ERR_UNSUPPORTED = 2,   /* dtype combination the library does not implement */
    GEMM_ERR_MISALIGNED = 3,    /* an array not aligned as its entry point needs (gemm() itself never returns it) */
    GEMM_ERR_WORKSPACE = 4,     /* workspace missing or smaller than gemm_workspace_size() */
    GEMM_ERR_CUDA = 5,          /* a CUDA runtime/driver call failed (launch, attribute, tensor map) */
    GEMM_ERR_TIMEOUT = 6        /* a device-side wait gave up (reported by gemm_device_status) */
} gemm_status_t;

/* Which kernel family a call runs on (see gemm_query_path).  The grouped and 8-bit products report TCGEN05 for
 * their tcgen05 kernels, EPILOGUE_ONLY without a product, and SIMT for every other kernel (few rows: mma.sync and
 * dot products; any strides: multiply-adds).  fp32 inputs report
 * GEMM_PATH_SIMT, the path without a workspace; given a workspace of
 * gemm_workspace_size() bytes they run as 3xTF32 on the tensor cores. */
typedef enum {
    GEMM_PATH_NOOP = 0,           /* M == 0 or N == 0: nothing to do */
    GEMM_PATH_EPILOGUE_ONLY = 1,  /* K == 0 or alpha == 0: C = cast(epilogue(beta*C + bias)) */
    GEMM_PATH_TCGEN05 = 2,        /* TMA -> shared memory -> tcgen05.mma (TMEM accumulators) */
    GEMM_PATH_SIMT = 3            /* CUDA-core FFMA kernel (fp32 inputs, or strides TMA cannot take) */
} gemm_path_t;

/*
 * gemm -- C = cast(epilogue(alpha*A*B + beta*C + bias)), C updated in place.
 *
 *   M, N, K        problem sizes, each >= 0.  M == 0 or N == 0 is a no-op.
 *                  K == 0 (or alpha == 0) gives C = cast(epilogue(beta*C + bias))
 *                  and reads neither A nor B (BLAS convention).
 *   ab_dtype       element type of A and B: F32, F16, BF16 or E4M3.
 *   A              element (i, k) is A[i*a_stride_m + k*a_stride_k].
 *   B              element (k, j) is B[k*b_stride_k + j*b_stride_n].
 *                  Transposition is expressed only through these strides; any
 *                  non-negative strides are accepted.  When one stride of an
 *                  operand is 1, the base is 16-byte aligned and the other
 *                  stride is a multiple of 16 bytes, the operand is streamed
 *                  by TMA; otherwise the call runs on the SIMT kernel.
 *   C, ldc         row-major M x N output (and input when beta != 0) inside an
 *                  M x ldc buffer, ldc >= N.  Columns N..ldc-1 and anything
 *                  outside the M x N block are never written.
 *   c_dtype        F32, F16 or BF16.  F32 inputs require F32 output; E4M3
 *                  inputs require BF16 or F32 output.
 *   alpha, beta    fp32 scalars.  beta == 0: C is not read (NaNs in C do not
 *                  propagate).  For fp8 with per-tensor dequantisation scales
 *                  s_a, s_b, pass alpha * s_a * s_b.
 *   bias           fp32[N] device array, required (non-NULL) for every
 *                  epilogue other than GEMM_EPI_NONE, ignored for NONE.
 *   epilogue       a gemm_epilogue_t; the order is z = alpha*AB + beta*C +
 *                  bias, then the activation, then the cast (round to nearest
 *                  even).
 *   workspace      optional device scratch, 256-byte aligned, owned by the
 *   workspace_bytes  caller: with at least gemm_workspace_size(...) bytes the
 *                  last waves of output tiles are split along K over all SM
 *                  pairs (stream-K: partial sums go through the workspace);
 *                  with less, or NULL / 0, whole tiles only.  Calls that share
 *                  a workspace must not run concurrently.  Its contents need no
 *                  initialisation (each call tags its flags with a fresh value).
 *   stream         CUDA stream the work is enqueued on.
 *
 * Aliasing: C must not overlap A, B or bias.  Returns GEMM_OK once enqueued.
 */
gemm_status_t gemm(int64_t M, int64_t N, int64_t K,
                   gemm_dtype_t ab_dtype,
                   const void *A, int64_t a_stride_m, int64_t a_stride_k,
                   const void *B, int64_t b_stride_k, int64_t b_stride_n,
                   void *C, int64_t ldc, gemm_dtype_t c_dtype,
                   float alpha, float beta,
                   const float *bias, gemm_epilogue_t epilogue,
                   void *workspace, size_t workspace_bytes,
                   gemm_stream_t stream);

/*
 * Scales of gemm_ex, each a DEVICE pointer read when the kernel runs (so a
 * scale computed by an earlier kernel needs no host round trip), each
 * optional (NULL = absent):
 *   alpha_scale  fp32[1]  per-tensor product scale, e.g. s_a * s_b of fp8 operands;
 *   row_scale    fp32[M]  per row of A / C (per token);
 *   col_scale    fp32[N]  per column of B / C (per output channel);
 *   out_scale    fp32[1]  E4M3 output only: C stores y / out_scale[0] (NULL = 1),
 *                         rounded to nearest even and saturated to +-448;
 *   amax         fp32[1]  raised atomically to max |y| over the M x N outputs,
 *                         y being the activated value (plus the residual)
 *                         before out_scale and the cast; the caller sets it
 *                         (e.g. to 0) beforehand.
 *   residual     M x ldr row-major array of the OUTPUT type (F32, F16 or BF16;
 *                         not with an E4M3 output), added after the activation:
 *                         y = act(z) + residual[i][j] -- the post-activation
 *                         residual of a transformer block.  ldr >= N (elements);
 *                         columns N..ldr-1 are never read.  It must not overlap
 *                         C.  NULL = none (ldr ignored).
 * The product term becomes alpha * alpha_scale[0] * row_scale[i] *
 * col_scale[j] * sum_k A[i][k] B[k][j]; beta*C, the bias and the residual are
 * not scaled.  ("Case Study: Steel's BlockMMA", the paragraph on the ending
 * where fusion plugs in: the epilogue is a functor applied to every
 * accumulator before the store; these are its per-row / per-column forms, the
 * fp8 output with its amax the quantising store of a low-precision path, and
 * the residual one more input of that functor.)
 */
typedef struct {
    const float *alpha_scale;
    const float *row_scale;
    const float *col_scale;
    const float *out_scale;
    float *amax;
    const void *residual;
    int64_t ldr;
} gemm_scales_t;

/*
 * gemm_ex -- gemm() with the scales and the residual above (scales may be
 * NULL: then exactly gemm()).  Same arguments, conventions and errors, plus
 * c_dtype E4M3 (fp8 output, from F16, BF16 or E4M3 inputs, beta == 0;
 * otherwise GEMM_ERR_UNSUPPORTED).  The scale and residual arrays are checked
 * against their device allocations like every other buffer; a residual with
 * an E4M3 output is GEMM_ERR_UNSUPPORTED, ldr < N GEMM_ERR_INVALID_ARG.  With
 * K == 0 or alpha == 0 the product scales are not read (out_scale, amax and
 * the residual still apply).
 */
gemm_status_t gemm_ex(int64_t M, int64_t N, int64_t K,
                      gemm_dtype_t ab_dtype,
                      const void *A, int64_t a_stride_m, int64_t a_stride_k,
                      const void *B, int64_t b_stride_k, int64_t b_stride_n,
                      void *C, int64_t ldc, gemm_dtype_t c_dtype,
                      float alpha, float beta,
                      const float *bias, gemm_epilogue_t epilogue,
                      const gemm_scales_t *scales,
                      void *workspace, size_t workspace_bytes,
                      gemm_stream_t stream);

/*
 * gemm_workspace_size -- bytes of device scratch that let gemm() use its
 * fastest path.  fp16 / bf16 / fp8 inputs: the stream-K schedule on the
 * current device, 256 KB of partial sums and 64 bytes of flags per pair of SMs
 * (about 19 MB on a 152-SM GB300), independent of M, N, K; 0 when the device
 * cannot be queried.  fp32 inputs: the 3xTF32 split of both operands, hi and
 * lo copies in K-major rows padded to 16 bytes, 2*(M+N)*ceil4(K)*4 bytes
 * (each half rounded up to 256); with it gemm() runs fp32 on the tensor
 * cores, without it on the FFMA kernel.  Never fails.
 */
size_t gemm_workspace_size(int64_t M, int64_t N, int64_t K, gemm_dtype_t ab_dtype);

/* How the tcgen05 pair kernel distributes tiles (a per-thread setting). */
typedef enum {
    GEMM_SCHED_AUTO = 0,     /* stream-K for the last waves when the tiles do not divide evenly */
    GEMM_SCHED_TILES = 1,    /* whole tiles only */
    GEMM_SCHED_STREAM_K = 2  /* every tile's k-blocks in one range split over all SM pairs */
} gemm_schedule_t;

/*
 * gemm_set_schedule -- schedule of the calling thread's later gemm() calls on
 * the pair kernel (stream-K still needs a large enough workspace); other
 * threads keep their own setting.  Meant for tuning and tests.
 * GEMM_ERR_INVALID_ARG for an unknown value; never touches the device.
 */
gemm_status_t gemm_set_schedule(gemm_schedule_t schedule);

/*
 * Operand order of the pair kernel.  The kernel can compute C = A*B as
 * C^T = B^T * A^T, with B's transpose as the MMA's first operand and C^T's
 * rows written as C's columns.  On GB300 a second MMA operand that is
 * N-contiguous (B stored K x N row-major) keeps the tensor pipe measurably
 * less busy than a K-contiguous one (79.5 % vs 86.5 % of cycles, bf16
 * 8192^3), so AUTO transposes exactly that case for fp16 / bf16 inputs: A
 * K-contiguous, B N-contiguous, 16-bit output, C base, pitch and row length
 * usable by TMA (multiples of 16 bytes; fp8 inputs measured no faster transposed and keep the given order).
 * The result is the same product; only the summation order inside fp32
 * accumulation may differ.
 */
typedef enum {
    GEMM_ORDER_AUTO = 0,        /* transpose when it is the faster orientation (above) */
    GEMM_ORDER_AS_GIVEN = 1,    /* never transpose */
    GEMM_ORDER_TRANSPOSED = 2   /* transpose whenever the output allows (16-bit, TMA-able C) */
} gemm_operand_order_t;

/*
 * gemm_set_operand_order -- operand order of the calling thread's later
 * gemm() calls on the pair kernel; other threads keep their own setting.
 * Meant for tuning and tests.  GEMM_ERR_INVALID_ARG for an unknown value;
 * never touches the device.
 */
gemm_status_t gemm_set_operand_order(gemm_operand_order_t order);

/*
 * Cluster shape of the pair kernel.  A cluster can hold two SM pairs that
 * compute two output tiles side by side along N, over the same rows of A:
 * each CTA then fetches half of its A rows and the TMA multicasts them to the
 * CTA in the same place of the other pair, so every A panel crosses from L2
 * to shared memory once per two tiles (a quarter fewer operand bytes per SM).
 * Tiles, results and the summation order are the same either way.  Four-CTA
 * clusters may fit on fewer SMs (GB300: 144 of 152), so AUTO uses them where
 * that costs less than the traffic saves: when the tile columns pair up
 * evenly and either no SM is lost or the problem has at most four waves of
 * tiles.  Both shapes need A's tile rows to split into whole TMA boxes (any
 * K-contiguous A; an M-contiguous A with 16-bit elements).  ON forces
 * two-pair clusters wherever A splits, even with an odd number of tile
 * columns (the last pair then computes a tile outside the matrix and stores
 * nothing).
 *
 * A multicast load's tensor map may cover only the calling GPU's own memory:
 * the pair kernel's first operand (A, or B when it computes C^T = B^T A^T)
 * must be a device allocation of the current device, else the call runs
 * one-pair clusters whatever the setting (pinned host memory or another
 * GPU's memory is read by plain per-CTA TMA loads).
 */
typedef enum {
    GEMM_MCAST_AUTO = 0,   /* two-pair clusters where they measured faster (above) */
    GEMM_MCAST_OFF = 1,    /* one pair per cluster */
    GEMM_MCAST_ON = 2      /* two pairs per cluster wherever A's rows split between them */
} gemm_multicast_t;

/*
 * gemm_set_multicast -- cluster shape of the calling thread's later gemm()
 * calls on the pair kernel; other threads keep their own setting.  Meant for
 * tuning and tests.  GEMM_ERR_INVALID_ARG for an unknown value; never touches
 * the device.
 */
gemm_status_t gemm_set_multicast(gemm_multicast_t mode);

/*
 * gemm_query_path -- validate the same arguments gemm() takes and report, in
 * *path (host pointer), which kernel family gemm() would launch.  Launches
 * nothing and touches no device memory.  Returns the status gemm() would
 * return before enqueueing.
 */
gemm_status_t gemm_query_path(int64_t M, int64_t N, int64_t K,
                              gemm_dtype_t ab_dtype,
                              const void *A, int64_t a_stride_m, int64_t a_stride_k,
                              const void *B, int64_t b_stride_k, int64_t b_stride_n,
                              const void *C, int64_t ldc, gemm_dtype_t c_dtype,
                              float alpha, float beta,
                              const float *bias, gemm_epilogue_t epilogue,
                              gemm_path_t *path);

/* Tile policy of the tcgen05 path (a per-thread setting; see gemm_set_tile_policy). */
typedef enum {
    GEMM_TILE_AUTO = 0,     /* cost model: wave balance over the SMs and shared-memory bandwidth */
    GEMM_TILE_1SM_256 = 1,  /* one SM per 128 x 256 output tile */
    GEMM_TILE_1SM_128 = 2,  /* one SM per 128 x 128 output tile */
    GEMM_TILE_PAIR = 3      /* a cluster of two SMs per 256 x bn output tile (cta_group::2 MMA) */
} gemm_tile_policy_t;

/*
 * gemm_set_tile_policy -- choose how the calling thread's later gemm() calls
 * tile the output on the tcgen05 path; other threads keep their own setting.
 * `bn` is used with
 * GEMM_TILE_PAIR only: a multiple of 32 in 128..256, or 0 to let the cost
 * model pick the width.  Meant for tuning and tests; GEMM_TILE_AUTO (the
 * default) is the right choice otherwise.  Returns GEMM_ERR_INVALID_ARG for an
 * unknown policy or width; never touches the device.
 */
gemm_status_t gemm_set_tile_policy(gemm_tile_policy_t policy, int bn);

/*
 * gemm_query_tile -- the tile the tcgen05 path would use on the current device
 * for an M x N x K problem: *kind = 1 for one SM per tile, 2 for a pair of SMs;
 * *bn = tile width; *units = tiles in flight at once (CTAs, or two-CTA
 * clusters).  All three are host pointers.  Reads device attributes; launches
 * nothing.  GEMM_ERR_CUDA if the device cannot be queried.
 */
gemm_status_t gemm_query_tile(int64_t M, int64_t N, int64_t K, gemm_dtype_t ab_dtype, gemm_dtype_t c_dtype,
                              int *kind, int *bn, int *units);

/*
 * What the calling thread's last gemm() (or gemm_builtin_scratch()) call
 * enqueued, for tuning, tests and reports.  No counterpart on the pages.
 */
typedef struct {
    int path;          /* gemm_path_t of the kernel family launched (NOOP when nothing was) */
    int kind;          /* tcgen05 path: 1 one SM per tile, 2 a pair of SMs per tile; SIMT path of the grouped
                          and 8-bit products: 3 their streaming kernel for few rows; else 0 */
    int bn;            /* tcgen05 path: tile width in columns of the MMA's output; kind 3: rows of a tile */
    int transposed;    /* 1 when the pair kernel ran C^T = B^T A^T */
    int cluster_ctas;  /* CTAs per cluster: 1 (one-SM kernel), 2 (one pair) or 4 (two pairs sharing A) */
    int grid_ctas;     /* CTAs of the tcgen05 GEMM kernel (0 on the other paths) */
    int tiles;         /* its scheduling units: output tiles, or pairs of tiles side by side for
                          4-CTA clusters (0 on the other paths) */
    int stream_k_tiles;/* of those, units whose k-blocks are split over all clusters */
    int tf32x3;        /* 1 when fp32 inputs ran as 3xTF32 (split pre-pass + tensor cores) */
} gemm_launch_info_t;

/*
 * gemm_last_launch -- copy the calling thread's record of its last gemm()
 * call that returned GEMM_OK into *info (host pointer).  A call that failed
 * leaves the record as it was.  GEMM_ERR_INVALID_ARG for info == NULL.
 * Touches no device.
 */
gemm_status_t gemm_last_launch(gemm_launch_info_t *info);

/*
 * gemm_builtin_scratch -- gemm() for callers that cannot allocate device
 * memory.  (The pages have no counterpart: this is a deployment convenience
 * of this library, not part of the method.)
 *
 * gemm() takes the stream-K scratch (partial sums and ready flags) from a
 * workspace the caller allocates.  Code that cannot call cudaMalloc or any
 * allocating routine where it multiplies -- inside CUDA stream capture, on
 * real-time paths, or in processes whose device memory belongs to another
 * allocator -- calls this instead: same arguments and result as gemm()
 * without the workspace pair, with the scratch taken from a fixed array of
 * 20,976,640 bytes (enough for 80 pairs of SMs) that the library reserves in
 * device memory on every device that loads it, for as long as it is loaded.
 * It allocates nothing.
 *
 *   - The first call on a device looks the array's device address up
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.
 *   - Every call shares the one array and leaves its contents behind; nothing
 *     in it needs clearing between calls.  Calls that overlap on the GPU (on
 *     different streams, or from different threads) race on it: serialise
 *     them.
 *   - A device with more than 80 pairs of SMs needs a larger stream-K
 *     workspace than the array holds: such calls return GEMM_ERR_WORKSPACE
 *     (use gemm() with a workspace there).
 *   - fp32 inputs run on the CUDA-core FFMA kernel here, as gemm() without a
 *     workspace does: the 3xTF32 split needs a workspace that grows with M,
 *     N and K, which no fixed array can hold (about 8x slower at 4096^3).
 *   - Other errors as gemm().
 */
gemm_status_t gemm_builtin_scratch(int64_t M, int64_t N, int64_t K,
                                   gemm_dtype_t ab_dtype,
                                   const void *A, int64_t a_stride_m, int64_t a_stride_k,
                                   const void *B, int64_t b_stride_k, int64_t b_stride_n,
                                   void *C, int64_t ldc, gemm_dtype_t c_dtype,
                                   float alpha, float beta,
                                   const float *bias, gemm_epilogue_t epilogue,
                                   gemm_stream_t stream);

/*
 * gemm_bias_gelu -- the UNFUSED second pass, for measuring what fusion saves
 * (Rigel abstract: fused GEMM + bias + GELU against the decomposed path):
 * C[i][j] = cast(GELU(C[i][j] + bias[j])) in place, for an M x N block of an
 * M x ldc row-major buffer of type c_dtype (F32, F16 or BF16).  bias is fp32[N]
 * on the device.  Asynchronous on `stream`; same error behaviour as gemm().
 */
gemm_status_t gemm_bias_gelu(int64_t M, int64_t N, void *C, int64_t ldc, gemm_dtype_t c_dtype,
                             const float *bias, gemm_stream_t stream);

/*
 * Products with 4-bit group-quantized weights.  "X3: Metal GEMM" section 7
 * names quantized matmul -- a memory-bound GEMV when decoding, a GEMM when
 * filling the prompt -- as the main LLM workload; the pages give no storage
 * format, so this library takes the affine one with groups of 64 along K:
 *
 *     W[n][k] = s[n][k/64] * q[n][k] + b[n][k/64],   q[n][k] in 0..15,
 *
 * W being N x K (output features x input features).
 *   Wq          N*K/8 32-bit words, 16-byte aligned: q[n][k] is bits
 *               4*(k%8) .. 4*(k%8)+3 of word n*K/8 + k/8.
 *   scale_bias  N*K/64 pairs of binary16 values (s, b), in that order, one
 *               pair per group (n, g) at pair index n*K/64 + g; 4-byte aligned.
 */

/*
 * gemm_q4 -- C = cast(epilogue(alpha * x W^T + beta*C + bias)) for M rows of
 * x (M == 0 or N == 0 is a no-op).
 *   x_dtype     F16 or BF16.  X is M x ldx row-major, 16-byte aligned base,
 *               ldx >= K with ldx*2 a multiple of 16.
 *   K           a multiple of 64.
 *   C, c_dtype, ldc, alpha, beta, bias, epilogue: as in gemm(), with the
 *               output M x N and bias fp32[N]; the same fused epilogues.
 * Decode (1 <= M <= 8) runs an HBM-streaming kernel (gemm_q4_kernel_t below).
 * Prefill (M > 8) runs on the tensor cores with the dequantisation fused in:
 * each 64-k group of W is expanded to x's 16-bit type, round(s*q + b), straight
 * into tensor memory as the MMA's operand (never written to memory), and
 * multiplied with x in fp32 accumulation -- the rounding of W that
 * gemm_q4_dequantize followed by gemm() also has (at most 2^-11 of each |W|
 * for F16 x, 2^-8 for BF16).  Asynchronous on `stream`; errors as gemm().
 */
gemm_status_t gemm_q4(int64_t M, int64_t N, int64_t K, gemm_dtype_t x_dtype,
                      const void *X, int64_t ldx,
                      const uint32_t *Wq, const void *scale_bias,
                      void *C, int64_t ldc, gemm_dtype_t c_dtype,
                      float alpha, float beta,
                      const float *bias, gemm_epilogue_t epilogue,
                      gemm_stream_t stream);

/*
 * gemm_q4_ws -- gemm_q4 with a caller-owned workspace, for long prompts.  The
 * fused prefill converts each 64-k group of W once per 128 rows of x, so from
 * a few hundred rows of x up it is faster to expand W once into 16 bits and
 * run the dense tensor-core kernel (GB300, N = K = 4096: fused 31 / 33 / 60 /
 * 187 us at M = 64 / 256 / 1024 / 4096 against 35 / 35 / 37 / 93 us for
 * gemm_q4_dequantize + gemm()).  When gemm_q4_workspace_size(M, N, K,
 * x_dtype) is non-zero and the workspace (256-byte aligned device memory, not
 * overlapping any operand) holds that many bytes, the call does exactly
 * that: W into the workspace as x_dtype (the same rounding of W as the fused
 * kernel), then gemm() with the rest of the workspace for its partial sums.
 * Otherwise it runs gemm_q4.  Same arguments, results within the same
 * tolerances, and errors as gemm_q4; asynchronous on `stream`.
 */
gemm_status_t gemm_q4_ws(int64_t M, int64_t N, int64_t K, gemm_dtype_t x_dtype,
                         const void *X, int64_t ldx,
                         const uint32_t *Wq, const void *scale_bias,
                         void *C, int64_t ldc, gemm_dtype_t c_dtype,
                         float alpha, float beta,
                         const float *bias, gemm_epilogue_t epilogue,
                         void *workspace, size_t workspace_bytes,
                         gemm_stream_t stream);

/*
 * gemm_q4_workspace_size -- bytes of workspace gemm_q4_ws uses for this shape:
 * 0 below GEMM_Q4_DEQUANT_ROWS rows of x (the fused kernel is faster there) or
 * for an x_dtype other than F16 / BF16, else the 16-bit W (256-byte rounded)
 * plus gemm_workspace_size(M, N, K, x_dtype).  Pure function of its
 * arguments; touches no device.
 */
#define GEMM_Q4_DEQUANT_ROWS 384
size_t gemm_q4_workspace_size(int64_t M, int64_t N, int64_t K, gemm_dtype_t x_dtype);

/*
 * The kernel behind gemm_q4.  Both compute the same sums (per 64-k group,
 * s * sum_k x q + b * sum_k x, in fp32) and meet the same tolerances; they
 * differ in how the weights move and where the products are formed.
 */
typedef enum {
    GEMM_Q4_AUTO = 0,   /* the one measured faster for the number of rows of x */
    GEMM_Q4_FFMA = 1,   /* CUDA-core kernel: 16-byte loads into registers, codes to fp32, f32x2 multiply-add */
    GEMM_Q4_MMA = 2     /* tensor-core kernel: codes and x staged in shared memory by bulk copies, exact
                           16-bit codes times x by mma.sync.m16n8k16 (rows of x as the 8 columns) */
} gemm_q4_kernel_t;

/*
 * gemm_set_q4_kernel -- kernel of the calling thread's later gemm_q4() calls;
 * other threads keep their own setting.  Meant for tuning and tests.
 * GEMM_ERR_INVALID_ARG for an unknown value; never touches the device.
 */
gemm_status_t gemm_set_q4_kernel(gemm_q4_kernel_t kind);

/*
 * The calling thread's tuning settings, as the gemm_set_* calls left them
 * (every thread starts with all of them AUTO and bn 0).  No counterpart on
 * the pages.
 */
typedef struct {
    int tile_policy;    /* gemm_tile_policy_t */
    int tile_bn;        /* pair tile width forced with GEMM_TILE_PAIR, 0 = cost model */
    int schedule;       /* gemm_schedule_t */
    int operand_order;  /* gemm_operand_order_t */
    int multicast;      /* gemm_multicast_t */
    int q4_kernel;      /* gemm_q4_kernel_t */
} gemm_tuning_t;

/*
 * gemm_get_tuning -- copy the calling thread's settings into *out (host
 * pointer).  GEMM_ERR_INVALID_ARG for out == NULL; touches no device.
 */
gemm_status_t gemm_get_tuning(gemm_tuning_t *out);

/*
 * gemm_q4_dequantize -- W[n][k] = round(s*q + b) into the N x K row-major
 * device array W of type w_dtype (F16 or BF16; 16-byte aligned), for
 * gemm(M, N, K, w_dtype, X, ldx, 1, W, 1, K, ...) to multiply (W^T as B,
 * K-contiguous) -- the unfused alternative to gemm_q4's prefill, for a W
 * used by many calls.  The rounding to 16 bits is the only difference from the
 * exact product: at most 2^-11 (F16) or 2^-8 (BF16) of each |W| value.
 * K a multiple of 64.  Asynchronous on `stream`; errors as gemm().
 */
gemm_status_t gemm_q4_dequantize(int64_t N, int64_t K, const uint32_t *Wq, const void *scale_bias,
                                 void *W, gemm_dtype_t w_dtype, gemm_stream_t stream);

/*
 * Block-scaled ("microscaling", MX) products.  Rigel section 1 lists fp4 and
 * block-scaled MXFP4 next to fp8 among the low-precision rows of the matrix
 * units without defining them; the formats here are those of the OCP
 * Microscaling Formats (MX) specification v1.0.  Each block of 32 consecutive
 * k of a row shares one scale, an E8M0 code c standing for 2^(c - 127) (0xFF:
 * NaN), and each element is an E4M3 (MXFP8) or E2M1 (MXFP4) number:
 *
 *     a[i][k] = 2^(a_scale[i][k/32] - 127) * PA[i][k],  b[k][j] likewise with
 *     b_scale[j][k/32] and PB[j][k]
 *     C = cast(epilogue(alpha * sum_k a[i][k] b[k][j] + beta*C + bias))
 *
 * with gemm()'s epilogues, output types (F32, F16, BF16) and conventions.
 */
typedef enum {
    GEMM_MX_E4M3 = 0,   /* MXFP8: one E4M3 element per byte */
    GEMM_MX_E2M1 = 1    /* MXFP4: two E2M1 elements per byte, even k in the low nibble */
} gemm_mx_elem_t;

/*
 * gemm_mx -- the block-scaled product above on the tensor cores
 * (tcgen05.mma kind::mxf8f6f4 / kind::mxf4, scales applied by the MMA): up
 * to 128 rows of A one SM per 128 x 256 output tile, beyond that SM pairs
 * (cta_group::2) per 256 x 256 tile.
 *   K              a multiple of 32 (whole scale blocks); M, N, K >= 0.
 *   A, lda         M x K elements, row-major (K-contiguous), row pitch lda
 *                  ELEMENTS (lda >= K; even for E2M1).  16-byte aligned base,
 *                  row pitch a multiple of 16 bytes, else GEMM_ERR_MISALIGNED.
 *   a_scale        M x K/32 E8M0 codes, row-major (pitch K/32 bytes), device.
 *   B, ldb         B given as its transpose: N x K elements, K-contiguous, row
 *                  pitch ldb elements, same alignment rules.
 *   b_scale        N x K/32 E8M0 codes, row-major.
 *   C, ldc, c_dtype, alpha, beta, bias, epilogue: as in gemm() (c_dtype F32,
 *                  F16 or BF16; alpha == 0 or K == 0 reads neither operands
 *                  nor scales).
 *   workspace      device scratch, 256-byte aligned, of at least
 *                  gemm_mx_workspace_size() bytes (GEMM_ERR_WORKSPACE
 *                  otherwise): the scales rearranged for the tensor cores.
 *                  Calls sharing it must not overlap; no initialisation needed.
 * Asynchronous on `stream`; errors as gemm().
 */
gemm_status_t gemm_mx(int64_t M, int64_t N, int64_t K, gemm_mx_elem_t elem,
                      const void *A, int64_t lda, const uint8_t *a_scale,
                      const void *B, int64_t ldb, const uint8_t *b_scale,
                      void *C, int64_t ldc, gemm_dtype_t c_dtype,
                      float alpha, float beta,
                      const float *bias, gemm_epilogue_t epilogue,
                      void *workspace, size_t workspace_bytes,
                      gemm_stream_t stream);

/*
 * gemm_mx_workspace_size -- bytes of workspace gemm_mx needs: 512 bytes per
 * 128 rows of A and of B per 128 (E4M3) or 256 (E2M1) k, each half rounded up
 * to 256 bytes.  0 for invalid sizes (K not a multiple of 32).  Never fails,
 * touches no device.
 */
size_t gemm_mx_workspace_size(int64_t M, int64_t N, int64_t K, gemm_mx_elem_t elem);

/*
 * Baselines of the cheap-baseline gate (Rigel section 3; section 4, signal
 * 2): a claim that the tensor path is fast stands only once the trivial
 * explanations have run and lost -- a GEMM on the ordinary ALUs, and the
 * legacy warp-matrix instruction (simdgroup_matrix on the pages).  For
 * measurement and tests only; gemm() never runs them.
 */
typedef enum {
    GEMM_BASELINE_SIMT = 0,     /* threadgroup-tiled CUDA-core FFMA kernel (no matrix instructions) */
    GEMM_BASELINE_MMA_SYNC = 1  /* warp-level mma.sync.m16n8k16 kernel, fp16 / bf16 inputs */
} gemm_baseline_t;

/*
 * gemm_baseline -- the same operation and arguments as gemm() (no workspace),
 * computed by the baseline kernel `kind`.  GEMM_BASELINE_SIMT takes every
 * combination gemm() takes.  GEMM_BASELINE_MMA_SYNC takes F16 or BF16 inputs
 * whose operands are TMA-streamable in gemm()'s sense (one unit stride,
 * 16-byte aligned base and other stride) and whose contiguous extents (K for
 * a K-contiguous operand, M or N otherwise) are multiples of 8; anything else
 * returns GEMM_ERR_UNSUPPORTED.  K == 0, alpha == 0, M == 0 and N == 0
 * behave as in gemm().  Asynchronous on `stream`; errors as gemm().
 */
gemm_status_t gemm_baseline(gemm_baseline_t kind, int64_t M, int64_t N, int64_t K,
                            gemm_dtype_t ab_dtype,
                            const void *A, int64_t a_stride_m, int64_t a_stride_k,
                            const void *B, int64_t b_stride_k, int64_t b_stride_n,
                            void *C, int64_t ldc, gemm_dtype_t c_dtype,
                            float alpha, float beta,
                            const float *bias, gemm_epilogue_t epilogue,
                            gemm_stream_t stream);

/*
 * gemm_device_status -- synchronise `stream`, then return and clear the
 * device-side status word of the current device: GEMM_ERR_TIMEOUT if any
 * kernel gave up on a bounded wait since the last call, GEMM_ERR_CUDA if the
 * synchronisation itself failed, GEMM_OK otherwise.
 */
gemm_status_t gemm_device_status(gemm_stream_t stream);

/*
 * Products grouped by expert.  A mixture of experts sends each row (token) to
 * some of G experts; with the rows sorted by expert, the rows of expert g are
 * rows offsets[g] .. offsets[g+1]-1 of one array, and each expert multiplies
 * its own rows.  The pages know one matrix product per call; this is G of them
 * with ragged row counts in one launch, for the same epilogues.
 *
 *   offsets        int32[G + 1] on the DEVICE, non-decreasing, 0 <= offsets <=
 *                  M.  The host never reads it: a router's counts need no copy
 *                  back.  Groups may be empty; rows below offsets[0] or from
 *                  offsets[G] on are not touched.  Values outside these rules
 *                  are clamped to [0, M], one below an earlier one to that
 *                  (no access leaves the arrays and no row of C is written
 *                  twice), with unspecified results.  At most
 *                  GEMM_MAX_GROUPS groups.
 *
 * M, N, K (and T) of these and of the 8-bit products are at most
 * GEMM_GROUPED_MAX_EXTENT; larger ones are GEMM_ERR_UNSUPPORTED.
 */
#define GEMM_MAX_GROUPS 1024
#define GEMM_GROUPED_MAX_EXTENT 2147482624 /* 2^31 - 1024 */

/*
 * gemm_grouped -- for every row r of group g and every column j:
 *
 *     z = alpha * row_scale[r] * sum_k A[r][k] * B[g][k][j] + beta * C[r][j] + bias[g][j]
 *     C[r][j] = cast(act(z))
 *
 * with fp32 accumulation and rounding to nearest even once.
 *   A              element (r, k) at A[r*a_stride_m + k*a_stride_k], M rows.
 *   B              element (g, k, j) at B[g*b_stride_g + k*b_stride_k + j*b_stride_n].
 *                  Weights stored G x N x K are b_stride_k = 1, b_stride_n =
 *                  their pitch; swapping the two strides multiplies by the
 *                  transposed weights, which is the gradient of the rows.
 *   C, ldc         M x ldc row-major, as in gemm().
 *   types          ab_dtype F16 or BF16 with c_dtype F32, F16 or BF16; or all F32.
 *   bias           fp32[G x N] (row g: expert g's), required unless GEMM_EPI_NONE.
 *   row_scale      fp32[M] or NULL (1): e.g. the router's weight of each row.
 *                  Not read when K == 0 or alpha == 0 (the product term is 0).
 * F16 / BF16 inputs run on the tensor cores when A is contiguous along k, B
 * along k or j, both bases are 16-byte aligned and the other strides multiples
 * of 16 bytes; anything else on the CUDA cores.  The activations take the
 * forms of fp32 outputs whatever c_dtype.  C must not overlap the inputs.
 * Asynchronous on `stream`; errors as gemm(), GEMM_ERR_MISALIGNED for an
 * array that is read or written and does not start at a multiple of its
 * element's size.
 */
gemm_status_t gemm_grouped(int64_t G, int64_t M, int64_t N, int64_t K, gemm_dtype_t ab_dtype, const int32_t *offsets,
                           const void *A, int64_t a_stride_m, int64_t a_stride_k, const void *B, int64_t b_stride_g,
                           int64_t b_stride_k, int64_t b_stride_n, void *C, int64_t ldc, gemm_dtype_t c_dtype,
                           float alpha, float beta, const float *bias, gemm_epilogue_t epilogue,
                           const float *row_scale, gemm_stream_t stream);

/*
 * gemm_grouped_wgrad -- the weight gradient of gemm_grouped: for every group g,
 *
 *     C[g][m][n] = cast(alpha * sum_{r in g} A[r][m] * D[r][n] + beta * C[g][m][n])
 *     a_sum[g][m] = alpha * sum_{r in g} A[r][m] + beta * a_sum[g][m]
 *
 * over the T rows of A (T x M) and D (T x N), element (r, m) at
 * A[r*a_stride_r + m*a_stride_m], D likewise.  With A = the gradient of the
 * rows' outputs and D = the rows, C[g] is the gradient of weights stored N x K
 * and a_sum the gradient of the bias; beta = 1 accumulates into main gradients.
 * A group without rows gets beta * C[g] (zeros for beta == 0, C unread).
 *   C              element (g, m, n) at C[g*c_stride_g + m*ldc + n]; the groups
 *                  must not overlap (c_stride_g >= (M-1)*ldc + N).
 *   a_sum          fp32[G x M] or NULL.
 *   types          as gemm_grouped.
 * Sums run in a fixed order: the same call gives the same bits.  F16 / BF16
 * inputs run on the tensor cores when both are contiguous along m / n with
 * 16-byte aligned bases and row pitches.  Errors as gemm_grouped.
 */
gemm_status_t gemm_grouped_wgrad(int64_t G, int64_t T, int64_t M, int64_t N, gemm_dtype_t ab_dtype,
                                 const int32_t *offsets, const void *A, int64_t a_stride_r, int64_t a_stride_m,
                                 const void *D, int64_t d_stride_r, int64_t d_stride_n, void *C, int64_t c_stride_g,
                                 int64_t ldc, gemm_dtype_t c_dtype, float alpha, float beta, float *a_sum,
                                 gemm_stream_t stream);

/*
 * Products of 8-bit integers with a scale for each row (token) and each output
 * channel: "X3: Metal GEMM" section 7's quantized matmul with the rows quantised
 * too.
 *
 * gemm_i8 -- C[i][j] = cast(act(alpha * x_scale[i] * w_scale[j] * sum_k
 * X[i][k] * W[j][k] + beta * C[i][j] + bias[j])).
 *   X, ldx         int8, M x ldx row-major, ldx >= K.
 *   W, ldw         int8, N x ldw row-major, ldw >= K (output channels x inputs).
 *   x_scale        fp32[M] or NULL (1); w_scale fp32[N] or NULL (1).  Not read
 *                  when K == 0 or alpha == 0.
 *   K              at most GEMM_I8_MAX_K: the integer sum is exact (32 bits)
 *                  for all codes -128 .. 127, so the result does not depend on
 *                  M or on the kernel that a call runs.  It is rounded to fp32
 *                  once, scaled, and rounded to c_dtype (F32, F16 or BF16).
 *   bias           fp32[N]; C, ldc, alpha, beta, epilogue as in gemm().
 * Any alignment of the codes; 16-byte aligned bases and pitches run on the
 * fast kernels.  The other arrays as in gemm_grouped.
 *
 * gemm_i8_grouped -- the same, grouped by expert: rows of group g use W[g] =
 * W + g*w_stride_g, w_scale[g] and bias[g] (fp32[G x N] each); offsets as in
 * gemm_grouped.
 */
#define GEMM_I8_MAX_K 131071
gemm_status_t gemm_i8(int64_t M, int64_t N, int64_t K, const int8_t *X, int64_t ldx, const float *x_scale,
                      const int8_t *W, int64_t ldw, const float *w_scale, void *C, int64_t ldc, gemm_dtype_t c_dtype,
                      float alpha, float beta, const float *bias, gemm_epilogue_t epilogue, gemm_stream_t stream);
gemm_status_t gemm_i8_grouped(int64_t G, int64_t M, int64_t N, int64_t K, const int32_t *offsets, const int8_t *X,
                              int64_t ldx, const float *x_scale, const int8_t *W, int64_t w_stride_g, int64_t ldw,
                              const float *w_scale, void *C, int64_t ldc, gemm_dtype_t c_dtype, float alpha,
                              float beta, const float *bias, gemm_epilogue_t epilogue, gemm_stream_t stream);

/*
 * gemm_i8_quantize -- the rows that gemm_i8 takes, from F32, F16 or BF16 values:
 *
 *     scale[i] = max_k |X[i][k]| / 127,   Q[i][k] = round_even(127 * X[i][k] / max_k |X[i][k]|)
 *
 * A row of zeros (or K == 0) gets scale 0 and codes 0.  A row that holds a NaN
 * or an infinity gets a NaN scale, so that the product's row shows it, and
 * codes 0.  Columns K..ldq-1 of Q are not written.  X and scale start at a
 * multiple of their element's size (else GEMM_ERR_MISALIGNED).
 */
gemm_status_t gemm_i8_quantize(int64_t M, int64_t K, gemm_dtype_t x_dtype, const void *X, int64_t ldx, int8_t *Q,
                               int64_t ldq, float *scale, gemm_stream_t stream);

/*
 * Block-scaled rows and products for experts: the formats of gemm_mx (a shared
 * power of two per 32 k, E4M3 or E2M1 elements), with a pitch for the scales.
 *
 * gemm_mx_quantize -- M rows of K values (K a multiple of 32) to codes and scales:
 *
 *     scale[i][b] = clamp(floor(log2 max |x|) - emax + 127, 0, 254), the maximum over x[i][32 b .. 32 b + 31]
 *     Q[i][k]     = round_even(x[i][k] * 2^(127 - scale)), saturated
 *
 * with emax 2 (E2M1, largest 6) or 8 (E4M3, largest 448).  A block of zeros gets
 * scale 0, one that holds a NaN or an infinity 0xFF (NaN) and elements 0.
 *   X, x_dtype     F32, F16 or BF16, rows_x rows, pitch ldx >= K.
 *   source         int32[M] on the device, or NULL.  Row i is row source[i] / top
 *                  of X (as gemm_route_rows has it); where that is none of X's
 *                  rows (source[i] < 0, or past the last), row i of Q and its
 *                  scales are left as they were.  NULL: row i of X (rows_x >= M,
 *                  top not used).
 *   Q, ldq         M rows of pitch ldq elements (even for E2M1), as gemm_mx's A.
 *   scale, lds     M rows of K/32 codes, pitch lds bytes.
 * Any alignment of bytes; 16-byte aligned rows of X are read faster, and gemm_mx_grouped
 * wants pitches of Q and scale of whole 16 bytes.
 *
 * gemm_mx_dequantize -- Y[i][k] = cast(Q[i][k] * 2^(scale - 127)) as F32, F16 or
 * BF16 (exact before the cast); e.g. weights for gemm_grouped's gradients.
 */
gemm_status_t gemm_mx_quantize(int64_t M, int64_t K, gemm_mx_elem_t elem, gemm_dtype_t x_dtype, const void *X,
                               int64_t ldx, int64_t rows_x, const int32_t *source, int64_t top, void *Q, int64_t ldq,
                               uint8_t *scale, int64_t lds, gemm_stream_t stream);
gemm_status_t gemm_mx_dequantize(int64_t M, int64_t K, gemm_mx_elem_t elem, const void *Q, int64_t ldq,
                                 const uint8_t *scale, int64_t lds, gemm_dtype_t y_dtype, void *Y, int64_t ldy,
                                 gemm_stream_t stream);

/*
 * gemm_mx_grouped -- gemm_grouped over block-scaled codes: for every row r of group
 * g and every column j,
 *
 *     C[r][j] = cast(act(alpha * row_scale[r] * sum_k x[r][k] w[g][j][k] + beta * C[r][j] + bias[g][j]))
 *
 *   X, ldx         M rows of K elements; x_scale: their scales, pitch ldxs bytes.
 *   W, ldw         G matrices of N rows of K elements, w_stride_g elements apart;
 *                  w_scale: theirs, pitch ldws, ws_stride_g bytes apart.
 *   K              a multiple of 32.  Bases are 16-byte aligned, pitches and strides
 *                  multiples of 16 bytes (those of a single row or matrix are not
 *                  used), else GEMM_ERR_MISALIGNED; with G > 1 the strides between
 *                  matrices are positive.
 *   offsets        as in gemm_grouped; NULL with G == 1: one group of all rows.
 *   C, bias, row_scale, epilogue, alpha, beta: as in gemm_grouped.  K == 0 or
 *                  alpha == 0 reads neither operands, scales nor row_scale.
 * No workspace.  Sums are fp32: E4M3 ones joined in registers every 1024 k, E2M1
 * ones the tensor cores' own, exact as long as they stay below 2^24 of the smallest
 * product (a quarter of the product of two scales) and beyond that cut off by a unit
 * in the last place per 64 k at most.  Errors as gemm_grouped.
 */
gemm_status_t gemm_mx_grouped(int64_t G, int64_t M, int64_t N, int64_t K, gemm_mx_elem_t elem, const int32_t *offsets,
                              const void *X, int64_t ldx, const uint8_t *x_scale, int64_t ldxs, const void *W,
                              int64_t w_stride_g, int64_t ldw, const uint8_t *w_scale, int64_t ws_stride_g,
                              int64_t ldws, void *C, int64_t ldc, gemm_dtype_t c_dtype, float alpha, float beta,
                              const float *bias, gemm_epilogue_t epilogue, const float *row_scale,
                              gemm_stream_t stream);

/*
 * Routing: a router's logits to each token's experts, in the form that the
 * grouped products take.
 *
 * gemm_route -- for T tokens and E experts (at most GEMM_MAX_GROUPS), the `top` (at
 * most GEMM_ROUTE_MAX_TOP) chosen ones of each token and their weights:
 *
 *     s = softmax(logits over all experts) or sigmoid(logits),  sel = s + bias
 *     a group's worth is the sum of the group_sum (1 or 2) highest sel of its E / groups
 *     experts; experts outside the top_groups worthiest groups are not chosen
 *     expert[t] = those of the `top` highest sel, the highest first
 *     weight[t] = scale * s, or renormalised scale * s / (sum of the chosen s)
 *
 * Equal ones go to the lower index (expert, group).  The choice is made as by
 * 64-bit scores; without a bias and with group_sum 1, by the logits, whose order
 * the scores have.  An expert whose logit or bias is -infinity or NaN, or whose
 * group has no available expert, is not available; logits of +infinity count as the
 * largest finite number.  Where fewer than `top` are left, the other slots get
 * expert -1 and weight 0, which the calls below leave out.
 *   logits, ldl    T x E, pitch ldl, F32, F16 or BF16.
 *   bias           fp32[E] or NULL.  It moves the choice, not the weights.
 *   groups         1 (no limit; top_groups and group_sum are not used) .. GEMM_ROUTE_MAX_GROUPS,
 *                  a divisor of E; 1 <= top_groups <= groups.
 *   expert, weight int32 and fp32, T x top, contiguous.
 *
 * gemm_route_grad -- dlogits (T x E, pitch ldd, l_dtype; every element written) for
 * the weights' gradient dweight, the choice held fixed.  Takes the logits, score,
 * renormalise and scale of the forward call and its `expert`; slots whose expert is
 * outside 0 .. E-1 are left out.  The bias has no gradient.  dlogits and logits must not
 * overlap.
 */
#define GEMM_ROUTE_MAX_TOP 32
#define GEMM_ROUTE_MAX_GROUPS 32
typedef enum { GEMM_SCORE_SOFTMAX = 0, GEMM_SCORE_SIGMOID = 1 } gemm_score_t;
gemm_status_t gemm_route(int64_t T, int64_t E, int64_t top, gemm_dtype_t l_dtype, const void *logits, int64_t ldl,
                         const float *bias, gemm_score_t score, int64_t groups, int64_t top_groups, int64_t group_sum,
                         int renormalise, float scale, int32_t *expert, float *weight, gemm_stream_t stream);
gemm_status_t gemm_route_grad(int64_t T, int64_t E, int64_t top, gemm_dtype_t l_dtype, const void *logits, int64_t ldl,
                              gemm_score_t score, int renormalise, float scale, const int32_t *expert,
                              const float *dweight, void *dlogits, int64_t ldd, gemm_stream_t stream);

/*
 * gemm_route_rows -- the T x top pairs p = t * top + slot, sorted by expert: pairs
 * of one expert keep their order, so the same call gives the same rows.
 *   offsets        int32[E + 1]: what gemm_grouped and gemm_mx_grouped take.
 *   row            int32[T * top]: the row of each pair, -1 where expert is outside
 *                  0 .. E-1 (or NULL: not wanted).
 *   source         int32[T * top]: the pair of each row, -1 behind the last row.
 *   workspace      device scratch, 16-byte aligned, gemm_route_rows_workspace_size()
 *                  bytes (0 for few pairs: may be NULL).  Calls sharing it must not
 *                  overlap; no initialisation needed.
 * T * top is at most GEMM_ROUTE_MAX_PAIRS in this and the calls below.
 */
#define GEMM_ROUTE_MAX_PAIRS 1073741824 /* 2^30 */
gemm_status_t gemm_route_rows(int64_t T, int64_t top, int64_t E, const int32_t *expert, int32_t *offsets, int32_t *row,
                              int32_t *source, void *workspace, size_t workspace_bytes, gemm_stream_t stream);
size_t gemm_route_rows_workspace_size(int64_t T, int64_t top, int64_t E);

/*
 * Rows between token order (X: T rows) and expert order (Y: R rows) of D columns.
 * Indexes outside their arrays are left out; sums run in fp32 in the slots' order.
 *
 * gemm_rows_gather -- Y[r] = weight[source[r]] * X[source[r] / top] (weight NULL:
 * 1, a copy); rows whose source is none stay as they were.  Also the gradient of a
 * combination's rows.
 *
 * gemm_rows_combine -- Out[t] = cast(sum over slots of weight[t][s] * Y[row[t][s]]
 * + beta * Out[t]) (weight NULL: 1; slots without a row add nothing; Out unread for
 * beta == 0).  With weight NULL also the gradient of a gather.  Out is F32 or of
 * Y's type, or F16 / BF16 from F32 rows.
 *
 * gemm_rows_combine_grad -- dY[row[t][s]] = cast(weight[t][s] * dOut[t]) in Y's type
 * and dweight[t][s] = dOut[t] . Y[row[t][s]] (fp32; 0 without a row).  Either may
 * be NULL (not wanted; Y is not read without dweight).  dOut is F32 or of Y's type.
 * No row may be named twice, as gemm_route_rows names none; rows of dY that are not
 * named stay as they were.
 *
 * D <= GEMM_ROWS_MAX_D.  Bases and pitches of whole 16 bytes run fastest; any
 * others work.  The output must not overlap the inputs.
 */
#define GEMM_ROWS_MAX_D 8388608 /* 2^23 */
gemm_status_t gemm_rows_gather(int64_t R, int64_t D, int64_t T, int64_t top, gemm_dtype_t dtype, const void *X,
                               int64_t ldx, const int32_t *source, const float *weight, void *Y, int64_t ldy,
                               gemm_stream_t stream);
gemm_status_t gemm_rows_combine(int64_t T, int64_t top, int64_t D, int64_t R, gemm_dtype_t y_dtype, const void *Y,
                                int64_t ldy, const int32_t *row, const float *weight, float beta,
                                gemm_dtype_t out_dtype, void *Out, int64_t ldo, gemm_stream_t stream);
gemm_status_t gemm_rows_combine_grad(int64_t T, int64_t top, int64_t D, int64_t R, gemm_dtype_t d_dtype,
                                     const void *dOut, int64_t ldd, gemm_dtype_t y_dtype, const void *Y, int64_t ldy,
                                     const int32_t *row, const float *weight, void *dY, int64_t lddy, float *dweight,
                                     gemm_stream_t stream);

/*
 * gemm_wait_selftest -- exercise the bounded waits the GEMM kernels rely on
 * instead of hanging.  Enqueues on `stream` a one-warp kernel that waits on an
 * mbarrier nobody arrives at and then on *never_set (a device word the caller
 * guarantees nobody sets to 0xFFFFFFFF during the call), each for at most
 * limit_ns nanoseconds (1 .. 1e9).  Each wait that gives up records a timeout,
 * so the next gemm_device_status() returns GEMM_ERR_TIMEOUT; the CUDA context
 * stays usable.  (Failure-detection aid; the pages have no counterpart.)
 */
gemm_status_t gemm_wait_selftest(const unsigned int *never_set, uint64_t limit_ns, gemm_stream_t stream);

/* gemm_status_string -- static, NUL-terminated description of a status code. */
const char *gemm_status_string(gemm_status_t status);

/* gemm_version -- static version string of the library build. */
const char *gemm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_GB300_H */
