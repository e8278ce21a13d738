/*
 * fp32gemm — single-precision GEMM and small-M GEMV for AMD MI355X (gfx950).
 *
 * C ABI of libfp32gemm.so.  Plain pointers and sizes only; no HIP or torch
 * header is needed to call it (the stream is an opaque pointer that is
 * ABI-identical to hipStream_t).
 *
 * The operation is the one defined on the page "GPU GEMM 优化完全拆解（一）：
 * 从朴素 Kernel 到共享内存分块", section "什么是 GEMM" (A is M x K, B is K x N,
 * C is M x N, alpha and beta scalars, C <- alpha * A B + beta * C), with the
 * row-major element update of the naive kernel in "CUDA 矩阵乘法优化：从朴素
 * Kernel 到接近 cuBLAS", section "1. Kernel 1: 朴素实现".  The small-M
 * product is the decode-phase matrix-vector shape of the first page's
 * section "LLM 推理本质上是 GEMM 的串联" (M = batch, usually 1 to 8).
 *
 * Conventions shared by every entry point:
 *  - Layout: row-major fp32.  Element (i, k) of A is A[i * lda + k], element
 *    (k, j) of B is B[k * ldb + j], element (i, j) of C is C[i * ldc + j].
 *  - Memory: A, B and C are device pointers (hipMalloc / torch CUDA tensors)
 *    owned by the caller.  The library keeps no reference after the call's
 *    kernels finish.  C must not overlap A or B.
 *  - Arithmetic: fp32 throughout (fp32 MFMA or fp32 FMA); no conversion to a
 *    narrower format (the s8 routines below say what theirs is).  The order
 *    of the k-sum is unspecified, so results may differ from a sequential
 *    loop by rounding.  Repeated calls with the same arguments and
 *    configuration give bit-identical results (no atomics on floats).
 *  - Reads: when beta == 0, C is not read (NaN in C does not propagate).
 *    When alpha == 0 or K == 0, A and B are not read (they may be NULL) and
 *    C <- beta * C.  When M == 0 or N == 0 the call does nothing.
 *  - Alignment: any 4-byte alignment is accepted.  The 128-bit load path is
 *    used when A and B are 16-byte aligned and K, N, lda and ldb are
 *    multiples of 4; otherwise a 32-bit load path computes the same result.
 *  - Asynchrony: work is enqueued on `stream` (NULL = the null stream) and
 *    the call returns without synchronising.
 *  - Return value: 0 on success; -p when argument p (1-based, in the order of
 *    the routine's own parameter list) is invalid; FP32GEMM_ERR_CONFIG for an
 *    unknown configuration id; a positive hipError_t value when a HIP call or
 *    kernel launch fails.  Nothing is enqueued when a negative code is
 *    returned.
 *  - Threads: every entry point is reentrant; calls on different streams
 *    may run concurrently.  The library allocates no device memory at run
 *    time; the split-K decode kernel (see sgemv) uses device memory reserved
 *    statically when the library is loaded, per stream.
 */
#ifndef FP32GEMM_H
#define FP32GEMM_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t *fp32gemm_stream_t;

#define FP32GEMM_OK 0
#define FP32GEMM_ERR_CONFIG (-100)
#define FP32GEMM_ERR_SCRATCH (-101)

/*
 * C[M x N] <- alpha * A[M x K] . B[K x N] + beta * C.
 * Argument checks: M, N, K >= 0; lda >= max(1, K); ldb >= max(1, N);
 * ldc >= max(1, N); A and B non-NULL when alpha != 0 and K > 0; C non-NULL
 * when M > 0 and N > 0.  M <= 8 is routed to the GEMV kernel (sgemv), and
 * M = 9..128 to the skinny MFMA kernel where it is the faster (M <= 48
 * and M = 65..80 always, M <= 96 up to N = 8192, otherwise while the tiled
 * kernel has fewer than 160 64x64 tiles);
 * larger M runs the LDS-tiled fp32 MFMA kernel with the tile configuration
 * that the per-shape table selects for (M, N, K).
 */
int sgemm(int M, int N, int K, float alpha, const float *A, int lda,
          const float *B, int ldb, float beta, float *C, int ldc,
          fp32gemm_stream_t stream);

/*
 * The same operation for 1 <= M <= 128 (the decode shape: X = A is M x K, the
 * weight W = B is K x N, Y = C is M x N; M is the number of sequences
 * decoded at once).  Bandwidth-bound: the time is one pass over W.  The
 * library picks the kernel by shape:
 *  - large W with few 256-column blocks (for example 4096 x 4096 at any
 *    M up to 8): K is split across workgroups, each reading 1 KB runs of W's
 *    rows over a chunk of K; the chunks' partial sums are added in chunk
 *    order by the last workgroup of each column block, in the same kernel.
 *    The partial sums and arrival counters live in device memory the
 *    library reserves statically (about 16 MB per device, in 8 slots); each
 *    stream gets its own slot on its first call, so calls on different
 *    streams never share one.  Calls on further streams run a form without
 *    scratch that adds the same partial sums in the same order
 *    (bit-identical results).  A call captured in a HIP graph keeps the
 *    capturing stream's slot: two replays of it must not run concurrently
 *    with each other or with calls on that stream.
 *  - otherwise each workgroup streams a narrow block of W's columns over
 *    all of K, its waves split K, and the partial sums are added inside the
 *    workgroup; up to M = 32 the multiply can run on the vector ALUs
 *    (128-bit loads of W), up to M = 128 on the matrix cores (16-column
 *    stripes, v_mfma_f32_16x16x4_f32).
 * Every path adds in a fixed order (integer atomics only, none on floats),
 * so repeated calls give bit-identical results.  Returns -1 when M is
 * outside 1..128.
 */
int sgemv(int M, int N, int K, float alpha, const float *A, int lda,
          const float *B, int ldb, float beta, float *C, int ldc,
          fp32gemm_stream_t stream);

/*
 * Transposed operands.  op(X) = X for FP32GEMM_OP_N and X^T for FP32GEMM_OP_T.
 * C[M x N] <- alpha * op(A)[M x K] . op(B)[K x N] + beta * C, row-major
 * storage: A is M x K (lda >= K) for N, or stored K x M (lda >= M) with
 * op(A)[i][k] = A[k * lda + i] for T; B is K x N (ldb >= N) for N, or stored
 * N x K (ldb >= K) with op(B)[k][j] = B[j * ldb + k] for T.  These are the
 * projection products of a transformer layer ("GPU GEMM 优化完全拆解（一）",
 * section "LLM 推理本质上是 GEMM 的串联": QKV, Q K^T, FFN), where weights and
 * keys are commonly stored transposed.  The 128-bit path needs 16-byte
 * aligned operands whose contiguous dimension and leading dimension are
 * multiples of 4.  M <= 8 runs a GEMV kernel: with op(B) = B the one sgemm
 * uses; with op(B) = B^T (a linear layer's weight stored N x K, y = x W^T) a
 * row-dot kernel that streams each stored row of B contiguously.  Either
 * takes op(A) = A^T as well, up to lda = 2^17 (beyond that the tiled kernel
 * runs).  Both reduce in a fixed order, so results are bit-reproducible.
 * Argument positions for error codes: transA 1,
 * transB 2, M 3, N 4, K 5, alpha 6, A 7, lda 8, B 9, ldb 10, beta 11, C 12,
 * ldc 13, stream 14.
 */
#define FP32GEMM_OP_N 0
#define FP32GEMM_OP_T 1
int sgemm_ex(int transA, int transB, int M, int N, int K, float alpha,
             const float *A, int lda, const float *B, int ldb, float beta,
             float *C, int ldc, fp32gemm_stream_t stream);

/*
 * batch_count independent products of the same shape: entry b uses
 * A + b * strideA, B + b * strideB and C + b * strideC (element strides).
 * strideA or strideB may be 0 (one operand shared by every entry); the C
 * entries must not overlap: strideC >= (M - 1) * ldc + N when
 * batch_count > 1.  Per-head attention products (Q K^T and P V for every
 * head) are this shape; with M <= 8 (decode: one query row per head) the
 * entries run on the GEMV kernels, with one grid over all entries.
 * 0 <= batch_count <= 65535; batch_count == 0 does nothing.  Argument positions: transA 1, transB 2, M 3, N 4, K 5, alpha 6,
 * A 7, lda 8, strideA 9, B 10, ldb 11, strideB 12, beta 13, C 14, ldc 15,
 * strideC 16, batch_count 17, stream 18.
 */
int sgemm_strided_batched(int transA, int transB, int M, int N, int K,
                          float alpha, const float *A, int lda,
                          long long strideA, const float *B, int ldb,
                          long long strideB, float beta, float *C, int ldc,
                          long long strideC, int batch_count,
                          fp32gemm_stream_t stream);

/*
 * Fused epilogue: C[i][j] <- act(alpha * (op(A) op(B))[i][j] + beta * C[i][j]
 * + bias[j]), operands as in sgemm_ex.  This is the operator fusion of "GPU
 * 基础原理" (a translation of "Basic facts about GPUs"), section "4.1 算子融合":
 * the elementwise chain (the page's example is y = relu(x + 1)) runs on the
 * product in registers, so C is stored once instead of being written, read
 * and written again by separate kernels.
 *
 * bias: device pointer to N floats, one per column of C (a linear layer's
 * output features), owned by the caller; NULL = no bias.  act:
 * FP32GEMM_ACT_NONE or FP32GEMM_ACT_RELU (v < 0 becomes 0; NaN and -0.0 pass
 * unchanged).  The bias is added first, then the activation is applied.
 * alpha = 0 or K = 0 still applies the epilogue to beta * C.  Routing as in
 * sgemm_ex (M <= 8 takes a GEMV kernel).  Argument positions for error
 * codes: as sgemm_ex for 1..13, bias 14, act 15 (unknown activation),
 * stream 16.
 */
#define FP32GEMM_ACT_NONE 0
#define FP32GEMM_ACT_RELU 1
int sgemm_fused(int transA, int transB, int M, int N, int K, float alpha,
                const float *A, int lda, const float *B, int ldb, float beta,
                float *C, int ldc, const float *bias, int act,
                fp32gemm_stream_t stream);

/*
 * Split-K: the same product as sgemm_ex, computed as `splits` partial
 * products over consecutive chunks of K that run as one grid, then added in
 * ascending chunk order (so results are bit-reproducible) with alpha and
 * beta applied once.  This is the K split of "CUDA 矩阵乘法优化：从朴素
 * Kernel 到接近 cuBLAS", section "10. cuBLAS 领先的性能差异", for shapes
 * whose C has too few tiles to fill the GPU but whose K is long.
 *
 * splits = 0 lets the library choose (fp32gemm_splitk_splits); otherwise
 * 1 <= splits <= 65535, rounded so that every chunk is a multiple of 32
 * values of K (the call may use fewer chunks than asked).  With one chunk,
 * or M <= 8, the call is exactly sgemm_ex and needs no workspace.
 *
 * workspace: device memory owned by the caller, at least
 * sgemm_splitk_workspace_size(M, N, K, splits) bytes, 16-byte aligned for
 * the fastest path; it holds the partial products (chunks x M x N floats,
 * packed) between the two kernels, must not overlap A, B or C, and must not
 * be used by another call until this one has completed on its stream.  The
 * library allocates nothing.
 *
 * Argument positions for error codes: transA 1, transB 2, M 3, N 4, K 5,
 * alpha 6, A 7, lda 8, B 9, ldb 10, beta 11, C 12, ldc 13, splits 14,
 * workspace 15 (NULL when needed), workspace_bytes 16 (too small),
 * stream 17.
 */
int sgemm_splitk(int transA, int transB, int M, int N, int K, float alpha,
                 const float *A, int lda, const float *B, int ldb, float beta,
                 float *C, int ldc, int splits, float *workspace,
                 size_t workspace_bytes, fp32gemm_stream_t stream);

/*
 * sgemm_splitk for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same computation, kernels and summation order as sgemm_splitk with the
 * same splits (bit-identical results), but the partial products go to a
 * scratch array the library holds in device memory, 16 MiB on each GPU it
 * runs on, kept until the process ends.  No hipMalloc, hipFree or other
 * allocating call is made.
 *
 * Limit: chunks x M x N floats (the chunk count as sgemm_splitk would use
 * it, see sgemm_splitk_workspace_size / 4) must be at most 4 Mi; larger
 * calls return FP32GEMM_ERR_SCRATCH and enqueue nothing.  Calls that need
 * no scratch (one chunk, M <= 8, quick returns) run as sgemm_ex does.
 *
 * All calls on one GPU share its scratch array, which keeps the last call's
 * contents: calls that overlap in time on one GPU (on different streams,
 * or graph replays running concurrently) race and give undefined results.
 * Calls in sequence on one stream are safe.
 *
 * Argument positions for error codes: transA 1, transB 2, M 3, N 4, K 5,
 * alpha 6, A 7, lda 8, B 9, ldb 10, beta 11, C 12, ldc 13, splits 14,
 * stream 15.
 */
int sgemm_splitk_noalloc(int transA, int transB, int M, int N, int K,
                         float alpha, const float *A, int lda, const float *B,
                         int ldb, float beta, float *C, int ldc, int splits,
                         fp32gemm_stream_t stream);

/*
 * Stream-K: the same product as sgemm_ex, as one persistent grid whose
 * workgroups each take an equal run of the product's (C tile, K slice)
 * units, crossing tile boundaries; a tile shared by several workgroups is
 * finished in the same kernel by the last of them to arrive, which adds the
 * others' partial tiles in K order and applies alpha, beta.  This is the
 * pages' remedy for grids that leave compute units idle ("CUDA 矩阵乘法优化：
 * 从朴素 Kernel 到接近 cuBLAS", section "10. cuBLAS 领先的性能差异": split
 * K where the tiles of C alone do not fill the GPU), without split-K's
 * second kernel and with every workgroup doing the same amount of work.
 * Results are bit-reproducible (the order of the additions depends only on
 * the shape).
 *
 * workspace: device memory owned by the caller, at least
 * sgemm_streamk_workspace_size(M, N, K) bytes; it holds partial tiles (two
 * per workgroup at most) and must not overlap A, B or C or be used by
 * another call until this one has completed on its stream.  Arrival
 * counters live in device memory the library reserves statically per
 * stream (8 streams per device, up to 4096 C tiles per call; past either
 * limit they go to the end of the workspace, cleared by a small kernel
 * before the main one).  M <= 8 runs the GEMV kernels as sgemm_ex does and
 * needs no workspace.
 *
 * Argument positions for error codes: transA 1, transB 2, M 3, N 4, K 5,
 * alpha 6, A 7, lda 8, B 9, ldb 10, beta 11, C 12, ldc 13, workspace 14
 * (NULL), workspace_bytes 15 (too small), stream 16.
 */
int sgemm_streamk(int transA, int transB, int M, int N, int K, float alpha,
                  const float *A, int lda, const float *B, int ldb, float beta,
                  float *C, int ldc, float *workspace, size_t workspace_bytes,
                  fp32gemm_stream_t stream);

/* Workspace bytes sgemm_streamk needs for this shape (0 when M <= 8). */
size_t sgemm_streamk_workspace_size(int M, int N, int K);

/* Workspace bytes sgemm_splitk needs for this shape and splits (0 = the
 * library's choice); 0 when the call runs as a single chunk. */
size_t sgemm_splitk_workspace_size(int M, int N, int K, int splits);

/* The number of K chunks sgemm_splitk uses with splits = 0: a model of the
 * tiled kernel's rate for the enlarged grid plus the reduction's traffic. */
int fp32gemm_splitk_splits(int M, int N, int K);

/*
 * The 8-bit linear layer: y = x W^T with x and W in 8-bit integer codes, a
 * scale for each token (row of x) and one for each channel (row of W, stored
 * N x K).  s8_quantize and s8_rmsnorm make codes and scales from floats;
 * s8gemm multiplies them exactly in integers and returns floats.  W's codes
 * are a quarter of its fp32 bytes, which is what a decode step's time is.
 * A code c with scale s stands for the value c * s.
 *
 * The float operands (X, R, H, W of the norm, C) are fp32, fp16 or bf16, one
 * type in a call; scales and bias are fp32.  Codes are signed char; those the
 * library makes lie in -127 .. 127, s8gemm takes -128 too.  Any alignment of
 * codes is accepted and any leading dimension up to 2^20; float operands are
 * aligned to their type (an argument error otherwise).
 *
 * Rows of codes that start at multiples of 16 bytes (base address and leading
 * dimension) take 128-bit loads; the up to 15 bytes that follow a row's K
 * codes, inside its leading dimension, may then be read, and their values do
 * not matter.  The path is chosen for both operands together.  Rows from
 * multiples of 128 bytes are whole cache lines (s8gemm of 777 x 1280 x 4096,
 * fp32 out: 13.8 us; with a leading dimension of 4112 16.3, of 4099 22.1).
 *
 * Beyond that the conventions at the top of this file hold: asynchronous, no
 * allocation, no workspace, results that are bit-identical from call to call,
 * argument p invalid = -p and nothing enqueued.  Outputs must not overlap
 * inputs, other than as s8_rmsnorm says.
 */
#define FP32GEMM_TYPE_F32 0
#define FP32GEMM_TYPE_F16 1
#define FP32GEMM_TYPE_BF16 2

/*
 * Codes and scales of the rows of op(X), M x K: X is M x K (ldx >= K) for
 * FP32GEMM_OP_N, or stored K x M (ldx >= M) with op(X)[i][k] = X[k * ldx + i]
 * for FP32GEMM_OP_T (a weight stored K x N gives the N x K codes that s8gemm
 * reads).  Q is M x K (ldq >= K), scales has M values:
 *
 *   scales[i] = max_k |x_ik| / 127, rounded to fp32,
 *   Q[i][k]   = x_ik / scales[i], rounded to the nearest integer, halves to
 *               even, the quotient not rounded before.
 *
 * (In a row so small that its scale is subnormal or underflows to zero, codes
 * past 127 become 127, and with a zero scale all are 0.)  A row that holds an
 * infinity or a NaN gets the scale NaN and codes 0, so that the products of
 * that row, and of no other, are NaN.  A row of zeros has scale 0; K == 0
 * gives scale 0.  Bytes of Q past a row's K codes are left as they were.  Few
 * columns of a long K run as four kernels in a row, with `scales` in use
 * between them.
 * Argument positions for error codes: trans 1, M 2, K 3, type 4, X 5, ldx 6,
 * Q 7, ldq 8, scales 9, stream 10.
 */
int s8_quantize(int trans, int M, int K, int type, const void *X, int ldx,
                signed char *Q, int ldq, float *scales,
                fp32gemm_stream_t stream);

/*
 * The residual stream's addition, the root-mean-square norm, and the codes of
 * its result, row by row:
 *
 *   h_ik      = x_ik + r_ik, rounded to the operands' type (x_ik when R is
 *               NULL); stored in H unless H is NULL,
 *   v_ik      = h_ik * W[k], rounded to fp32,
 *   step_i    = max_k |v_ik| / 127, rounded to fp32,
 *   Q[i][k]   = v_ik / step_i, rounded as in s8_quantize,
 *   scales[i] = step_i / sqrt(sum_k h_ik^2 / K + eps), rounded to fp32,
 *
 * so that Q * scales is rmsnorm(x + r) * W.  The norm divides a row by one
 * number, which moves the scale and no code.  The sum of squares is kept in
 * 64 bits.  H may be X or R itself (the same address and leading dimension)
 * to update the residual stream in place; it must not overlap them otherwise.
 * R's and H's leading dimensions are not looked at when they are NULL.  Rows
 * with an infinity or a NaN among their v_ik (a sum past the type's range or a
 * product past fp32's is one), of zeros, or of no values, as in s8_quantize.
 * Argument positions for error codes: M 1, K 2, type 3, X 4, ldx 5, R 6,
 * ldr 7, H 8, ldh 9, W 10, eps 11 (negative or not finite), Q 12, ldq 13,
 * scales 14, stream 15.
 */
int s8_rmsnorm(int M, int K, int type, const void *X, int ldx, const void *R,
               int ldr, void *H, int ldh, const void *W, float eps,
               signed char *Q, int ldq, float *scales,
               fp32gemm_stream_t stream);

/*
 * C[i][j] <- act(scaleA[i] * scaleB[j] * sum_k A[i][k] B[j][k]
 *                + beta * C[i][j] + bias[j]),
 * A the M x K codes of the tokens (lda >= K), B the N x K codes of the weight
 * (ldb >= K), C M x N of `type`.  The sum is exact; it is rounded to fp32,
 * scaled and added to in fp32, and rounded once to C's type.  Scales may be
 * any fp32 values: scaleA[i] * sum past fp32's range does no harm where
 * scaleA[i] * scaleB[j] * sum is inside it.  bias (N fp32 values) may be NULL;
 * act is FP32GEMM_ACT_NONE or FP32GEMM_ACT_RELU (as in sgemm_fused).  When
 * beta == 0, C is not read.  K <= 131071, which keeps every sum inside 32
 * bits; K == 0 reads neither codes nor scales.  M == 0 or N == 0 does
 * nothing.  Argument positions for error codes: M 1, N 2, K 3,
 * A 4, lda 5, scaleA 6, B 7, ldb 8, scaleB 9, beta 10, type 11, C 12, ldc 13,
 * bias 14, act 15, stream 16.
 */
int s8gemm(int M, int N, int K, const signed char *A, int lda,
           const float *scaleA, const signed char *B, int ldb,
           const float *scaleB, float beta, int type, void *C, int ldc,
           const float *bias, int act, fp32gemm_stream_t stream);

/* Human-readable text for a return code (static storage, never NULL). */
const char *fp32gemm_strerror(int code);

/*
 * Tuning and testing hooks.  These expose the per-shape parameter search of
 * "CUDA 矩阵乘法优化：从朴素 Kernel 到接近 cuBLAS", section "8. Kernel 9:
 * 参数自动调优": the tile parameters (block tile, K depth, wave tile) are
 * enumerated, each candidate is timed on the target GPU, and the fastest per
 * shape goes into a table, because the best choice differs between GPUs.
 * The tuner (fp32_gemm_06_amd/tune.py) drives the sweep of kinds 0 and 1
 * through these calls.
 * kind 0 = the SGEMM kernel family, kind 1 = the GEMV family, kind 2 = the
 * 8-bit product (s8gemm), whose choice is by fitted times and not a table.
 * Configurations are numbered 0 .. fp32gemm_num_configs(kind)-1 and named by
 * fp32gemm_config_name (NULL for an unknown id); an unknown kind gives 0
 * configurations, NULL names and FP32GEMM_ERR_CONFIG selections.
 */
int fp32gemm_num_configs(int kind);
const char *fp32gemm_config_name(int kind, int cfg);

/* The configuration sgemm()/sgemv()/s8gemm() would pick for this shape (kind as above). */
int fp32gemm_select_config(int kind, int M, int N, int K);

/* The largest M a configuration runs (kind as above; -1 for an unknown id):
 * 8, 32, 64 or 128 for the GEMV family, INT_MAX for the tiled family and the
 * 8-bit product. */
int fp32gemm_config_max_rows(int kind, int cfg);

/* Whether the tiled kernel runs this product (batch entries of M x N x K) as
 * two launches: 0 = one launch; 1 = columns [0, *first) of C in whole rounds
 * of 256x256 tiles, then the remaining columns; 2 = the same over rows.
 * *first (may be NULL) receives the split point, 0 for one launch. */
int fp32gemm_round_split(int M, int N, int K, int batch, int *first);

/*
 * sgemm / sgemv with a forced configuration (cfg = -1 picks as the plain
 * entry point does).  Same contract and codes as sgemm; the M <= 8 routing
 * is not applied: fp32gemm_sgemm_with_config always runs the MFMA kernel and
 * fp32gemm_sgemv_with_config always the GEMV family (M must be 1..128, and at
 * most fp32gemm_config_max_rows of the configuration, else
 * FP32GEMM_ERR_CONFIG).
 */
int fp32gemm_sgemm_with_config(int cfg, int M, int N, int K, float alpha,
                               const float *A, int lda, const float *B,
                               int ldb, float beta, float *C, int ldc,
                               fp32gemm_stream_t stream);
int fp32gemm_sgemv_with_config(int cfg, int M, int N, int K, float alpha,
                               const float *A, int lda, const float *B,
                               int ldb, float beta, float *C, int ldc,
                               fp32gemm_stream_t stream);

/* s8gemm with a forced configuration (cfg = -1 picks as s8gemm does); error
 * positions as s8gemm shifted by one (FP32GEMM_ERR_CONFIG for an unknown
 * id). */
int fp32gemm_s8gemm_with_config(int cfg, int M, int N, int K,
                                const signed char *A, int lda,
                                const float *scaleA, const signed char *B,
                                int ldb, const float *scaleB, float beta,
                                int type, void *C, int ldc, const float *bias,
                                int act, fp32gemm_stream_t stream);

/*
 * Stream-K tuning and testing hooks.  Tiles are numbered 0 ..
 * (number of names) - 1 and named by fp32gemm_streamk_tile_name (NULL past
 * the end).  fp32gemm_streamk_plan reports the plan for a shape with a
 * forced tile and / or workgroup count (-1 / 0 = the library's choice): the
 * tile, workgroups and K slices per workgroup, and returns the workspace
 * bytes it needs (0 for invalid arguments).  fp32gemm_streamk_with_config
 * runs sgemm_streamk with that plan, for any M >= 1; error positions as
 * sgemm_streamk shifted by two (tile 1, groups 2; FP32GEMM_ERR_CONFIG for an
 * unknown tile).
 */
const char *fp32gemm_streamk_tile_name(int tile);
size_t fp32gemm_streamk_plan(int M, int N, int K, int tile, int groups,
                             int *tile_out, int *groups_out, int *ipw_out);
int fp32gemm_streamk_with_config(int tile, int groups, int transA, int transB,
                                 int M, int N, int K, float alpha,
                                 const float *A, int lda, const float *B,
                                 int ldb, float beta, float *C, int ldc,
                                 float *workspace, size_t workspace_bytes,
                                 fp32gemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP32GEMM_H */
