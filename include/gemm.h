/*
 * gemm.h -- C ABI of the GB300 (sm_103a) dense GEMM library.
 *
 * The plain products (gemm_f32 and its kin) compute, on the GPU,
 *
 *     D = alpha * op(A) * op(B) + beta * C
 *
 * the general matrix multiplication of "GEMM on NVIDIA GPUs: from naive
 * kernel to tiled pipeline", section 1 "GEMM definition": op(A) is M x K,
 * op(B) is K x N, C and D are M x N, and
 *
 *     D_ij = alpha * sum_{k<K} A_ik * B_kj + beta * C_ij.
 *
 * "op" (identity or transpose) is expressed as the storage order of each
 * operand, which is exactly the BLAS "trans" flag:
 *
 *     GEMM_ROW_MAJOR:  X(r, q) is stored at X[r * ld + q]
 *     GEMM_COL_MAJOR:  X(r, q) is stored at X[r + q * ld]
 *
 * where (r, q) index the LOGICAL matrix: A(i, k), B(k, j), C(i, j), D(i, j).
 * C and D share one order.  Leading dimensions are in elements.
 *
 * Common contract of gemm_f32 and gemm_bf16_f32acc
 * -------------------------------------------------
 * Ownership: A, B, C and D are device pointers owned by the caller (for
 *   example torch CUDA tensors).  The library keeps no pointer after the call
 *   returns; tensor maps travel by value in the launch parameters.
 *   Workspace: a kernel may split the K range of some tiles across CTAs (to
 *   keep every SM busy).  Such a kernel takes a temporary workspace for the
 *   partial sums (a few tens of MiB at most) from a memory pool the library
 *   owns, one per device, allocated and freed in stream order on `stream`.
 *   The pool keeps up to 256 MiB of freed memory for later calls.  Kernels
 *   that split a tile's K range over the CTAs of one thread-block cluster
 *   (small tensor-core and FP32 problems) add the partial sums in the
 *   cluster's shared memory and take neither workspace nor counters.
 *   Split counters: the split pieces count themselves in small counters that
 *   the library keeps per (device, stream) -- streams told apart by their
 *   unique id, so cudaStreamPerThread is a different stream in each host
 *   thread -- and that every kernel returns to zero, so no call clears them.
 *   They take what the largest split call on the stream needed (64 bytes
 *   to a few KiB) and come from the same pool.  A stream's counters that
 *   a larger problem outgrows are freed in stream order.  What a device
 *   holds is reported by gemm_memory_info(); gemm_release_memory() frees it.
 *   Graph capture: while `stream` is being captured, each call takes fresh
 *   counters and workspace as graph memory.  The graph may therefore be
 *   replayed on any stream, beside other calls.
 *   Threads: any number of host threads may call at once, on one stream or
 *   on several.  A call holds its stream's counters from the moment it takes
 *   them until its kernel is enqueued, so calls on one stream are enqueued
 *   one after another.
 * Asynchrony: the work is enqueued on `stream` (0 = the legacy default
 *   stream) and the call returns without waiting for it.  The caller keeps
 *   the buffers alive until the stream has passed the call.
 * Shapes: M, N, K >= 0 and each <= 2^31 - 1, and M * N <= 2^43 (no device
 *   holds a larger D).  M == 0 or N == 0 is a no-op that returns GEMM_OK
 *   without touching any pointer.  K == 0 or alpha == 0 gives
 *   D = beta * C (A and B are not read).
 * beta == 0: C is never read and may be NULL (BLAS convention; C traffic
 *   only counts when beta != 0 in "GEMM on NVIDIA GPUs", section 2, "GEMM
 *   arithmetic intensity").  C == D with the same ldc/ldd is allowed
 *   (in-place update).  Any other overlap of D with A, B or C is undefined.
 * Leading dimensions: lda >= max(1, K) if A is row-major, >= max(1, M) if
 *   column-major; ldb >= max(1, N) row-major / max(1, K) column-major;
 *   ldc, ldd >= max(1, N) row-major / max(1, M) column-major.
 * Alignment: pointers must be aligned to their element size.  Any leading
 *   dimension is accepted; wide loads and TMA are used when pointers and
 *   leading dimensions allow it, narrower guarded accesses otherwise.  This
 *   never changes the result beyond the stated tolerances and is never an
 *   error.
 * Edges: any M, N, K is handled; tiles past the matrix edge read zeros and
 *   never store outside D.
 * Errors: argument errors return synchronously before any launch and leave
 *   D untouched.  A launch failure returns GEMM_ERR_LAUNCH.  A device without
 *   sm_103 support returns GEMM_ERR_UNSUPPORTED_DEVICE (no CPU fallback
 *   exists).  The tensor-core kernel bounds every wait on its pipeline
 *   barriers; if one runs out it records GEMM_ERR_TIMEOUT in a per-device
 *   status word, read by gemm_last_device_status().  Nothing is printed.
 */
#ifndef DENSE_GEMM_08_GB300_GEMM_H
#define DENSE_GEMM_08_GB300_GEMM_H

#include <stdint.h>
#include <cuda_runtime_api.h> /* cudaStream_t */

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GEMM_ROW_MAJOR = 0, GEMM_COL_MAJOR = 1 } gemm_order_t;

typedef enum {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_VALUE = 1,     /* bad shape, leading dimension, order, NULL or misaligned pointer */
    GEMM_ERR_UNSUPPORTED_DEVICE = 2, /* current device is not sm_103 */
    GEMM_ERR_LAUNCH = 3,            /* the CUDA runtime refused the launch */
    GEMM_ERR_TIMEOUT = 4,           /* a bounded device-side wait ran out (see gemm_last_device_status) */
    GEMM_ERR_INTERNAL = 5           /* a CUDA runtime or driver call failed (e.g. tensor-map encoding) */
} gemm_status_t;

/* One BF16 number as its raw 16-bit pattern (the upper half of an FP32). */
typedef uint16_t gemm_bf16_t;

/* One IEEE 754 binary16 (FP16) number as its raw 16-bit pattern. */
typedef uint16_t gemm_f16_t;

/*
 * gemm_f32 -- FP32 inputs, FP32 arithmetic on the CUDA cores (no TF32),
 * FP32 output.  The kernel tiles D into CTA tiles staged through shared
 * memory, each thread accumulates an 8 x 8 register block with FP32 FMA
 * ("Worklog: optimising GEMM on NVIDIA H100", kernels 2-6: shared-memory
 * tiling, register tiling, vectorised loads, warp tiling).
 *
 *   M, N, K        logical sizes of op(A) (M x K), op(B) (K x N), C/D (M x N)
 *   alpha, beta    scalars (FP32)
 *   A, lda, order_a   device pointer to op(A)'s storage, its leading dimension, its order
 *   B, ldb, order_b   same for op(B)
 *   C, ldc         device pointer to C (read only if beta != 0), leading dimension
 *   D, ldd         device pointer to D (written), leading dimension
 *   order_cd       storage order of both C and D
 *   stream         CUDA stream the kernel is enqueued on
 *
 * Accuracy: |D - D_ref| <= 1e-5 * sum_k |alpha A_ik B_kj| + 1e-6 * |beta C_ij|
 * against the exact result; bit-exact when every partial sum is an integer
 * below 2^24 and alpha = 1, beta = 0.
 */
gemm_status_t gemm_f32(int64_t M, int64_t N, int64_t K, float alpha,
                       const float *A, int64_t lda, gemm_order_t order_a,
                       const float *B, int64_t ldb, gemm_order_t order_b,
                       float beta, const float *C, int64_t ldc,
                       float *D, int64_t ldd, gemm_order_t order_cd,
                       cudaStream_t stream);

/*
 * gemm_bf16_f32acc -- BF16 inputs, FP32 accumulation, FP32 C and D.
 *
 * The tensor-core path (tcgen05.mma with the accumulator in tensor memory,
 * "GEMM on NVIDIA GPUs", section 4 "Tensor Core pipeline"; TMA-fed
 * multi-stage shared-memory ring with a producer/consumer split,
 * "Worklog: optimising GEMM on NVIDIA H100", kernels 7-9) runs when A and B
 * are 16-byte aligned and lda, ldb are multiples of 8 elements.  Otherwise a
 * CUDA-core kernel with the same results contract runs.  Arguments as for
 * gemm_f32; A and B point to BF16 bit patterns.
 *
 * Accuracy: |D - D_ref| <= 4e-3 * sum_k |alpha A_ik B_kj| + 1e-6 against the
 * exact result over the same BF16 inputs; bit-exact when every partial sum
 * is an integer below 2^24 and alpha = 1, beta = 0.
 */
gemm_status_t gemm_bf16_f32acc(int64_t M, int64_t N, int64_t K, float alpha,
                               const gemm_bf16_t *A, int64_t lda, gemm_order_t order_a,
                               const gemm_bf16_t *B, int64_t ldb, gemm_order_t order_b,
                               float beta, const float *C, int64_t ldc,
                               float *D, int64_t ldd, gemm_order_t order_cd,
                               cudaStream_t stream);

/*
 * gemm_f16_f32acc -- FP16 inputs, FP32 accumulation, FP32 C and D.
 *
 * The FP16-input, FP32-accumulate GEMM measured in "High-Performance FP16
 * General Matrix Multiplication on NVIDIA Ada Lovelace via CUTLASS and
 * WMMA" (methodology and results: FP16 -> FP32 at M = N = K = 8192), on the
 * same tcgen05 kernels as gemm_bf16_f32acc (kind::f16 with the FP16 operand
 * format) and the same CUDA-core fallback.  Arguments, contract and
 * accuracy bound as for gemm_bf16_f32acc; A and B point to binary16 bit
 * patterns.
 */
gemm_status_t gemm_f16_f32acc(int64_t M, int64_t N, int64_t K, float alpha,
                              const gemm_f16_t *A, int64_t lda, gemm_order_t order_a,
                              const gemm_f16_t *B, int64_t ldb, gemm_order_t order_b,
                              float beta, const float *C, int64_t ldc,
                              float *D, int64_t ldd, gemm_order_t order_cd,
                              cudaStream_t stream);

/*
 * gemm_f32_noalloc -- gemm_f32 for callers that cannot allocate device
 * memory.  The GEMM pages have no counterpart to this entry point.  It is
 * for code that must not call the CUDA allocator: code running under a
 * device-memory budget fixed in advance, code inside an allocator's own
 * callbacks, or code on a path where an allocation could block or fail.
 *
 * Arguments, results and accuracy are those of gemm_f32, and it picks the
 * same kernel with the same work split (the small-M kernel for M <= 8, the
 * cluster kernel for small problems, the CUDA-core kernel's tile
 * configurations otherwise).  The only difference: when that kernel splits
 * the K range of some tiles, the split pieces' counters and partial sums go
 * to a fixed 32 MiB array compiled into the library (a file-scope __device__
 * array that every device holding the library keeps until the process
 * exits) instead of pool memory and the stream's counters.  So the call
 * allocates nothing: no cudaMalloc, no cudaFree, no pool.
 *
 * Limits and rules:
 *   - The first 16 KiB of the array hold the counters, the rest (32 MiB -
 *     16 KiB) the partial sums.  A problem whose split needs more is refused
 *     with GEMM_ERR_INVALID_VALUE before anything is enqueued (gemm_f32
 *     handles it).  Problems that split no tile need no scratch.
 *   - The first call on each device sets up the array: it looks up that
 *     device's address of it (cudaGetSymbolAddress), zeroes the counters on
 *     `stream` and waits for that.  Make that first call before any stream
 *     capture on that device (under capture it returns GEMM_ERR_INTERNAL).
 *   - Every kernel leaves the counters it used at zero, so later calls clear
 *     nothing.  All calls on a device share the one array, and it keeps what
 *     the last call left in it.  Calls whose work overlaps on the GPU
 *     (different streams, no ordering between them) race on the array and
 *     give wrong results: order them on one stream or with events.
 */
gemm_status_t gemm_f32_noalloc(int64_t M, int64_t N, int64_t K, float alpha,
                               const float *A, int64_t lda, gemm_order_t order_a,
                               const float *B, int64_t ldb, gemm_order_t order_b,
                               float beta, const float *C, int64_t ldc,
                               float *D, int64_t ldd, gemm_order_t order_cd,
                               cudaStream_t stream);

/*
 * gemm_bf16_f32acc_ex -- gemm_bf16_f32acc with a fused epilogue:
 *
 *     D = act(alpha * op(A) * op(B) + beta * C + bias)
 *
 * stored as FP32 or as BF16 (round to nearest even), all in the same kernel
 * ("GEMM on NVIDIA GPUs", section 4 "Epilogue": alpha, beta, bias,
 * activation and dtype conversion in the epilogue, no extra round trip;
 * BF16 output as in "Worklog: optimising GEMM on NVIDIA H100", kernels 7-9).
 *
 *   epilogue->bias        N FP32 values, bias[j] added to column j of D, or
 *                         NULL for none (device pointer, 4-byte aligned)
 *   epilogue->activation  GEMM_ACT_NONE, GEMM_ACT_RELU (max(x, 0)) or
 *                         GEMM_ACT_GELU (tanh form:
 *                         0.5 x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))))
 *   epilogue->d_type      GEMM_D_F32 (D is float) or GEMM_D_BF16 (D holds
 *                         gemm_bf16_t; its pointer must be 2-byte aligned)
 *
 * epilogue == NULL means no bias, no activation, FP32 D (= gemm_bf16_f32acc).
 * C stays FP32; with a BF16 D, C and D must not overlap.  Everything else
 * as for gemm_bf16_f32acc.  Accuracy: the bound of gemm_bf16_f32acc on the
 * pre-activation value, times 1.13 for GELU (its largest slope) plus
 * 1e-6 |x|, plus 2^-8 |D| for BF16 rounding (half an ulp at 8 significant
 * bits).
 */
typedef enum {
    GEMM_ACT_NONE = 0,
    GEMM_ACT_RELU = 1,
    GEMM_ACT_GELU = 2,
    GEMM_ACT_SILU = 3 /* gemm_fused_* only */
} gemm_activation_t;
typedef enum {
    GEMM_D_F32 = 0,
    GEMM_D_BF16 = 1,
    GEMM_D_F16 = 2 /* not of the dense products above */
} gemm_d_type_t;
typedef struct {
    const float *bias;
    gemm_activation_t activation;
    gemm_d_type_t d_type;
} gemm_epilogue_t;

gemm_status_t gemm_bf16_f32acc_ex(int64_t M, int64_t N, int64_t K, float alpha,
                                  const gemm_bf16_t *A, int64_t lda, gemm_order_t order_a,
                                  const gemm_bf16_t *B, int64_t ldb, gemm_order_t order_b,
                                  float beta, const float *C, int64_t ldc,
                                  void *D, int64_t ldd, gemm_order_t order_cd,
                                  const gemm_epilogue_t *epilogue, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Grouped operators: products whose weight matrix depends on the row (the
 * experts of a mixture, the low-rank adapters of many requests).  The GEMM
 * pages have no counterpart to them.
 *
 * Common contract.  Ownership, workspace, graph capture, threads,
 * asynchrony and errors are those of gemm_f32 above; in addition:
 * Rows of a group: product row r belongs to the group g with
 *   offsets[g] <= r < offsets[g + 1].  `offsets` holds groups + 1
 *   non-decreasing int32 values on the device (what gemm_group_rows writes);
 *   the host does not read it, so a call never waits for the sizes and can be
 *   captured in a graph.  The kernels clamp each value to [0, rows] and take
 *   a falling pair as an empty group: other values than the above give
 *   unspecified results, but no access outside the operands.  Rows past
 *   offsets[groups] (and before offsets[0]) belong to no group: no value
 *   computed from them is stored.
 * row_index (or NULL): product row r reads row row_index[r] of A, so rows
 *   need not be copied into group order first; an index outside [0, rows_a)
 *   reads a row of zeros (rows_a == 0: A may be NULL).  Without it row r of A is
 *   read and rows_a >= rows.
 * Matrices: A and D are row-major (a group is a run of rows).  Matrix g of a
 *   stack starts stride elements after matrix g - 1 (stride_b = 0: one B for
 *   all groups).  Every matrix and group stride is in elements.
 * Types: FP32 accumulation.  d_type is GEMM_D_F32, or the inputs' 16-bit
 *   type (GEMM_D_BF16, GEMM_D_F16): rounded once, to nearest even, after the
 *   whole epilogue.
 * Kernels: tensor cores (tcgen05) for 16-bit inputs that TMA can describe
 *   (16-byte aligned pointers, leading dimensions and strides multiples of 8
 *   elements), CUDA cores otherwise, for FP32 (no TF32) and for adapters of
 *   rank above 256.  D may have any alignment.
 * Sums: FP32 throughout.  The tensor cores cut what an addition cannot hold
 *   instead of rounding it, by about 1e-9 of a sum per step of K; an FP32 D is
 *   therefore summed 768 steps at a time and the parts added with rounding
 *   (relative error 7e-7 with BF16 inputs, 9e-7 with FP16, at any K or number
 *   of rows of a group; measured on normally distributed values).
 * Workspace, from the library's pool as above: gathered rows are copied into
 *   group order where that is faster (16-bit inputs: rows x K values, or
 *   rows x M for the weight gradient); gemm_lora keeps X LA of up to 128 MiB at
 *   a time, its partial sums and a few words per row; gemm_group_rows up to
 *   128 x groups counts.
 * Special values: a row's infinities and NaNs reach that row's results only
 *   (for the weight gradient: that group's); the activations pass NaNs on.
 * Sizes: each of rows, M, N, K, groups is at most 2^31 - 1 (gemm_grouped_*:
 *   2^24 groups, which each CTA walks to find its rows); no rows or no
 *   columns is a no-op (the weight gradient's groups without rows still give
 *   beta * C).  K == 0 or alpha == 0: A and B are not read.
 */

/*
 * gemm_group_rows -- rows grouped by a number: a stable counting sort, one
 * kernel up to 2048 rows and two beyond.
 *
 *   group_of_row  rows int32 numbers (device); numbers outside [0, groups)
 *                 drop their row
 *   offsets       groups + 1 int32: rows whose number is below g (dropped
 *                 rows do not count); offsets[groups] = rows kept
 *   order         rows int32: the row at each place, by number and then by
 *                 row (stable); -1 past offsets[groups].  As row_index (or
 *                 divided by the number of experts per token) it gathers the
 *                 rows of A for the grouped products.
 *   position      rows int32 or NULL: the place of each row, -1 if dropped
 * groups >= 1; rows == 0 writes zeros to offsets.
 */
gemm_status_t gemm_group_rows(int64_t rows, int64_t groups, const int32_t *group_of_row,
                              int32_t *offsets, int32_t *order, int32_t *position,
                              cudaStream_t stream);

/*
 * gemm_grouped_* -- one product per group of rows:
 *
 *     D(r, :) = act(alpha * A(idx(r), :) * op(B_g) + bias_g),  r in group g
 *
 * op(B_g) is K x N, stored in order_b.  epilogue->bias points to groups x N
 * FP32 values (row g for group g) or is NULL; epilogue may be NULL (no bias,
 * no activation, FP32 D).  The input gradient of a grouped product is the
 * same call with the other order_b (K and N exchanged).
 * Accuracy: |D - D_ref| <= rel * sum_k |alpha A B| + 1e-6 before the
 * activation, rel = 1e-5 (FP32) or 4e-3 (16-bit inputs), plus D's rounding.
 */
gemm_status_t gemm_grouped_f32(int64_t groups, int64_t rows, int64_t N, int64_t K, float alpha,
                               const float *A, int64_t lda, int64_t rows_a,
                               const int32_t *row_index, const int32_t *offsets, const float *B,
                               int64_t ldb, int64_t stride_b, gemm_order_t order_b, void *D,
                               int64_t ldd, const gemm_epilogue_t *epilogue, cudaStream_t stream);
gemm_status_t gemm_grouped_bf16_f32acc(int64_t groups, int64_t rows, int64_t N, int64_t K,
                                       float alpha, const gemm_bf16_t *A, int64_t lda,
                                       int64_t rows_a, const int32_t *row_index,
                                       const int32_t *offsets, const gemm_bf16_t *B, int64_t ldb,
                                       int64_t stride_b, gemm_order_t order_b, void *D,
                                       int64_t ldd, const gemm_epilogue_t *epilogue,
                                       cudaStream_t stream);
gemm_status_t gemm_grouped_f16_f32acc(int64_t groups, int64_t rows, int64_t N, int64_t K,
                                      float alpha, const gemm_f16_t *A, int64_t lda,
                                      int64_t rows_a, const int32_t *row_index,
                                      const int32_t *offsets, const gemm_f16_t *B, int64_t ldb,
                                      int64_t stride_b, gemm_order_t order_b, void *D,
                                      int64_t ldd, const gemm_epilogue_t *epilogue,
                                      cudaStream_t stream);

/*
 * gemm_grouped_wgrad_* -- the weight gradients of the grouped products:
 *
 *     D_g = alpha * sum over the rows r of group g of A(idx(r), :)^T B(r, :)
 *           + beta * C_g
 *
 * A has M columns (the product's inputs), B has N columns (the gradient of
 * its outputs, row-major, one row per product row), D_g and C_g are M x N
 * row-major with group strides stride_d and stride_c.  C is FP32 and not read
 * when beta == 0; C == D with equal strides is allowed when D is FP32
 * (accumulation in place); the matrices of D must not overlap.
 * Accuracy as gemm_grouped_*, plus 1e-6 |beta C|.
 */
gemm_status_t gemm_grouped_wgrad_f32(int64_t groups, int64_t rows, int64_t M, int64_t N,
                                     float alpha, const float *A, int64_t lda, int64_t rows_a,
                                     const int32_t *row_index, const int32_t *offsets,
                                     const float *B, int64_t ldb, float beta, const float *C,
                                     int64_t ldc, int64_t stride_c, void *D, int64_t ldd,
                                     int64_t stride_d, gemm_d_type_t d_type, cudaStream_t stream);
gemm_status_t gemm_grouped_wgrad_bf16_f32acc(int64_t groups, int64_t rows, int64_t M, int64_t N,
                                             float alpha, const gemm_bf16_t *A, int64_t lda,
                                             int64_t rows_a, const int32_t *row_index,
                                             const int32_t *offsets, const gemm_bf16_t *B,
                                             int64_t ldb, float beta, const float *C, int64_t ldc,
                                             int64_t stride_c, void *D, int64_t ldd,
                                             int64_t stride_d, gemm_d_type_t d_type,
                                             cudaStream_t stream);
gemm_status_t gemm_grouped_wgrad_f16_f32acc(int64_t groups, int64_t rows, int64_t M, int64_t N,
                                            float alpha, const gemm_f16_t *A, int64_t lda,
                                            int64_t rows_a, const int32_t *row_index,
                                            const int32_t *offsets, const gemm_f16_t *B,
                                            int64_t ldb, float beta, const float *C, int64_t ldc,
                                            int64_t stride_c, void *D, int64_t ldd,
                                            int64_t stride_d, gemm_d_type_t d_type,
                                            cudaStream_t stream);

/*
 * gemm_lora_* -- a shared projection with each row's own low-rank adapter:
 *
 *     D(i, :) = act(X(i, :) op(W) + scale[a] (X(i, :) op(LA_a)) op(LB_a) + bias),
 *     a = adapter_of_row[i]
 *
 * X is M x K row-major, op(W) K x N; every op(LA_a) is K x rank and op(LB_a)
 * rank x N, in stacks of `adapters` matrices.  A row whose number lies outside
 * [0, adapters) has no adapter.  Rows come in any order: nothing is sorted
 * and the host does not read the numbers.  scale is `adapters` FP32 values or
 * NULL (all 1); epilogue as for gemm_grouped_* with one bias of N values.
 * The input gradient is the same call with W, LA and LB exchanged:
 * dX = dD op(W)^T + scale (dD LB^T) LA^T.  The adapters' own gradients come from
 * rows grouped by adapter (gemm_group_rows): U = X LA and T = dD LB^T are
 * gemm_grouped_*, dLB = scale U^T dD and dLA = scale X^T T gemm_grouped_wgrad_*.
 * An adapter's values reach the rows that use it only (also infinities and
 * NaNs).  Rounding: the first product scale * X LA is summed in FP32 and
 * enters the second one rounded to the inputs' type when D has that type, and
 * as the sum of two such values (about 16 bits for BF16, 22 for FP16) when D
 * is FP32.  Rows where it passes FP16's range are computed by their definition
 * in FP32 instead, far more slowly; where it is small, FP16 holds it in steps
 * of 2^-24, so a first product below 2^-25 (a tiny scale, X or LA) counts as 0.
 * Accuracy: the bound of gemm_grouped_* on X W, plus 2^-8 (2^-15 with an FP32
 * D) of sum |scale (X LA)| |LB|; with FP16 inputs also 2^-25 sum |LB|.
 */
gemm_status_t gemm_lora_bf16_f32acc(int64_t M, int64_t N, int64_t K, const gemm_bf16_t *X,
                                    int64_t ldx, const gemm_bf16_t *W, int64_t ldw,
                                    gemm_order_t order_w, int64_t adapters, int64_t rank,
                                    const int32_t *adapter_of_row, const float *scale,
                                    const gemm_bf16_t *LA, int64_t ld_a, int64_t stride_a,
                                    gemm_order_t order_a, const gemm_bf16_t *LB, int64_t ld_b,
                                    int64_t stride_b, gemm_order_t order_b, void *D, int64_t ldd,
                                    const gemm_epilogue_t *epilogue, cudaStream_t stream);
gemm_status_t gemm_lora_f16_f32acc(int64_t M, int64_t N, int64_t K, const gemm_f16_t *X,
                                   int64_t ldx, const gemm_f16_t *W, int64_t ldw,
                                   gemm_order_t order_w, int64_t adapters, int64_t rank,
                                   const int32_t *adapter_of_row, const float *scale,
                                   const gemm_f16_t *LA, int64_t ld_a, int64_t stride_a,
                                   gemm_order_t order_a, const gemm_f16_t *LB, int64_t ld_b,
                                   int64_t stride_b, gemm_order_t order_b, void *D, int64_t ldd,
                                   const gemm_epilogue_t *epilogue, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * A mixture's router and the way back from its experts, and dense products
 * with the element-wise work around them, each with its gradient.  The GEMM
 * pages have no counterpart to them.
 *
 * Common contract.  Ownership, graph capture, threads, asynchrony and errors
 * are those of gemm_f32 above.  All results are deterministic: no sum's order
 * depends on timing.  A `type` says what a matrix holds (gemm_d_type_t):
 * GEMM_D_F32, GEMM_D_BF16 or GEMM_D_F16.  Matrices are row-major unless an
 * order is given; leading dimensions are in elements; any alignment to the
 * element size is accepted (16-byte aligned rows are faster).  Arithmetic is
 * FP32; a result of 16 bits is rounded once, to nearest even.
 */

/*
 * gemm_route -- the experts of each token and their weights:
 *
 *     s(t, e) = softmax over e or logistic function of logits(t, e)
 *     c(t, e) = s(t, e) + bias[e]
 *     chosen(t, 0 .. k-1) = the experts of the k largest c, by falling c
 *     weights(t, j) = scale * s(t, chosen(t, j)) / S,
 *     S = renormalize ? sum of s over the token's chosen experts : 1
 *
 * The bias (for balance) counts in the choice only.  With groups > 1 the
 * experts form `groups` runs of experts / groups; a group's score is the sum
 * of its group_top (1 or 2) largest c, and the choice is among the
 * groups_kept groups of the largest scores.
 * Order: values are compared as computed in 64 bits (without a bias c has the
 *   order of the logits, and they are compared), equal ones by the lower
 *   index.  A NaN counts as larger than everything.
 * Masks: an expert whose logit or bias is -infinity is never chosen and adds
 *   nothing to its group's score.  Where fewer than k experts can be chosen,
 *   the places left have chosen = -1 and weights = 0 (gemm_group_rows drops
 *   them, gemm_combine skips them).  Finite logits, however low, are no mask.
 * NaNs and +infinities of the logits reach the token's weights as the
 *   formulas say; chosen holds valid numbers in any case.
 *
 *   tokens, experts, k   experts 1 .. 1024, k 1 .. min(experts, 32); more
 *                        than that is refused
 *   logits, ld, type     tokens x experts
 *   rule                 NULL: softmax, no bias, no groups, renormalised, scale 1
 *   chosen               tokens x k int32, contiguous (device)
 *   weights              tokens x k FP32, contiguous (device)
 * With the numbers in row order, chosen is what gemm_group_rows takes (rows =
 * tokens * k, row t * k + j belonging to token t).
 * groups: 1 .. 32, a divisor of experts; groups_kept 1 .. groups.
 */
typedef enum { GEMM_SCORE_SOFTMAX = 0, GEMM_SCORE_SIGMOID = 1 } gemm_score_t;
typedef struct {
    gemm_score_t score;
    int32_t renormalize; /* 0 or 1 */
    float scale;
    const float *bias;   /* experts FP32 values (device) or NULL */
    int32_t groups;      /* 1: no groups (the next two are then not read) */
    int32_t groups_kept;
    int32_t group_top;   /* 1 or 2 */
} gemm_route_rule_t;
gemm_status_t gemm_route(int64_t tokens, int64_t experts, int64_t k, const void *logits,
                         int64_t ld, gemm_d_type_t type, const gemm_route_rule_t *rule,
                         int32_t *chosen, float *weights, cudaStream_t stream);

/*
 * gemm_route_grad -- the gradient of gemm_route's weights with respect to the
 * logits, for a fixed choice:
 *
 *     dlogits(t, e) = sum_j dweights(t, j) * d weights(t, j) / d logits(t, e)
 *
 * rule as in the forward call; its bias and groups are not read.  chosen is
 * the forward call's: a number outside [0, experts) has no weight, and its
 * dweights is not read as one; a number twice counts twice.  dlogits has the
 * logits' type (pitch ld_d) and may be logits itself.  Every element of it is
 * written (0 where the weights do not depend on the logit).  With sigmoid
 * scores or renormalised weights only the chosen experts' logits are read.
 */
gemm_status_t gemm_route_grad(int64_t tokens, int64_t experts, int64_t k, const void *logits,
                              int64_t ld, gemm_d_type_t type, const gemm_route_rule_t *rule,
                              const int32_t *chosen, const float *dweights, void *dlogits,
                              int64_t ld_d, cudaStream_t stream);

/*
 * gemm_combine -- the experts' rows back to the tokens:
 *
 *     D(t, :) = residual(t, :) + sum_{j < k} weights(t, j) * Y(position(t, j), :)
 *
 *   Y, ldy, rows_y, y_type   rows_y x N
 *   position    tokens x k int32, contiguous (gemm_group_rows's position);
 *               a number outside [0, rows_y) adds nothing, whatever its weight
 *   weights     tokens x k FP32, contiguous, or NULL (all 1: the gradient of a
 *               gather of rows, such as the experts' inputs)
 *   residual, ld_r           tokens x N of D's type, or NULL
 *   D, ldd, d_type           tokens x N; GEMM_D_F32 or Y's type.  D may be the
 *               residual (ldd = ld_r), and must not overlap Y.
 * The sum is FP32, in the order of j, the residual last.  tokens, k, N, rows_y
 * >= 0 and at most 2^31 - 1, tokens * k at most 2^40; k = 0 gives the residual
 * or zeros.
 */
gemm_status_t gemm_combine(int64_t tokens, int64_t k, int64_t N, const void *Y, int64_t ldy,
                           int64_t rows_y, gemm_d_type_t y_type, const int32_t *position,
                           const float *weights, const void *residual, int64_t ld_r, void *D,
                           int64_t ldd, gemm_d_type_t d_type, cudaStream_t stream);

/*
 * gemm_combine_grad -- its gradients (the residual's is dD itself):
 *
 *     dY(position(t, j), :) = weights(t, j) * dD(t, :)
 *     dweights(t, j) = <dD(t, :), Y(position(t, j), :)>
 *
 * dD is tokens x N of d_type (GEMM_D_F32 or y_type), dY rows_y x N of y_type.
 * The positions inside [0, rows_y) must differ from one another, as
 * gemm_group_rows's do (of a row named twice, each element of dY is one of the two's);
 * entries outside have dweights = 0.  Rows of dY that no position names are
 * left as they are.  weights NULL: all 1.  dY or dweights may be NULL (not
 * computed); Y is read for dweights only, and NULL without it.  dY must not
 * overlap Y or dD, nor dweights the weights.  k is at least 1.
 */
gemm_status_t gemm_combine_grad(int64_t tokens, int64_t k, int64_t N, const void *dD, int64_t ld_d,
                                gemm_d_type_t d_type, const void *Y, int64_t ldy, int64_t rows_y,
                                gemm_d_type_t y_type, const int32_t *position,
                                const float *weights, void *dY, int64_t ld_dy, float *dweights,
                                cudaStream_t stream);

/*
 * gemm_fused_* -- a product with the element-wise work that follows it:
 *
 *     Z = alpha * op(A) * op(B) + bias
 *     D = act(Z) + residual
 *
 * D, residual and pre are M x N row-major matrices of the inputs' type.
 *   fusion->bias        N FP32 values, one per column (device), or NULL
 *   fusion->activation  GEMM_ACT_NONE, _RELU, _GELU (tanh form) or _SILU
 *                       (x / (1 + exp(-x))); NaNs pass through
 *   fusion->residual, ld_residual   added after the activation, or NULL; may
 *                       be D (the same pitch)
 *   fusion->pre, ld_pre where Z is kept for the backward pass, or NULL; must
 *                       not overlap D, A, B or the residual
 * fusion == NULL: none of them (D = alpha op(A) op(B) in the inputs' type).
 * D is computed from Z before Z is rounded.  M, N, K as for gemm_f32; K == 0
 * or alpha == 0: A and B are not read, Z = bias.  D must not overlap A or B.
 * (Where two matrices of a call must not overlap, or only with the same pitch,
 * the same address is refused; parts of one another are not looked for.)
 * Kernels: tensor cores (tcgen05) for 16-bit inputs that TMA can describe
 *   (16-byte aligned A and B, leading dimensions multiples of 8 elements),
 *   CUDA cores otherwise and for FP32 (no TF32; a larger FP32 product by
 *   gemm_f32's kernels and a pass for what follows it, which where D is the
 *   residual or pre takes workspace of D's size).  D, pre, residual: any alignment.
 * Accuracy: |Z - Z_ref| <= rel * sum_k |alpha A B| + 1e-6 |Z|, rel = 1e-5
 *   (FP32) or 4e-3 (16-bit inputs); D as act's largest slope (1.13 for GELU,
 *   1.1 for SILU) times that plus 1e-6 |Z|; each plus its rounding.
 */
typedef struct {
    const float *bias;
    gemm_activation_t activation;
    const void *residual;
    int64_t ld_residual;
    void *pre;
    int64_t ld_pre;
} gemm_fusion_t;
gemm_status_t gemm_fused_f32(int64_t M, int64_t N, int64_t K, float alpha, const float *A,
                             int64_t lda, gemm_order_t order_a, const float *B, int64_t ldb,
                             gemm_order_t order_b, float *D, int64_t ldd,
                             const gemm_fusion_t *fusion, cudaStream_t stream);
gemm_status_t gemm_fused_bf16_f32acc(int64_t M, int64_t N, int64_t K, float alpha,
                                     const gemm_bf16_t *A, int64_t lda, gemm_order_t order_a,
                                     const gemm_bf16_t *B, int64_t ldb, gemm_order_t order_b,
                                     gemm_bf16_t *D, int64_t ldd, const gemm_fusion_t *fusion,
                                     cudaStream_t stream);
gemm_status_t gemm_fused_f16_f32acc(int64_t M, int64_t N, int64_t K, float alpha,
                                    const gemm_f16_t *A, int64_t lda, gemm_order_t order_a,
                                    const gemm_f16_t *B, int64_t ldb, gemm_order_t order_b,
                                    gemm_f16_t *D, int64_t ldd, const gemm_fusion_t *fusion,
                                    cudaStream_t stream);

/*
 * gemm_fused_grad_* -- the backward product through an activation:
 *
 *     D = (alpha * op(A) * op(B)) * act'(pre)      (element by element)
 *     dbias[n] = sum over the rows m of D(m, n)    (FP32, before D is rounded)
 *
 * With Y = act(X W + b) V and the pre = X W + b that gemm_fused kept, A = dY and
 * B = V^T (the other order of V) give D = the gradient of X W + b and dbias
 * that of b; gemm_fused with A = D, B = W^T and a residual is then the input
 * gradient of a residual block, and the weight gradients are plain products.
 * pre is M x N of the inputs' type and may be D (the same pitch); it is not
 * read when the activation is GEMM_ACT_NONE (NULL allowed).  act' of ReLU is 0
 * at 0; a NaN in pre gives NaN.  dbias may be NULL; it must not overlap
 * another matrix of the call.  M == 0 with N > 0: dbias = 0.
 * Kernels and D's accuracy are gemm_fused_*'s (the largest slope's factor is
 * the slope's own).  The tensor cores cut an accumulator's last place where
 * others round it, which only dbias shows: half a unit on the mean, 2^-25 to 2^-24 of
 * the sum so far for every 16 steps of K (FP16, whose products are longer than that
 * place, loses about four times as much).  Where dbias is wanted K is summed in
 * parts of 768 for that reason, so that D's last bit may differ from a call without
 * it.  At any K a part's sum is then smaller by at most 1.5e-6 of itself on the mean
 * (BF16); measured for dbias as a whole: 0.7e-6 (BF16) and 0.95e-6 (FP16) with operands of
 * random signs, 1.0e-6 and 3.9e-6 where all products have one sign.
 */
gemm_status_t gemm_fused_grad_f32(int64_t M, int64_t N, int64_t K, float alpha, const float *A,
                                  int64_t lda, gemm_order_t order_a, const float *B, int64_t ldb,
                                  gemm_order_t order_b, gemm_activation_t activation,
                                  const float *pre, int64_t ld_pre, float *D, int64_t ldd,
                                  float *dbias, cudaStream_t stream);
gemm_status_t gemm_fused_grad_bf16_f32acc(int64_t M, int64_t N, int64_t K, float alpha,
                                          const gemm_bf16_t *A, int64_t lda, gemm_order_t order_a,
                                          const gemm_bf16_t *B, int64_t ldb, gemm_order_t order_b,
                                          gemm_activation_t activation, const gemm_bf16_t *pre,
                                          int64_t ld_pre, gemm_bf16_t *D, int64_t ldd,
                                          float *dbias, cudaStream_t stream);
gemm_status_t gemm_fused_grad_f16_f32acc(int64_t M, int64_t N, int64_t K, float alpha,
                                         const gemm_f16_t *A, int64_t lda, gemm_order_t order_a,
                                         const gemm_f16_t *B, int64_t ldb, gemm_order_t order_b,
                                         gemm_activation_t activation, const gemm_f16_t *pre,
                                         int64_t ld_pre, gemm_f16_t *D, int64_t ldd,
                                         float *dbias, cudaStream_t stream);

/* Static English description of a status code; never NULL. */
const char *gemm_status_string(gemm_status_t status);

/*
 * gemm_last_device_status -- synchronises `stream`, then reads and clears
 * the current device's status word.  Returns GEMM_OK, or GEMM_ERR_TIMEOUT if
 * a tensor-core launch (or one of gemm_combine's and gemm_combine_grad's that
 * copy rows in bulk) on this device gave up a bounded wait since the last
 * read (its results are then incomplete), or GEMM_ERR_INTERNAL if the read itself
 * failed.  After a timeout it also synchronises the device and frees every
 * stream's split counters (the counts of finished K pieces that each stream
 * keeps between calls, and that a kernel which gave up may have left
 * mid-count); the next split call on a stream starts from zeroed ones.  Read
 * it after a timeout before the next call on this device.
 */
gemm_status_t gemm_last_device_status(cudaStream_t stream);

/*
 * What the library holds on the current device between calls (the split
 * counters of each stream and the workspace pool; see "Split counters" and
 * "Workspace" above).  Nothing in the pages corresponds to this: it is the
 * accounting of this library's own memory.
 *   split_streams        streams of this device that hold split counters
 *   split_bytes          bytes of those counters
 *   pool_used_bytes      pool memory in use: the split counters, plus the
 *                        workspace of calls the GPU has not finished yet
 *   pool_reserved_bytes  pool memory held from the driver (in use or kept
 *                        for reuse, at most 256 MiB beyond what is in use)
 * Returns GEMM_ERR_INVALID_VALUE for a NULL info, GEMM_ERR_INTERNAL if a
 * CUDA query failed.
 */
typedef struct {
    uint64_t split_streams;
    uint64_t split_bytes;
    uint64_t pool_used_bytes;
    uint64_t pool_reserved_bytes;
} gemm_memory_info_t;
gemm_status_t gemm_memory_info(gemm_memory_info_t *info);

/*
 * gemm_release_memory -- synchronises the current device, frees the split
 * counters of every stream on it and returns the pool's free memory to the
 * driver.  Later calls take what they need again.  Call it when no other
 * host thread is calling the library on this device.
 */
gemm_status_t gemm_release_memory(void);

/*
 * gemm_last_kernel -- name of the kernel the calling host thread's most
 * recent successful gemm_* call enqueued ("" if it enqueued none, e.g. for
 * M == 0).  Static string; for tests and launch accounting.
 */
const char *gemm_last_kernel(void);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_08_GB300_GEMM_H */
