// fused.h -- the fused products' problem, as the host dispatcher hands it to
// the kernel launchers (all argument checks done).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "grouped.h"  // kOutF32, kOutBf16, kOutF16
#include "internal.h"

namespace gemm {

enum : int { kActSilu = 3 };  // beside kActNone, kActRelu, kActGelu

// Forward:  Z = alpha op(A) op(B) + bias, D = act(Z) + residual, Z kept in `pre`.
// Gradient: D = alpha op(A) op(B) * act'(pre), dbias = D's column sums before rounding.
// D, residual and pre are row-major and of the inputs' type.
struct FusedProblem {
    int64_t M, N, K;  // K = 0: A and B are not read
    float alpha;
    const void *A;
    int64_t lda;
    bool a_kmajor;  // A(i, k) at A[i * lda + k]; else A[i + k * lda]
    const void *B;
    int64_t ldb;
    bool b_kmajor;  // B(k, j) at B[k + j * ldb]; else B[k * ldb + j]
    void *D;
    int64_t ldd;
    const float *bias;     // forward, or null
    int act;
    const void *residual;  // forward, or null
    int64_t ld_r;
    void *pre;             // forward: written, or null; gradient: read (null: no activation)
    int64_t ld_pre;
    bool grad;
    float *dbias;          // gradient, or null
};

// CUDA-core kernels: any type, order and alignment (fused_simt.cu).
// Few rows of A, and operands whose K is contiguous in 16-byte pieces: launch_fused_simt
// then streams B once, and is the faster one for 16-bit inputs too.
bool fused_rows_eligible(const FusedProblem &p, InType in);
cudaError_t launch_fused_simt(const FusedProblem &p, InType in, cudaStream_t stream,
                              const char **name);
// Tensor-core kernels (fused_tc.cu): BF16 or FP16 operands that TMA can describe.
bool fused_tc_eligible(const FusedProblem &p);
cudaError_t launch_fused_tc(const FusedProblem &p, InType in, cudaStream_t stream,
                            const char **name);
// Reads and clears those kernels' device status word (after a sync).
cudaError_t fused_tc_read_and_clear_status(cudaStream_t stream, int *status);
// dbias[n] = the sum of `blocks` rows of `part` (pitch N), in a fixed order.
cudaError_t launch_column_sums(const float *part, int64_t blocks, int64_t N, float *dbias,
                               cudaStream_t stream);

}  // namespace gemm
