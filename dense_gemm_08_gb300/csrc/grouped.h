// grouped.h -- the grouped operators' problems, as the host dispatcher hands
// them to the kernel launchers (all argument checks done).
//
// A group owns a run of rows: group g's rows are [offsets[g], offsets[g + 1])
// of the product's rows.  `offsets` (groups + 1 values) lives on the device
// and is read by the kernels only, so the host never waits for it; kernels
// clamp every value to [0, rows].  Product row r reads row row_index[r] of A
// (row r when row_index is null); an index outside [0, rows_a) reads zeros.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "internal.h"

namespace gemm {

enum : int { kOutF32 = 0, kOutBf16 = 1, kOutF16 = 2 };  // = gemm_d_type_t

// D(r, :) = act(alpha * A(idx(r), :) * op(B_g) + bias_g) for the rows r of group g.
struct GroupedProblem {
    int64_t groups, rows, N, K;
    float alpha;
    const void *A;
    int64_t lda, rows_a;
    const int32_t *row_index;
    const int32_t *offsets;
    const void *B;
    int64_t ldb, stride_b;
    bool b_kmajor;  // B_g(k, j) at B[g * stride_b + k + j * ldb]; else B[g * stride_b + k * ldb + j]
    void *D;
    int64_t ldd;
    const float *bias;  // [groups][N] or null
    int act, out;
};

// D_g = alpha * sum over the rows r of group g of A(idx(r), :)^T B(r, :) + beta * C_g.
struct WgradProblem {
    int64_t groups, rows, M, N;
    float alpha, beta;
    const void *A;
    int64_t lda, rows_a;
    const int32_t *row_index;
    const int32_t *offsets;
    const void *B;
    int64_t ldb;
    const float *C;
    int64_t ldc, stride_c;
    void *D;
    int64_t ldd, stride_d;
    int out;
};

// D(i, :) = act(X(i, :) * op(W) + s_a (X(i, :) * op(LA_a)) * op(LB_a) + bias),
// a = adapter[i]; rows whose a lies outside [0, adapters) take X op(W) + bias alone.
struct LoraProblem {
    int64_t M, N, K, adapters, rank;
    const void *X;
    int64_t ldx;
    const void *W;
    int64_t ldw;
    bool w_kmajor;  // as GroupedProblem::b_kmajor
    const int32_t *adapter;
    const float *scale;  // [adapters] or null (all 1)
    const void *LA;      // K x rank each
    int64_t ld_a, stride_a;
    bool a_kmajor;  // LA_a(k, j) at LA[a * stride_a + k + j * ld_a]; else [.. + k * ld_a + j]
    const void *LB;  // rank x N each
    int64_t ld_b, stride_b;
    bool b_kmajor;  // LB_a(j, n) at LB[a * stride_b + j + n * ld_b]; else [.. + j * ld_b + n]
    void *D;
    int64_t ldd;
    const float *bias;  // [N] or null
    int act, out;
};

// CUDA-core kernels: any type, order, leading dimension and alignment (grouped_simt.cu).
cudaError_t launch_grouped_simt(const GroupedProblem &p, InType in, cudaStream_t stream,
                                const char **name);
cudaError_t launch_wgrad_simt(const WgradProblem &p, InType in, cudaStream_t stream,
                              const char **name);
cudaError_t launch_lora_simt(const LoraProblem &p, InType in, cudaStream_t stream,
                             const char **name);

// Tensor-core kernels (grouped_tc.cu): BF16 or FP16 operands that TMA can describe.
bool grouped_tc_eligible(const GroupedProblem &p);
cudaError_t launch_grouped_tc(const GroupedProblem &p, InType in, cudaStream_t stream,
                              const char **name);
bool wgrad_tc_eligible(const WgradProblem &p);
cudaError_t launch_wgrad_tc(const WgradProblem &p, InType in, cudaStream_t stream,
                            const char **name);
bool lora_tc_eligible(const LoraProblem &p);
cudaError_t launch_lora_tc(const LoraProblem &p, InType in, cudaStream_t stream, const char **name);

// What the first product of gemm_lora leaves for the second (lora_shrink.cu).
// Rows are taken in tiles of tile_rows (at most 256); a tile's distinct
// adapters have slots 0 .. count - 1.  V is a matrix of one row per row of X
// with rc columns per slot: row i holds s_a X(i) LA_a rounded to the inputs'
// type in its own adapter's slot (r_pad columns, and, when rc = 2 r_pad, the
// rounding's remainder in r_pad more) and zeros in the tile's other slots.
struct LoraPlan {
    int tile_rows, r_pad, rc;
    uint16_t *V;
    int64_t ldv;
    int *count;  // [tiles] slots in use
    int *list;   // [tiles][tile_rows] the slots' adapters
    int *slot;   // [rows] each row's slot, -1: no adapter
    // lora_shrink_part_bytes of scratch, [parts of K][rows][r_pad] sums; it
    // leaves s_a X(i) LA_a, not rounded, in the first rows x r_pad of them
    float *part;
};
cudaError_t launch_lora_shrink(const LoraProblem &p, const LoraPlan &plan, InType in,
                               cudaStream_t stream);
bool lora_shrink_eligible(const LoraProblem &p);
size_t lora_shrink_part_bytes(int64_t rows, int r_pad);
cudaError_t lora_shrink_read_and_clear_status(cudaStream_t stream, int *status);

// Reads and clears those kernels' device status word (after a sync); 0 without a
// copy while none of them has been launched on the device.
cudaError_t grouped_tc_read_and_clear_status(cudaStream_t stream, int *status);

// Rows grouped by a number (group_rows.cu).
cudaError_t launch_group_rows(int64_t rows, int64_t groups, const int32_t *group_of_row,
                              int32_t *offsets, int32_t *order, int32_t *position,
                              cudaStream_t stream, const char **name);

}  // namespace gemm
