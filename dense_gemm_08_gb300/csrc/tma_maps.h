// tma_maps.h -- tensor maps of the grouped kernels' 16-bit operands.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

namespace gemm {
namespace tc {

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// A stack of `count` matrices of `outer` rows of `inner` 16-bit values: row
// pitch ld, matrix pitch stride (elements), boxes of box_inner x box_outer
// values of one matrix; values outside read as zero.  count = 1: 2-D maps.
inline bool encode_stack(CUtensorMap *map, bool bf16, const void *base, int64_t inner,
                         int64_t outer, int64_t ld, int64_t count, int64_t stride,
                         uint32_t box_inner, uint32_t box_outer, int rank,
                         CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
    const auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer),
                          static_cast<cuuint64_t>(count)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(stride) * 2};
    cuuint32_t box[3] = {box_inner, box_outer, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
              static_cast<cuuint32_t>(rank), const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same stack seen as blocks of 64 values of a row: a box is box_outer rows
// of box_blocks consecutive blocks, block after block.  Coordinates: 0, row,
// block, matrix (rank 3: without the matrix).  `inner` must be a multiple of 64.
inline bool encode_blocks(CUtensorMap *map, bool bf16, const void *base, int64_t inner,
                          int64_t outer, int64_t ld, int64_t count, int64_t stride,
                          uint32_t box_outer, uint32_t box_blocks, int rank) {
    const auto fn = tensor_map_encoder();
    if (fn == nullptr || inner % 64 != 0) return false;
    cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(outer), static_cast<cuuint64_t>(inner / 64),
                          static_cast<cuuint64_t>(count)};
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(ld) * 2, 128,
                             static_cast<cuuint64_t>(stride) * 2};
    cuuint32_t box[4] = {64, box_outer, box_blocks, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
              static_cast<cuuint32_t>(rank), const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A stack of K-major operands (rows of K values).  blocks = 1: boxes of box_rows
// rows of one block of 64, coordinates k, row, 0, matrix; more: encode_blocks.
inline bool encode_kmajor(CUtensorMap *map, bool bf16, const void *base, int64_t K, int64_t rows,
                          int64_t ld, int64_t count, int64_t stride, int box_rows, int blocks,
                          int rank) {
    if (blocks > 1)
        return encode_blocks(map, bf16, base, K, rows, ld, count, stride,
                             static_cast<uint32_t>(box_rows), static_cast<uint32_t>(blocks), rank);
    const auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows), 1,
                          static_cast<cuuint64_t>(count)};
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(ld) * 2,
                             static_cast<cuuint64_t>(stride) * 2};
    cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
              static_cast<cuuint32_t>(rank), const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A stack of N-major operands (rows of N values, one per K): `whole` copies
// box_cols / 64 blocks of 64 columns of box_k * 64 steps of K at once, for tiles
// inside the N / 64 whole blocks; `edge` one block (coordinates n, k, matrix).
static bool encode_nmajor(CUtensorMap *whole, CUtensorMap *edge, bool bf16, const void *base,
                          int64_t N, int64_t K, int64_t ld, int64_t count, int64_t stride,
                          int box_cols, int box_k) {
    const uint32_t steps = static_cast<uint32_t>(64 * box_k);
    if (!encode_stack(edge, bf16, base, N, K, ld, count, stride, 64, steps, 3)) return false;
    *whole = *edge;
    return N < 64 || encode_blocks(whole, bf16, base, N / 64 * 64, K, ld, count, stride, steps,
                                   static_cast<uint32_t>(box_cols / 64), 4);
}

// A stack of matrices as 32 x 32 boxes for the epilogue, of FP32 (128-byte rows
// and swizzle) or 16-bit values (64-byte).
inline bool encode_box32(CUtensorMap *map, int elt, bool bf16, const void *base, int64_t N, int64_t M,
                         int64_t ld, int64_t count, int64_t stride) {
    const auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M),
                          static_cast<cuuint64_t>(count)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * elt, static_cast<cuuint64_t>(stride) * elt};
    cuuint32_t box[3] = {32, 32, 1}, estr[3] = {1, 1, 1};
    const CUtensorMapDataType type = elt == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : bf16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return fn(map, type, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              elt == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What TMA asks of a matrix: 16-byte aligned base, row pitch (and matrix
// pitch) of whole 16 bytes and below 2^40 bytes.
inline bool tma_rows(const void *p, int64_t ld, int64_t stride = 0) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0 && stride % 8 == 0 &&
           ld < (int64_t(1) << 39) && stride < (int64_t(1) << 39);
}

}  // namespace tc
}  // namespace gemm
