// grouped.cuh -- device code shared by the grouped operators' kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "epilogue.cuh"
#include "grouped.h"

namespace gemm {

// Walks the tiles of all groups in order: a group of m rows has
// ceil(m / tile_rows) * per_row tiles.  The 32 lanes of a warp hold 32 groups
// at a time (one load and one warp scan per 32 groups), so a tile's group is
// found without a table in shared memory and without the host knowing the
// sizes.  Offsets count as the largest clamped value so far, so groups never
// share a row, whatever the values.  locate() must be called by the whole
// warp, with tile numbers that never fall.
struct GroupWalk {
    const int32_t *offsets;
    int groups;
    int64_t rows;
    int tile_rows;
    uint32_t per_row;
    int chunk = -32;         // first group the lanes hold
    uint32_t base = 0;       // tiles before that group
    uint32_t chunk_tiles = 0;
    uint32_t incl = 0;       // this lane's group and the ones before it in the chunk
    int32_t lo = 0, hi = 0;  // this lane's group's rows
    int32_t reached = 0;     // largest offset of the chunks before

    __device__ __forceinline__ GroupWalk(const int32_t *offsets, int64_t groups, int64_t rows,
                                         int tile_rows, uint32_t per_row)
        : offsets(offsets),
          groups(static_cast<int>(groups)),
          rows(rows),
          tile_rows(tile_rows),
          per_row(per_row) {}

    __device__ __forceinline__ int32_t bounded(int32_t v) const {
        return v < 0 ? 0 : (v > rows ? static_cast<int32_t>(rows) : v);
    }

    // The group, its rows and the tile's number inside it; false past the last tile.
    __device__ __forceinline__ bool locate(uint32_t t, int &g, int32_t &first, int32_t &last,
                                           uint32_t &in_group) {
        const int lane = threadIdx.x % 32;
        while (t >= base + chunk_tiles) {
            if (chunk + 32 >= groups) return false;
            base += chunk_tiles;
            chunk += 32;
            const int mine = chunk + lane;
            lo = hi = 0;
            if (mine < groups) {
                lo = bounded(__ldg(offsets + mine));
                hi = bounded(__ldg(offsets + mine + 1));
            }
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t below = __shfl_up_sync(0xffffffffu, lo, d);
                if (lane >= d && below > lo) lo = below;
            }
            if (lo < reached) lo = reached;
            if (hi < lo) hi = lo;
            reached = __shfl_sync(0xffffffffu, hi, 31);
            incl = static_cast<uint32_t>((static_cast<int64_t>(hi) - lo + tile_rows - 1) / tile_rows) * per_row;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t below = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += below;
            }
            chunk_tiles = __shfl_sync(0xffffffffu, incl, 31);
        }
        const uint32_t r = t - base;
        const int owner = __ffs(__ballot_sync(0xffffffffu, incl > r)) - 1;
        const uint32_t before = __shfl_sync(0xffffffffu, incl, owner ? owner - 1 : 0);
        g = chunk + owner;
        first = __shfl_sync(0xffffffffu, lo, owner);
        last = __shfl_sync(0xffffffffu, hi, owner);
        in_group = r - (owner ? before : 0u);
        return true;
    }
};

// The activation of a grouped product.  ReLU passes a NaN on, as the sum it
// comes from does (fmaxf(NaN, 0) would be 0).
__device__ __forceinline__ float grouped_activation(float x, int act) {
    if (act == kActRelu) return x <= 0.f ? 0.f : x;
    return apply_activation(x, act);
}

// One value in the type of D.  16-bit results are rounded to nearest even,
// once, from the FP32 accumulator after the whole epilogue.
__device__ __forceinline__ void store_out(void *D, int64_t at, float v, int out) {
    if (out == kOutF32)
        static_cast<float *>(D)[at] = v;
    else if (out == kOutBf16)
        static_cast<uint16_t *>(D)[at] = to_bf16_bits(v);
    else
        static_cast<__half *>(D)[at] = __float2half_rn(v);
}

}  // namespace gemm
