// combine.h -- what the two ways of combining rows share (combine.cu,
// combine_bulk.cu): pieces of 16 bytes of a row.
#pragma once

#include "mixture.h"
#include "values.cuh"

namespace gemm {

// Large batches of long rows (combine_bulk.cu).
bool combine_bulk_eligible(const CombineProblem &p, bool grad);
cudaError_t launch_combine_bulk(const CombineProblem &p, bool grad, cudaStream_t stream);

constexpr int kAll = 0, kAllOrNone = 1, kSome = 2;
template <int HELD>
__device__ __forceinline__ bool has(int i, int n) {
    return HELD == kAll || (HELD == kAllOrNone ? n > 0 : i < n);
}

// A thread's piece of a row: the 16 bytes from column c on, left packed until all
// loads are under way (unpacking them one by one waits for each: 16384 tokens, 8
// rows of 4096 BF16: 634 us).  n of its values are inside the row, the rest is 0.
// HELD: all are, all or none, any number.  VEC: the row starts on 16 bytes.
template <int TYPE, bool VEC, int HELD>
__device__ __forceinline__ uint4 load_piece(const void *matrix, int64_t row_at, int64_t c, int n) {
    using V = Value<TYPE>;
    using Raw = typename V::Raw;
    const Raw *const from = static_cast<const Raw *>(matrix) + row_at + c;
    if constexpr (VEC && HELD != kSome) {
        return HELD == kAll || n > 0 ? __ldg(reinterpret_cast<const uint4 *>(from)) : make_uint4(0, 0, 0, 0);
    } else {
        uint32_t w[4] = {};
#pragma unroll
        for (int i = 0; i < V::PER_16; ++i) {
            if (!has<HELD>(i, n)) continue;
            if constexpr (TYPE == kOutF32)
                w[i] = __float_as_uint(__ldg(from + i));
            else
                w[i / 2] |= static_cast<uint32_t>(__ldg(from + i)) << (i % 2 * 16);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// WIDE values of a matrix of another type (the result, the residual, dD), as above;
// vec: its rows start on 16 bytes.
// (Plain loads: the residual may be the result.)
template <int TYPE, int HELD, int WIDE>
__device__ __forceinline__ void store_values(void *matrix, int64_t row_at, int64_t c, int n, bool vec,
                                             const float (&v)[WIDE]) {
    using V = Value<TYPE>;
    typename V::Raw *const to = static_cast<typename V::Raw *>(matrix) + row_at + c;
    if (vec && HELD != kSome) {
#pragma unroll
        for (int i = 0; i < WIDE / V::PER_16; ++i)
            if (HELD == kAll || n > 0) reinterpret_cast<uint4 *>(to)[i] = V::pack(v + i * V::PER_16);
    } else {
#pragma unroll
        for (int i = 0; i < WIDE; ++i)
            if (has<HELD>(i, n)) to[i] = V::narrow(v[i]);
    }
}
template <int TYPE, int HELD, int WIDE>
__device__ __forceinline__ void load_values(const void *matrix, int64_t row_at, int64_t c, int n,
                                            bool vec, float (&v)[WIDE]) {
    using V = Value<TYPE>;
    const typename V::Raw *const from = static_cast<const typename V::Raw *>(matrix) + row_at + c;
    if (vec && HELD != kSome) {
#pragma unroll
        for (int i = 0; i < WIDE / V::PER_16; ++i) {
            float part[V::PER_16] = {};
            if (HELD == kAll || n > 0) V::unpack(reinterpret_cast<const uint4 *>(from)[i], part);
#pragma unroll
            for (int j = 0; j < V::PER_16; ++j) v[i * V::PER_16 + j] = part[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < WIDE; ++i) v[i] = has<HELD>(i, n) ? V::widen(from[i]) : 0.f;
    }
}

// One of C pieces from column c0 on, `apart` columns apart, holds the row's end and
// is not whole.
template <int WIDE, int C>
__device__ __forceinline__ bool has_end(int64_t N, int64_t c0, int64_t apart) {
    bool end = false;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t left = N - (c0 + c * apart);
        end |= left > 0 && left < WIDE;
    }
    return end;
}

}  // namespace gemm
