// tc_epilogue.cuh -- how the grouped tensor-core kernels write D: 32 x 32
// blocks from TMEM through registers, rows of any alignment.
#pragma once

#include "grouped.cuh"
#include "tcgen05.cuh"

namespace gemm {
namespace tc {

struct OutArgs {
    void *D;
    int64_t ldd;
    const float *bias;  // one value per column of D, or null
    const float *C;     // read when beta != 0
    int64_t ldc;
    float alpha, beta;
    int act, out;
    int row_vec;  // bytes every row of D (and C) is aligned to: 32, 16 or 0 (less)
};

__device__ __forceinline__ uint32_t pack_16(float lo, float hi, int out) {
    if (out == kOutBf16) return pack_bf16x2(lo, hi);
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void st_global_v4(void *p, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
    asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// The warp's 32 x 32 block held one row per lane becomes one column per lane
// (an exchange per bit of the index; indices into v are fixed at compile time).
__device__ __forceinline__ void transpose_32x32(float (&v)[32]) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        const bool high = (lane & s) != 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j & s) continue;
            const float give = high ? v[j] : v[j + s];
            const float got = __shfl_xor_sync(0xffffffffu, give, s);
            if (high)
                v[j] = got;
            else
                v[j + s] = got;
        }
    }
}

// This lane's 32 values of C, row `row`, from column c0 on (rows aligned to 16 bytes).
__device__ __forceinline__ void load_c_row(const OutArgs &a, int64_t row, int64_t c0,
                                           float (&c)[32]) {
    const float4 *p = reinterpret_cast<const float4 *>(a.C + row * a.ldc + c0);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const float4 v = p[q];
        c[q * 4 + 0] = v.x;
        c[q * 4 + 1] = v.y;
        c[q * 4 + 2] = v.z;
        c[q * 4 + 3] = v.w;
    }
}

// The warp's block of D: rows row0 .. row0 + nrows - 1 (nrows <= 32), columns
// c0 .. c0 + width - 1 (width <= 32); o holds lane l's row row0 + l of the
// accumulator, c (used when beta != 0 and the block is `direct`) its row of C.
// Whole blocks with aligned rows go straight from registers, each lane its own
// row (whole 32-byte sectors); others are transposed first, so that each store
// instruction writes consecutive columns of one row.
__device__ __forceinline__ bool direct_block(const OutArgs &a, int width) {
    return width == 32 && a.row_vec >= 16;
}

__device__ __forceinline__ void emit_block(float (&o)[32], const float (&c)[32], const OutArgs &a,
                                           int64_t row0, int nrows, int64_t c0, int width) {
    const int lane = threadIdx.x % 32;
    if (!direct_block(a, width)) {
        transpose_32x32(o);  // o[i] = row row0 + i, this lane's column
        if (lane >= width) return;
        const float b = a.bias != nullptr ? a.bias[c0 + lane] : 0.f;
        int64_t at = row0 * a.ldd + c0 + lane;
        const float *cp = a.beta != 0.f ? a.C + row0 * a.ldc + c0 + lane : nullptr;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if (i < nrows) {
                float v = o[i] * a.alpha + b;
                if (a.beta != 0.f) v = fmaf(a.beta, *cp, v);
                store_out(a.D, at, apply_activation(v, a.act), a.out);
            }
            at += a.ldd;
            if (a.beta != 0.f) cp += a.ldc;
        }
        return;
    }
    if (a.bias != nullptr) {
        const float mine = a.bias[c0 + lane];
#pragma unroll
        for (int j = 0; j < 32; ++j)
            o[j] = fmaf(o[j], a.alpha, __shfl_sync(0xffffffffu, mine, j));
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] *= a.alpha;
    }
    if (a.beta != 0.f) {
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = fmaf(a.beta, c[j], o[j]);
    }
    if (a.act != kActNone) {
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = apply_activation(o[j], a.act);
    }
    if (lane >= nrows) return;
    const int64_t at = (row0 + lane) * a.ldd + c0;
    if (a.out == kOutF32) {
        float *d = static_cast<float *>(a.D) + at;
        if (a.row_vec >= 32) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                st_global_v8(d + q * 8, __float_as_uint(o[q * 8 + 0]), __float_as_uint(o[q * 8 + 1]),
                             __float_as_uint(o[q * 8 + 2]), __float_as_uint(o[q * 8 + 3]),
                             __float_as_uint(o[q * 8 + 4]), __float_as_uint(o[q * 8 + 5]),
                             __float_as_uint(o[q * 8 + 6]), __float_as_uint(o[q * 8 + 7]));
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                st_global_v4(d + q * 4, __float_as_uint(o[q * 4 + 0]), __float_as_uint(o[q * 4 + 1]),
                             __float_as_uint(o[q * 4 + 2]), __float_as_uint(o[q * 4 + 3]));
        }
    } else {
        uint16_t *d = static_cast<uint16_t *>(a.D) + at;
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = pack_16(o[2 * j], o[2 * j + 1], a.out);
        if (a.row_vec >= 32) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                st_global_v8(d + q * 16, w[q * 8 + 0], w[q * 8 + 1], w[q * 8 + 2], w[q * 8 + 3],
                             w[q * 8 + 4], w[q * 8 + 5], w[q * 8 + 6], w[q * 8 + 7]);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                st_global_v4(d + q * 8, w[q * 4 + 0], w[q * 4 + 1], w[q * 4 + 2], w[q * 4 + 3]);
        }
    }
}

// Bytes (32, 16 or 0 for less) to which every row of a matrix of `elt`-byte
// values starting at p, with these pitches (elements), is aligned.
inline int row_alignment(const void *p, int64_t ld, int64_t stride, int64_t elt) {
    const auto all = static_cast<uint64_t>(reinterpret_cast<uintptr_t>(p)) |
                     static_cast<uint64_t>(ld * elt) | static_cast<uint64_t>(stride * elt);
    return all % 32 == 0 ? 32 : (all % 16 == 0 ? 16 : 0);
}

}  // namespace tc
}  // namespace gemm
