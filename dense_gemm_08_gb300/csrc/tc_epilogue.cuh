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

// GELU in its tanh form, x / (1 + exp(-2 u)) with u = sqrt(2/pi) (x + 0.044715 x^3):
// 0.5 (1 + tanh u) is the logistic function of 2 u.  The fast exponential and
// division are off by a few units of 2^-22, a quarter of a BF16 ulp's 2^-13.
__device__ __forceinline__ float activate(float x, int act) {
    if (act == kActGelu) {
        const float u = 0.7978845608028654f * fmaf(0.044715f * x, x * x, x);
        return __fdividef(x, 1.f + __expf(-2.f * u));
    }
    return apply_activation(x, act);
}

// A block is 32 rows of D from row0 on (nrows of them inside) and 32 columns
// from c0 on (width inside); v holds lane l's accumulators of row row0 + l.
// Whole blocks with aligned rows go straight from registers, each lane its own
// row (whole 32-byte sectors); others are transposed first, so that a store
// instruction writes consecutive columns of one row.
__device__ __forceinline__ bool direct_block(const OutArgs &a, int width) {
    return width == 32 && a.row_vec >= 16;
}

// v = act(alpha v + bias + beta c); c is this lane's row of C.
template <bool WITH_C>
__device__ __forceinline__ void finish_direct(float (&v)[32], const float (&c)[32],
                                              const OutArgs &a, int64_t c0) {
    if (!WITH_C && a.bias != nullptr) {
        const float mine = a.bias[c0 + threadIdx.x % 32];
#pragma unroll
        for (int j = 0; j < 32; ++j)
            v[j] = fmaf(v[j], a.alpha, __shfl_sync(0xffffffffu, mine, j));
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= a.alpha;
    }
    if (WITH_C && a.beta != 0.f) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = fmaf(a.beta, c[j], v[j]);
    }
    if (!WITH_C && a.act != kActNone) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = activate(v[j], a.act);
    }
}

__device__ __forceinline__ void store_direct(const float (&v)[32], const OutArgs &a, int64_t row0,
                                             int nrows, int64_t c0) {
    const int lane = threadIdx.x % 32;
    if (lane >= nrows) return;
    const int64_t at = (row0 + lane) * a.ldd + c0;
    if (a.out == kOutF32) {
        float *d = static_cast<float *>(a.D) + at;
        if (a.row_vec >= 32) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                st_global_v8(d + q * 8, __float_as_uint(v[q * 8 + 0]), __float_as_uint(v[q * 8 + 1]),
                             __float_as_uint(v[q * 8 + 2]), __float_as_uint(v[q * 8 + 3]),
                             __float_as_uint(v[q * 8 + 4]), __float_as_uint(v[q * 8 + 5]),
                             __float_as_uint(v[q * 8 + 6]), __float_as_uint(v[q * 8 + 7]));
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                st_global_v4(d + q * 4, __float_as_uint(v[q * 4 + 0]), __float_as_uint(v[q * 4 + 1]),
                             __float_as_uint(v[q * 4 + 2]), __float_as_uint(v[q * 4 + 3]));
        }
    } else {
        uint16_t *d = static_cast<uint16_t *>(a.D) + at;
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = pack_16(v[2 * j], v[2 * j + 1], a.out);
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

__device__ __forceinline__ void store_transposed(float (&v)[32], const OutArgs &a, int64_t row0,
                                                 int nrows, int64_t c0, int width) {
    const int lane = threadIdx.x % 32;
    transpose_32x32(v);  // v[i] = row row0 + i, this lane's column
    if (lane >= width) return;
    const float b = a.bias != nullptr ? a.bias[c0 + lane] : 0.f;
    const bool use_c = a.beta != 0.f;
    const float *cp = use_c ? a.C + row0 * a.ldc + c0 + lane : nullptr;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        v[i] = fmaf(v[i], a.alpha, b);
        if (use_c) {
            if (i < nrows) v[i] = fmaf(a.beta, *cp, v[i]);
            cp += a.ldc;
        }
        v[i] = activate(v[i], a.act);
    }
    const int64_t at = row0 * a.ldd + c0 + lane;
    if (a.out == kOutF32) {
        float *d = static_cast<float *>(a.D) + at;
#pragma unroll
        for (int i = 0; i < 32; ++i, d += a.ldd)
            if (i < nrows) *d = v[i];
    } else {
        uint16_t *d = static_cast<uint16_t *>(a.D) + at;
#pragma unroll
        for (int i = 0; i < 32; ++i, d += a.ldd)
            if (i < nrows) *d = static_cast<uint16_t>(pack_16(v[i], 0.f, a.out));
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
