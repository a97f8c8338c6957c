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
    int row_vec;  // bytes every row of D (and C) is aligned to: 16, 8 or 0 (less)
};

__device__ __forceinline__ uint32_t pack_16(float lo, float hi, int out) {
    if (out == kOutBf16) return pack_bf16x2(lo, hi);
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
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

// The same block so that lane l holds quad l % 8 (columns 4 (l % 8) .. + 3) of
// the rows 8 (l / 8) + i in v[4 i .. 4 i + 3]: eight lanes then cover a row's 32
// columns, and a warp's 16-byte access four whole 128-byte lines.  (One row per
// lane with 32-byte accesses costs a request per sector: a 256 x 256 FP32 tile
// took 4.2 us to write, 9 us with C.)
__device__ __forceinline__ void transpose_quads(float (&v)[32]) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int s = 4; s > 0; s >>= 1) {
        const bool high = (lane & s) != 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k & s) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float give = high ? v[k * 4 + j] : v[(k + s) * 4 + j];
                const float got = __shfl_xor_sync(0xffffffffu, give, s);
                if (high)
                    v[k * 4 + j] = got;
                else
                    v[(k + s) * 4 + j] = got;
            }
        }
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
    return grouped_activation(x, act);
}

// A block is 32 rows of D from row0 on (nrows of them inside) and 32 columns
// from c0 on (width inside); v holds lane l's accumulators of row row0 + l.
// Where rows start on whole quads (16 bytes of FP32, 8 of 16-bit values) the
// block is written in quads, otherwise one column per lane (transpose_32x32).
__device__ __forceinline__ bool in_quads(const OutArgs &a) {
    return a.row_vec >= (a.out == kOutF32 ? 16 : 8);
}

// This lane's quads of C.
__device__ __forceinline__ void load_c_quads(const OutArgs &a, int64_t row0, int nrows, int64_t c0,
                                             int width, float (&c)[32]) {
    const int lane = threadIdx.x % 32, col = (lane % 8) * 4, first = (lane / 8) * 8;
    const float *p = a.C + (row0 + first) * a.ldc + c0 + col;
#pragma unroll
    for (int i = 0; i < 8; ++i, p += a.ldc) {
        if (first + i >= nrows) continue;
        if (col + 4 <= width) {
            const float4 q = *reinterpret_cast<const float4 *>(p);
            c[i * 4 + 0] = q.x, c[i * 4 + 1] = q.y, c[i * 4 + 2] = q.z, c[i * 4 + 3] = q.w;
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (col + j < width) c[i * 4 + j] = p[j];
        }
    }
}

// v = act(alpha v + bias + beta c), in quads (after transpose_quads).
template <bool WITH_C>
__device__ __forceinline__ void finish_quads(float (&v)[32], const float (&c)[32],
                                             const OutArgs &a, int64_t c0, int width) {
    const int col = (threadIdx.x % 8) * 4;
    float b[4] = {};
    if (!WITH_C && a.bias != nullptr) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (col + j < width) b[j] = a.bias[c0 + col + j];
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = fmaf(v[i], a.alpha, b[i % 4]);
    if (WITH_C && a.beta != 0.f) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = fmaf(a.beta, c[i], v[i]);
    }
    if (!WITH_C && a.act != kActNone) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = activate(v[i], a.act);
    }
}

__device__ __forceinline__ void store_quads(const float (&v)[32], const OutArgs &a, int64_t row0,
                                            int nrows, int64_t c0, int width) {
    const int lane = threadIdx.x % 32, col = (lane % 8) * 4, first = (lane / 8) * 8;
    if (col >= width) return;
    const int64_t at = (row0 + first) * a.ldd + c0 + col;
    const bool whole = col + 4 <= width;
    if (a.out == kOutF32) {
        float *d = static_cast<float *>(a.D) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i, d += a.ldd) {
            if (first + i >= nrows) continue;
            if (whole) {
                *reinterpret_cast<float4 *>(d) =
                    make_float4(v[i * 4], v[i * 4 + 1], v[i * 4 + 2], v[i * 4 + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (col + j < width) d[j] = v[i * 4 + j];
            }
        }
    } else {
        uint16_t *d = static_cast<uint16_t *>(a.D) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i, d += a.ldd) {
            if (first + i >= nrows) continue;
            const uint32_t lo = pack_16(v[i * 4], v[i * 4 + 1], a.out);
            const uint32_t hi = pack_16(v[i * 4 + 2], v[i * 4 + 3], a.out);
            if (whole) {
                *reinterpret_cast<uint2 *>(d) = make_uint2(lo, hi);
            } else {
                d[0] = static_cast<uint16_t>(lo);
                if (col + 1 < width) d[1] = static_cast<uint16_t>(lo >> 16);
                if (col + 2 < width) d[2] = static_cast<uint16_t>(hi);
            }
        }
    }
}

// Rows that start anywhere: one column per lane (after transpose_32x32, v[i] is
// row row0 + i).  C is loaded ahead as for the quads.
__device__ __forceinline__ void load_c_columns(const OutArgs &a, int64_t row0, int nrows, int64_t c0,
                                               int width, float (&c)[32]) {
    const int lane = threadIdx.x % 32;
    if (lane >= width) return;
    const float *p = a.C + row0 * a.ldc + c0 + lane;
#pragma unroll
    for (int i = 0; i < 32; ++i, p += a.ldc)
        if (i < nrows) c[i] = *p;
}

template <bool WITH_C>
__device__ __forceinline__ void finish_columns(float (&v)[32], const float (&c)[32],
                                               const OutArgs &a, int64_t c0, int width) {
    const int lane = threadIdx.x % 32;
    const float b = !WITH_C && a.bias != nullptr && lane < width ? a.bias[c0 + lane] : 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = fmaf(v[i], a.alpha, b);
    if (WITH_C && a.beta != 0.f) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = fmaf(a.beta, c[i], v[i]);
    }
    if (!WITH_C && a.act != kActNone) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = activate(v[i], a.act);
    }
}

__device__ __forceinline__ void store_columns(const float (&v)[32], const OutArgs &a, int64_t row0,
                                              int nrows, int64_t c0, int width) {
    const int lane = threadIdx.x % 32;
    if (lane >= width) return;
    const int64_t at = row0 * a.ldd + c0 + lane;
    if (a.out == kOutF32) {
        float *d = static_cast<float *>(a.D) + at;
#pragma unroll
        for (int i = 0; i < 32; ++i, d += a.ldd)
            if (i < nrows) *d = v[i];
    } else {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack_16(v[2 * i], v[2 * i + 1], a.out);
        uint16_t *d = static_cast<uint16_t *>(a.D) + at;
#pragma unroll
        for (int i = 0; i < 32; ++i, d += a.ldd)
            if (i < nrows) *d = static_cast<uint16_t>(w[i / 2] >> (i % 2 * 16));
    }
}

// An FP32 block by way of a box of shared memory: 4 KiB of the warp's own,
// 1024-byte aligned, rows of 128 bytes whose 16-byte pieces change places with
// the row.  Lane l puts its 32 sums into row l; the warp takes whole rows out,
// four at a time in quads or one at a time.
__device__ __forceinline__ uint32_t box_quad(int row, int q) {
    return row * 128 + ((q ^ (row & 7)) << 4);
}

template <bool WITH_C>
__device__ __forceinline__ void store_from_box(uint32_t box, const OutArgs &a, int64_t row0,
                                               int nrows, int64_t c0, int width) {
    const int lane = threadIdx.x % 32;
    const bool with_c = WITH_C && a.beta != 0.f;
    if (a.row_vec >= 16 && width >= 32) {
        const int quad = lane % 8, first = lane / 8;
        const int64_t col = c0 + quad * 4;
        float b[4] = {};
        if (!WITH_C && a.bias != nullptr) {
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = a.bias[col + j];
        }
        float *d = static_cast<float *>(a.D) + (row0 + first) * a.ldd + col;
        const float *c = with_c ? a.C + (row0 + first) * a.ldc + col : nullptr;
        // (C may be D: a few rows of C are loaded before the first is stored)
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
            float4 q[4], x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = ld_shared_v4(box + box_quad(first + 4 * (h + i), quad));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (with_c && first + 4 * (h + i) < nrows)
                    q[i] = *reinterpret_cast<const float4 *>(c + 4 * (h + i) * a.ldc);
#pragma unroll
            for (int i = 0; i < 4; ++i, d += 4 * a.ldd) {
                const int row = first + 4 * (h + i);
                if (row >= nrows) continue;
                float v[4] = {fmaf(x[i].x, a.alpha, b[0]), fmaf(x[i].y, a.alpha, b[1]),
                              fmaf(x[i].z, a.alpha, b[2]), fmaf(x[i].w, a.alpha, b[3])};
                if (with_c) {
                    v[0] = fmaf(a.beta, q[i].x, v[0]), v[1] = fmaf(a.beta, q[i].y, v[1]);
                    v[2] = fmaf(a.beta, q[i].z, v[2]), v[3] = fmaf(a.beta, q[i].w, v[3]);
                }
                if (!WITH_C && a.act != kActNone) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = activate(v[j], a.act);
                }
                *reinterpret_cast<float4 *>(d) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
    } else if (lane < width) {
        const float b = !WITH_C && a.bias != nullptr ? a.bias[c0 + lane] : 0.f;
        float *d = static_cast<float *>(a.D) + row0 * a.ldd + c0 + lane;
        const float *c = with_c ? a.C + row0 * a.ldc + c0 + lane : nullptr;
#pragma unroll 1
        for (int h = 0; h < nrows; h += 8) {
            float q[8], x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = ld_shared_f32(box + box_quad(h + i, lane / 4) + lane % 4 * 4);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (with_c && h + i < nrows) q[i] = c[(h + i) * a.ldc];
#pragma unroll
            for (int i = 0; i < 8; ++i, d += a.ldd) {
                if (h + i >= nrows) continue;
                float v = fmaf(x[i], a.alpha, b);
                if (with_c) v = fmaf(a.beta, q[i], v);
                if (!WITH_C) v = activate(v, a.act);
                *d = v;
            }
        }
    }
}

// Bytes (16, 8 or 0 for less) to which every row of a matrix of `elt`-byte
// values starting at p, with these pitches (elements), is aligned.
inline int row_alignment(const void *p, int64_t ld, int64_t stride, int64_t elt) {
    const auto all = static_cast<uint64_t>(reinterpret_cast<uintptr_t>(p)) |
                     static_cast<uint64_t>(ld * elt) | static_cast<uint64_t>(stride * elt);
    return all % 16 == 0 ? 16 : (all % 8 == 0 ? 8 : 0);
}

}  // namespace tc
}  // namespace gemm
