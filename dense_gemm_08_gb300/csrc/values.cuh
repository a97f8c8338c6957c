// values.cuh -- values of the three types, one at a time and 16 bytes at a time,
// as FP32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "epilogue.cuh"
#include "grouped.h"

namespace gemm {

template <int TYPE>
struct Value {
    static constexpr int BYTES = TYPE == kOutF32 ? 4 : 2;
    static constexpr int PER_16 = 16 / BYTES;  // values in 16 bytes
    using Raw = typename std::conditional<TYPE == kOutF32, float, uint16_t>::type;

    static __device__ __forceinline__ float widen(Raw r) {
        if constexpr (TYPE == kOutF32)
            return r;
        else if constexpr (TYPE == kOutBf16)
            return __uint_as_float(static_cast<uint32_t>(r) << 16);
        else
            return __half2float(__ushort_as_half(r));
    }
    static __device__ __forceinline__ Raw narrow(float v) {  // to nearest even
        if constexpr (TYPE == kOutF32)
            return v;
        else if constexpr (TYPE == kOutBf16)
            return to_bf16_bits(v);
        else
            return __half_as_ushort(__float2half_rn(v));
    }
    static __device__ __forceinline__ float load(const void *p, int64_t at) {
        return widen(static_cast<const Raw *>(p)[at]);
    }
    static __device__ __forceinline__ void store(void *p, int64_t at, float v) {
        static_cast<Raw *>(p)[at] = narrow(v);
    }
    static __device__ __forceinline__ void unpack(const uint4 &q, float (&v)[PER_16]) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < PER_16; ++i) {
            if constexpr (TYPE == kOutF32)
                v[i] = __uint_as_float(w[i]);
            else
                v[i] = widen(static_cast<uint16_t>(w[i / 2] >> (i % 2 * 16)));
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *v) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (TYPE == kOutF32) {
                w[i] = __float_as_uint(v[i]);
            } else if constexpr (TYPE == kOutBf16) {
                w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            } else {
                const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Bytes of a value of `type`.
inline int64_t value_bytes(int type) { return type == kOutF32 ? 4 : 2; }
// Every row of a matrix starts on 16 bytes.
inline bool rows_on_16(const void *p, int64_t ld, int64_t bytes) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * bytes % 16 == 0;
}

}  // namespace gemm
