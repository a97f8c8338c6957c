// fused.cuh -- activations and their slopes.
//
// GELU (tanh form) and SiLU are x times a logistic function: of 2 u, u =
// sqrt(2/pi) (x + 0.044715 x^3), and of x, as 0.5 (1 + tanh u) = 1 / (1 + exp(-2u)).
// With e = exp(-|argument|), which cannot overflow, the logistic function of the
// argument's magnitude is 1 / (1 + e) and that of its negative e / (1 + e): both
// are as accurate as e, also far in the tails.  FAST takes the hardware's
// exponential and division (a few units of 2^-22) for results of 16 bits.
#pragma once

#include <cstdint>

#include "epilogue.cuh"
#include "fused.h"

namespace gemm {

template <bool FAST>
__device__ __forceinline__ void logistic(float arg, float &s, float &pair) {
    const float e = FAST ? __expf(-fabsf(arg)) : expf(-fabsf(arg));
    const float p = FAST ? __fdividef(1.f, 1.f + e) : 1.f / (1.f + e);
    const float q = e * p;
    s = arg >= 0.f ? p : q;  // (a NaN argument: e and q are NaN)
    pair = p * q;            // s (1 - s)
}

template <bool FAST>
__device__ __forceinline__ float fused_activation(float x, int act) {
    if (act == kActNone) return x;
    if (act == kActRelu) return x <= 0.f ? 0.f : x;
    const float arg = act == kActGelu ? 1.5957691216057308f * fmaf(0.044715f * x, x * x, x) : x;
    float s, pair;
    logistic<FAST>(arg, s, pair);
    return x * s;
}

// The derivative; a NaN stays one, infinities have the limits 0 and 1.
template <bool FAST>
__device__ __forceinline__ float fused_slope(float x, int act) {
    if (act == kActNone) return 1.f;
    if (act == kActRelu) return x > 0.f ? 1.f : (x <= 0.f ? 0.f : x);
    // past 12 (GELU) and 110 (SiLU) the slope is 0 or 1 in FP32
    const float most = act == kActGelu ? 12.f : 110.f;
    const float c = x > most ? most : (x < -most ? -most : x);  // (a NaN stays)
    float arg = c, rise = 1.f;
    if (act == kActGelu) {
        const float c2 = c * c;
        arg = 1.5957691216057308f * fmaf(0.044715f * c, c2, c);
        rise = 1.5957691216057308f * fmaf(3.f * 0.044715f, c2, 1.f);
    }
    float s, pair;
    logistic<FAST>(arg, s, pair);
    return fmaf(c * pair, rise, s);
}

}  // namespace gemm
