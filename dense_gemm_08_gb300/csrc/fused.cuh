// fused.cuh -- activations and their slopes.
//
// GELU (tanh form) and SiLU are x times a logistic function: of 2 u, u =
// sqrt(2/pi) (x + 0.044715 x^3), and of x, as 0.5 (1 + tanh u) = 1 / (1 + exp(-2u)).
// With e = exp(-|argument|), which cannot overflow, the logistic function of the
// argument's magnitude is 1 / (1 + e) and that of its negative e / (1 + e): both
// are as accurate as e, also far in the tails.  The forms for results of 16 bits
// (quick_*) take the hardware's exponential and reciprocal (off by 2 + 1.2 |argument|
// units of 2^-23) and are as short as they can be: the epilogue of a tile of the
// tensor cores is bound by their number of instructions.
#pragma once

#include <cstdint>

#include "epilogue.cuh"
#include "fused.h"

namespace gemm {

__device__ __forceinline__ void logistic(float arg, float &s, float &pair) {
    const float e = expf(-fabsf(arg)), p = 1.f / (1.f + e), q = e * p;
    s = arg >= 0.f ? p : q;  // (a NaN argument: e and q are NaN)
    pair = p * q;            // s (1 - s)
}

constexpr float kTwoSqrt2OverPi = 1.5957691216057308f;

__device__ __forceinline__ float fused_activation(float x, int act) {
    if (act == kActNone) return x;
    if (act == kActRelu) return x <= 0.f ? 0.f : x;
    float s, pair;
    logistic(act == kActGelu ? kTwoSqrt2OverPi * fmaf(0.044715f * x, x * x, x) : x, s, pair);
    return x * s;
}

// The derivative; a NaN stays one, infinities have the limits 0 and 1.
__device__ __forceinline__ float fused_slope(float x, int act) {
    if (act == kActNone) return 1.f;
    if (act == kActRelu) return x > 0.f ? 1.f : (x <= 0.f ? 0.f : x);
    // past 12 (GELU) and 110 (SiLU) the slope is 0 or 1 in FP32
    const float most = act == kActGelu ? 12.f : 110.f;
    const float c = x > most ? most : (x < -most ? -most : x);  // (a NaN stays)
    float arg = c, rise = 1.f;
    if (act == kActGelu) {
        const float c2 = c * c;
        arg = kTwoSqrt2OverPi * fmaf(0.044715f * c, c2, c);
        rise = kTwoSqrt2OverPi * fmaf(3.f * 0.044715f, c2, 1.f);
    }
    float s, pair;
    logistic(arg, s, pair);
    return fmaf(c * rise, pair, s);
}

// The same with the hardware's exponential and reciprocal.
__device__ __forceinline__ float quick_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float quick_inverse(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// x in [-most, most]; a NaN stays one.
__device__ __forceinline__ float within(float x, float most) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(most));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(y), "f"(-most));
    return y;
}

constexpr float kLog2E = 1.4426950408889634f;

// (exp of a large argument is infinite, its inverse 0: x times 0)
template <int ACT>
__device__ __forceinline__ float quick_activation(float x) {
    if constexpr (ACT == kActNone) return x;
    if constexpr (ACT == kActRelu) return x <= 0.f ? 0.f : x;
    constexpr float k = -kTwoSqrt2OverPi * kLog2E;
    const float power = ACT == kActGelu ? x * fmaf(x * x, k * 0.044715f, k) : x * -kLog2E;
    return x * quick_inverse(1.f + quick_exp2(power));
}

template <int ACT>
__device__ __forceinline__ float quick_slope(float x) {
    if constexpr (ACT == kActNone) return 1.f;
    if constexpr (ACT == kActRelu) return x > 0.f ? 1.f : (x <= 0.f ? 0.f : x);
    const float c = within(x, ACT == kActGelu ? 12.f : 110.f);
    float power = c * kLog2E, rise = c;  // (rise: c times the argument's derivative)
    if constexpr (ACT == kActGelu) {
        constexpr float k = kTwoSqrt2OverPi;
        const float c2 = c * c;
        power = c * fmaf(c2, k * kLog2E * 0.044715f, k * kLog2E);
        rise = c * fmaf(c2, k * 3.f * 0.044715f, k);
    }
    const float e = quick_exp2(-fabsf(power)), p = quick_inverse(1.f + e), q = e * p;
    return fmaf(rise, p * q, power >= 0.f ? p : q);
}

}  // namespace gemm
