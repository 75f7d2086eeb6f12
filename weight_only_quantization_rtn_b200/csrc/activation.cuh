// Activations of the gated feed-forward block, in binary32.
//
//   silu       x·p, p = 1/(1 + e^−x)                    derivative p·(1 + x·(1 − p))
//   gelu       x·Φ(x), Φ(x) = (1 + erf(x/√2))/2          Φ(x) + x·φ(x)
//   gelu_tanh  x/2·(1 + t), t = tanh(c·(x + a·x³))       (1 + t)/2 + x/2·(1 − t²)·c·(1 + 3a·x²)
//              with c = √(2/π), a = 0.044715
//   relu       max(x, 0)                                  1 for x > 0, else 0
// A NaN stays a NaN.  The results are rounded to bf16 (half a step is 2^-9 to 2^-8 of the value)
// after one more product.  The approximate exponential and quotient are off by about 2^-21 near 0
// and by more far out, where the argument's own rounding is multiplied: gelu by 1.7·10^-5 of its
// value at x = -11.7, 2^-15.8.
#pragma once

#include "../../include/w4a16.h"

namespace w4a16 {

__device__ __forceinline__ float sigmoid_f32(float x) {
    return __fdividef(1.0f, 1.0f + __expf(-x));     // e^−x = inf gives 0, e^−x = 0 gives 1
}

__device__ __forceinline__ float tanh_arg(float x) {
    return 0.7978845608028654f * (x + 0.044715f * x * x * x);
}

// (1 + erf(x/√2))/2 = erfc(−x/√2)/2.  erfc by the Chebyshev fit of Press et al., Numerical
// Recipes (function "erfcc"): t·exp(−z² + P(t)), t = 1/(1 + z/2), fractional error below
// 1.2·10^-7 for every z ≥ 0, and 2 − erfc(z) for the other sign.
__device__ __forceinline__ float normal_cdf(float x) {
    const float z = fabsf(x) * 0.7071067811865476f;
    const float t = __fdividef(1.0f, 1.0f + 0.5f * z);
    float p = 0.17087277f;
    p = p * t - 0.82215223f;
    p = p * t + 1.48851587f;
    p = p * t - 1.13520398f;
    p = p * t + 0.27886807f;
    p = p * t - 0.18628806f;
    p = p * t + 0.09678418f;
    p = p * t + 0.37409196f;
    p = p * t + 1.00002368f;
    p = p * t - 1.26551223f;
    const float c = 0.5f * t * __expf(p - z * z);         // Φ(−|x|)
    return x < 0.0f ? c : 1.0f - c;
}

__device__ __forceinline__ float act_value(int kind, float x) {
    if (kind == W4A16_ACT_SILU) return x * sigmoid_f32(x);
    if (kind == W4A16_ACT_GELU) return x * normal_cdf(x);
    // (1 + tanh y)/2 = sigmoid(2y)
    if (kind == W4A16_ACT_GELU_TANH) return x * sigmoid_f32(2.0f * tanh_arg(x));
    return x != x ? x : fmaxf(x, 0.0f);
}

// The activation and its derivative.
__device__ __forceinline__ void act_value_grad(int kind, float x, float& a, float& d) {
    if (kind == W4A16_ACT_SILU) {
        const float p = sigmoid_f32(x);
        a = x * p;
        d = p * (1.0f + x * (1.0f - p));
    } else if (kind == W4A16_ACT_GELU) {
        const float c = normal_cdf(x);
        a = x * c;
        d = c + x * (0.3989422804014327f * __expf(-0.5f * x * x));
    } else if (kind == W4A16_ACT_GELU_TANH) {
        const float c = sigmoid_f32(2.0f * tanh_arg(x));          // (1 + t)/2
        a = x * c;
        // (1 − t²)/2 = 2·c·(1 − c)
        // (x² bounded: far out the middle factor is 0, and 0·inf would be a NaN)
        d = c + x * (2.0f * c * (1.0f - c)) * (0.7978845608028654f * (1.0f + 0.134145f * fminf(x * x, 1e30f)));
    } else {
        a = x != x ? x : fmaxf(x, 0.0f);
        d = x > 0.0f ? 1.0f : 0.0f;
    }
}

}  // namespace w4a16
