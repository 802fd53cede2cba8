// dt_act.h -- the activations of the matrix products, and their slopes.
//   relu: max(z, 0), slope 0 at 0;   gelu: z Phi(z), Phi the distribution function of
//   the normal distribution;   silu: z s, s = 1 / (1 + exp(-z)).  NaN stays NaN.
#pragma once

#include "dt_step_device.h"

namespace dt {
namespace {

// Phi(z) and exp(-z^2 / 2).  With x = |z| / sqrt(2), t = 1 / (1 + 0.38 x):
// erfc(x) = exp(-x^2) t P(t), P a polynomial of degree 8 close to erfcx(x) / t by
// its relative error: 5.7e-8 for x up to 11 with the constants rounded to fp32 as
// they are here, 4.5e-8 at 0 (fitted in 64 bits by weighted least squares); so Phi
// keeps its digits in the tail as well.  The exponential's argument is off by half a
// step of z^2 / 2 and more counts in the tail: within 0.6 (4 z^2 + 20) half steps of
// fp32 in all, measured over |z| < 13.
// Eighteen instructions, where erfcf takes several times as many.
__device__ __forceinline__ float phi_of(float z, float& bell) {
    const float x = fabsf(z) * .70710678f;
    bell = __builtin_amdgcn_exp2f(x * x * -kLog2e);
    const float t = __builtin_amdgcn_rcpf(1.f + .38f * x);
    float q = .05904170870780945f;
    q = q * t - .2626591920852661f;
    q = q * t + .364676296710968f;
    q = q * t - .16243553161621094f;
    q = q * t + .23073482513427734f;
    q = q * t + .13833019137382507f;
    q = q * t + .20399367809295654f;
    q = q * t + .21390627324581146f;
    q = q * t + .21441179513931274f;
    const float half = .5f * bell * t * q;
    return z < 0.f ? half : 1.f - half;
}
// 1 / (1 + exp(-z)): the hardware's exponential and reciprocal are within a step.
__device__ __forceinline__ float logistic(float z) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -kLog2e)); }

__device__ __forceinline__ float act(float z, int kind) {
    if (kind == DT_ACT_RELU) return z < 0.f ? 0.f : z;
    if (kind == DT_ACT_GELU) {
        float bell;
        return z * phi_of(z, bell);
    }
    return kind == DT_ACT_SILU ? z * logistic(z) : z;
}
// value = act(z), slope = act'(z)
__device__ __forceinline__ void act_and_slope(float z, int kind, float& value, float& slope) {
    if (kind == DT_ACT_RELU) {
        value = z < 0.f ? 0.f : z;
        slope = z <= 0.f ? 0.f : 1.f;
    } else if (kind == DT_ACT_GELU) {
        float bell;
        const float phi = phi_of(z, bell);
        value = z * phi;
        slope = phi + z * .39894228f * bell;
    } else if (kind == DT_ACT_SILU) {
        const float s = logistic(z);
        value = z * s;
        slope = s * (1.f + z * (1.f - s));
    } else {
        value = z;
        slope = 1.f;
    }
}

}  // namespace
}  // namespace dt
