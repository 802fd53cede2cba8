// dt_act.h -- the activations of the matrix products, and their slopes.
//   relu: max(z, 0), slope 0 at 0;   gelu: z Phi(z), Phi the distribution function of
//   the normal distribution;   silu: z s, s = 1 / (1 + exp(-z)).  NaN stays NaN.
#pragma once

#include "dt_step_device.h"

namespace dt {
namespace {

// value = act(z), slope = act'(z)
template <int DT>
__device__ __forceinline__ void act_and_slope(float z, int kind, float& value, float& slope) {
    if (kind == DT_ACT_RELU) {
        value = z < 0.f ? 0.f : z;
        slope = z <= 0.f ? 0.f : 1.f;
    } else if (kind == DT_ACT_GELU) {
        const float phi = .5f * erfcf(-.70710678f * z);
        value = z * phi;
        slope = phi + z * .39894228f * expf(-.5f * z * z);
    } else if (kind == DT_ACT_SILU) {
        const float s = 1.f / (1.f + expf(-z));
        value = z * s;
        slope = s * (1.f + z * (1.f - s));
    } else {
        value = z;
        slope = 1.f;
    }
}
template <int DT>
__device__ __forceinline__ float act(float z, int kind) {
    float value, slope;
    act_and_slope<DT>(z, kind, value, slope);
    return value;
}

}  // namespace
}  // namespace dt
