// dt_step_device.h -- device-side building blocks of the model-step kernels:
// element access by dtype, wave and workgroup sums, the row's rank.
#pragma once

#include "dt_device.h"
#include "dt_step.h"

namespace dt {

template <int DT>
struct Elem;
template <>
struct Elem<kF32> {
    typedef float type;
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<kBF16> {
    typedef uint16_t type;
    static __device__ __forceinline__ float get(uint16_t v) { return bf16_at(v); }
    static __device__ __forceinline__ uint16_t put(float v) { return uint16_t(to_bf16(v)); }
};

constexpr float kLog2e = 1.44269504088896340736f;

// The rank that holds global row `row` (uniform across the lanes).
__device__ __forceinline__ int rank_of_row(const RowTable& t, int nranks, uint32_t row) {
    int r = 0;
    while (r + 1 < nranks && row >= t.start[r + 1]) r++;
    return r;
}

// Sums and maxima over the wave's 64 lanes, the same value in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
    return v;
}

// Sum over a workgroup of WAVES waves in a fixed order, the same value in
// every thread.  `tmp` holds WAVES floats and may be used again after the
// caller's next barrier.
template <int WAVES>
__device__ __forceinline__ float block_sum(float v, float* tmp) {
    v = wave_sum(v);
    if constexpr (WAVES == 1) return v;
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; w++) s += tmp[w];
    return s;
}

}  // namespace dt
