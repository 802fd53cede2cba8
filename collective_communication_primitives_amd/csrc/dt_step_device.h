// dt_step_device.h -- device-side building blocks of the model-step kernels:
// element access by dtype, wave and workgroup sums, the row's rank.
#pragma once

#include <type_traits>

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

// 16 bytes at an address that is aligned to elements of ES bytes only: one
// access, which the memory unit splits where it crosses a line.
template <int ES>
struct Loose;
template <>
struct Loose<2> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Loose<4> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4)));
};
// Unit u (16 bytes) of a row of `bytes` bytes that starts and ends anywhere:
// zeros behind the row's end, where nothing is read and nothing stored.
template <int ES>
__device__ __forceinline__ u32x4 load_loose(const char* row, uint32_t u, uint32_t bytes) {
    const uint32_t at = u * 16;
    u32x4 x = {0, 0, 0, 0};
    if (at + 16 <= bytes) {
        x = __builtin_nontemporal_load(reinterpret_cast<const typename Loose<ES>::type*>(row + at));
    } else if (at < bytes) {
        typedef typename std::conditional<ES == 2, uint16_t, uint32_t>::type T;
        T t[16 / ES];
#pragma unroll
        for (int e = 0; e < 16 / ES; e++)
            t[e] = at + e * ES < bytes ? *reinterpret_cast<const T*>(row + at + e * ES) : T(0);
        __builtin_memcpy(&x, t, 16);
    }
    return x;
}
template <int ES>
__device__ __forceinline__ void store_loose(char* row, uint32_t u, uint32_t bytes, u32x4 x) {
    const uint32_t at = u * 16;
    if (at + 16 <= bytes) {
        const typename Loose<ES>::type v = x;
        __builtin_nontemporal_store(v, reinterpret_cast<typename Loose<ES>::type*>(row + at));
    } else if (at < bytes) {
        // eight, four and two bytes of what is left of the row
        typedef uint32_t Two __attribute__((ext_vector_type(2), aligned(2)));
        typedef uint32_t One __attribute__((aligned(2)));
        char* to = row + at;
        if ((bytes - at) & 8) {
            *reinterpret_cast<Two*>(to) = Two{x[0], x[1]};
            x[0] = x[2];
            x[1] = x[3];
            to += 8;
        }
        if ((bytes - at) & 4) {
            *reinterpret_cast<One*>(to) = x[0];
            x[0] = x[1];
            to += 4;
        }
        if (ES == 2 && ((bytes - at) & 2)) *reinterpret_cast<uint16_t*>(to) = uint16_t(x[0]);
    }
}

// Reductions over 16 neighbouring lanes, the same value in all of them: neighbours, pairs, halves of eight, then the two eights.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140, kRotate = 0x120;
template <typename F>
__device__ __forceinline__ void over16(F&& step) {
    step(std::integral_constant<int, kSwap1>());
    step(std::integral_constant<int, kSwap2>());
    step(std::integral_constant<int, kHalfMirror>());
    step(std::integral_constant<int, kMirror>());
}
// The other 15 lanes' values, one rotation at a time.
template <typename F>
__device__ __forceinline__ void rotations(F&& step) {
    step(std::integral_constant<int, kRotate + 1>());
    step(std::integral_constant<int, kRotate + 2>());
    step(std::integral_constant<int, kRotate + 3>());
    step(std::integral_constant<int, kRotate + 4>());
    step(std::integral_constant<int, kRotate + 5>());
    step(std::integral_constant<int, kRotate + 6>());
    step(std::integral_constant<int, kRotate + 7>());
    step(std::integral_constant<int, kRotate + 8>());
    step(std::integral_constant<int, kRotate + 9>());
    step(std::integral_constant<int, kRotate + 10>());
    step(std::integral_constant<int, kRotate + 11>());
    step(std::integral_constant<int, kRotate + 12>());
    step(std::integral_constant<int, kRotate + 13>());
    step(std::integral_constant<int, kRotate + 14>());
    step(std::integral_constant<int, kRotate + 15>());
}
// step(k, control that gives every lane of the 16 lane k's value), k = 0 .. 15.
template <int K = 0, typename F>
__device__ __forceinline__ void broadcasts16(F&& step) {
    step(std::integral_constant<int, K>(), std::integral_constant<int, 0x150 + K>());
    if constexpr (K < 15) broadcasts16<K + 1>(step);
}
__device__ __forceinline__ float max16(float v) {
    over16([&](auto c) { v = fmaxf(v, dpp<decltype(c)::value>(v)); });
    return v;
}
__device__ __forceinline__ int32_t max16(int32_t v) {
    over16([&](auto c) {
        const int32_t o = int32_t(dpp<decltype(c)::value>(uint32_t(v)));
        v = o > v ? o : v;
    });
    return v;
}
__device__ __forceinline__ float sum16(float v) {
    over16([&](auto c) { v += dpp<decltype(c)::value>(v); });
    return v;
}
// Sums and maxima over the wave's 64 lanes, the same value in every lane.
__device__ __forceinline__ float wave_sum(float v) {
    v = sum16(v);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ float wave_max(float v) {
    v = max16(v);
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
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
