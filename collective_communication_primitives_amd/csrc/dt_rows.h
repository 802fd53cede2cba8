// dt_rows.h -- rows held in the registers of one or more waves, as the norms
// hold them: units of 16 bytes, buffer resources, sums over a row's waves.
#pragma once

#include "dt_step_device.h"

namespace dt {
namespace {

// A lane's units of a row: 16 bytes.  VEC: rows start and end on 16-byte
// boundaries; the others are read at their elements' alignment, with a last
// unit that may be partly behind the row's end.
template <int DT>
struct Unit {
    typedef typename Elem<DT>::type T;
    static constexpr int elems = 16 / int(sizeof(T));
    T v[elems];
    __device__ __forceinline__ float get(int e) const { return Elem<DT>::get(v[e]); }
    __device__ __forceinline__ void put(int e, float f) { v[e] = Elem<DT>::put(f); }
};
// A row as a buffer resource: a vector past its end loads zeros and is not
// stored, so the last vectors need no branch.  Row addresses are the same in
// every lane of a wave.
struct Row {
    const char* p;
    rsrc_t r;
    uint32_t bytes;
};
__device__ __forceinline__ Row row_at(const void* base, uint64_t row, uint32_t pitch) {
    const char* p = static_cast<const char*>(base) + row * pitch;
    return Row{p, make_rsrc(p, pitch), pitch};
}
template <int DT, bool VEC, int POL>
__device__ __forceinline__ Unit<DT> load_unit(const Row& row, uint32_t u) {
    Unit<DT> x;
    u32x4 v;
    if constexpr (VEC) v = bload16<POL>(row.r, u * 16);
    else v = load_loose<int(sizeof(typename Unit<DT>::T))>(row.p, u, row.bytes);
    __builtin_memcpy(x.v, &v, 16);
    return x;
}
template <int DT, bool VEC>
__device__ __forceinline__ void store_unit(const Row& row, uint32_t u, const Unit<DT>& x) {
    u32x4 v;
    __builtin_memcpy(&v, x.v, 16);
    if constexpr (VEC) bstore16<kPolNT | kPolDevice>(row.r, u * 16, v);
    else store_loose<int(sizeof(typename Unit<DT>::T))>(const_cast<char*>(row.p), u, row.bytes, v);
}

// Sum over the WPR waves that hold a row; `slot` is one of the workgroup's
// exchange cells, not used again before the next-but-one barrier.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* slot) {
    v = wave_sum(v);
    if constexpr (WPR == 1) return v;
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; w++) s += slot[w];
    return s;
}

template <int WPR>
struct Group {
    static constexpr int waves = WPR > 4 ? WPR : 4;   // waves of a workgroup
    static constexpr int threads = waves * 64;
    static constexpr int rows = WPR == 1 ? waves : 1;  // rows in flight in a workgroup
    static constexpr int lanes = 64 * WPR;             // lanes that share a row
};

}  // namespace
}  // namespace dt
