// dt_stream.h -- few rows against many weights: weights go from memory straight into
// the registers of the matrix instructions, 16 rows by 64 bytes at a time, with the
// few rows as the other operand; a workgroup's waves share the summed index.
// Bound by the weights' bytes, each read once.
#pragma once

#include "dt_matrix.h"

namespace dt {
namespace {

// A lane's 16 bytes of a row.  Those of a weight row are read by no other workgroup,
// but not past the cache for all that: an instruction takes half of each 128-byte
// line, the next one the rest (past it: 544 us instead of 474).
template <int DT, bool VEC>
__device__ __forceinline__ u32x4 lane_at(const char* row, uint32_t at) {
    if constexpr (VEC) return *reinterpret_cast<const u32x4*>(row + at);
    else return *reinterpret_cast<const typename Loose<DT == kBF16 ? 2 : 4>::type*>(row + at);
}
// The same where the row may end inside the 16 bytes or before them.
template <int DT, bool VEC>
__device__ __forceinline__ u32x4 end_at(const char* row, uint32_t at, uint32_t bytes) {
    if constexpr (VEC) return at < bytes ? *reinterpret_cast<const u32x4*>(row + at) : u32x4{0, 0, 0, 0};
    else return read_loose<DT == kBF16 ? 2 : 4>(row, at, bytes);
}

// Four neighbouring lanes load 64 bytes of one row, which the memory unit takes as
// one request (a row per lane as the matrix instructions want it takes four times as
// many: 441 and 289 us for the products of 128 tokens to 4 of 64 experts, 0 and 0
// this way); the registers go to their lanes afterwards: row lane % 16, 16 bytes
// lane / 16.
__device__ __forceinline__ u32x4 to_rows(u32x4 v) {
    const int from = int(((threadIdx.x & 15) * 4 + (threadIdx.x >> 4 & 3)) * 4);
#pragma unroll
    for (int e = 0; e < 4; e++) v[e] = uint32_t(__builtin_amdgcn_ds_bpermute(from, int(v[e])));
    return v;
}

// acc[k][g][e] += sum over the steps of 64 bytes [lo, hi) of weight row 4 (lane / 16)
// + e of the 16 rows w[k] times row lane % 16 of x[part][g], over all parts.  Each
// lane passes the first byte of the row that it loads: w and x of row lane / 4.
// `bytes` and `xbytes`: of a row; the step that it ends in is masked.
//
// Steps are loaded in pairs, whole lines of 128 bytes, P of which are on their way at
// any time: a pair's registers take the load of the P-th pair behind it as soon as
// they are multiplied.  Single steps bring each line to the CU twice (the same
// products 415 and 278 us with four steps on their way, 389 and 239 with two pairs;
// three pairs 414 and 262: fewer waves fit).
//
// fp32: a sum runs over kRunSteps steps of 16 terms at most, as in matrix_walk, and
// these sums are added up apart (8 runs of 48 rows of 4096 to 2048 97 us either way,
// gated 173 instead of 165; one run of 40 rows of 8192 to 4096 82 instead of 90).
//
// A second part, what rounding left of the first, has sums of its own, added where
// the first part's sum is finite: it is zero or of the other sign as it happens, and
// an infinite weight would make NaN of it where the whole value makes an infinity.
template <int DT, bool VEC, int W, int G, int PARTS, int P>
__device__ __forceinline__ void stream_rows(const char* const (&w)[W], const char* const (&x)[PARTS][G], uint32_t lo, uint32_t hi, uint32_t bytes,
                                            uint32_t xbytes, f32x4 (&acc)[W][G]) {
    const uint32_t from = (threadIdx.x & 3) * 16, whole = bytes / kStepBytes, end = hi < whole ? hi : whole;
    static_assert(PARTS == 1 || (PARTS == 2 && DT == kBF16), "fp32 is whole");
    u32x4 a[P][2][W], b[P][2][PARTS][G];
    f32x4 rest[PARTS == 2 ? W : 1][PARTS == 2 ? G : 1];
    if constexpr (PARTS == 2) {
#pragma unroll
        for (int k = 0; k < W; k++)
#pragma unroll
            for (int g = 0; g < G; g++) rest[k][g] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    auto load = [&](int i, uint32_t s) {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int k = 0; k < W; k++) a[i][h][k] = lane_at<DT, VEC>(w[k], (s + h) * kStepBytes + from);
#pragma unroll
        for (int p = 0; p < PARTS; p++)
#pragma unroll
            for (int g = 0; g < G; g++)
#pragma unroll
                for (int h = 0; h < 2; h++) b[i][h][p][g] = lane_at<DT, VEC || PARTS == 2>(x[p][g], (s + h) * kStepBytes + from);
    };
    auto multiply_step = [&](const u32x4 (&fa)[W], const u32x4 (&fb)[PARTS][G]) {
        u32x4 t[PARTS][G];
#pragma unroll
        for (int p = 0; p < PARTS; p++)
#pragma unroll
            for (int g = 0; g < G; g++) t[p][g] = to_rows(fb[p][g]);
#pragma unroll
        for (int k = 0; k < W; k++) {
            const u32x4 f = to_rows(fa[k]);
#pragma unroll
            for (int g = 0; g < G; g++) {
                acc[k][g] = multiply<DT>(f, t[0][g], acc[k][g]);
                if constexpr (PARTS == 2) rest[k][g] = multiply<DT>(f, t[1][g], rest[k][g]);
            }
        }
    };
    auto multiply_pair = [&](int i) {
        multiply_step(a[i][0], b[i][0]);
        multiply_step(a[i][1], b[i][1]);
    };
    constexpr bool RUNS = DT == kF32;
    f32x4 total[RUNS ? W : 1][RUNS ? G : 1];
    if constexpr (RUNS) {
#pragma unroll
        for (int k = 0; k < W; k++)
#pragma unroll
            for (int g = 0; g < G; g++) total[k][g] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    auto run_ends = [&] {
        if constexpr (RUNS) {
#pragma unroll
            for (int k = 0; k < W; k++)
#pragma unroll
                for (int g = 0; g < G; g++) {
                    total[k][g] += acc[k][g];
                    acc[k][g] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
        }
    };
    constexpr uint32_t U = 2 * P;
    static_assert(kRunSteps % U == 0, "a run is whole turns of the loop");
    uint32_t s = lo;
    if (s + U <= end) {
#pragma unroll
        for (int i = 0; i < P; i++) load(i, s + 2 * i);
        for (; s + 2 * U <= end; s += U) {
            if ((s - lo) % kRunSteps == 0) run_ends();
#pragma unroll
            for (int i = 0; i < P; i++) {
                multiply_pair(i);
                load(i, s + U + 2 * i);
            }
        }
        run_ends();   // fewer than 2 U steps are left, and at most one that the row ends in
#pragma unroll
        for (int i = 0; i < P; i++) {
            multiply_pair(i);
            if (s + U + 2 * i + 2 <= end) load(i, s + U + 2 * i);
        }
        s += U;
#pragma unroll
        for (int i = 0; i < P; i++)
            if (s + 2 <= end) {
                multiply_pair(i);
                s += 2;
            }
    }
    for (; s < hi; s++) {   // what is left, the row's end among it
        const uint32_t at = s * kStepBytes + from;
        u32x4 fa[W], fb[PARTS][G];
#pragma unroll
        for (int p = 0; p < PARTS; p++)
#pragma unroll
            for (int g = 0; g < G; g++) fb[p][g] = end_at<DT, VEC || PARTS == 2>(x[p][g], at, xbytes);
#pragma unroll
        for (int k = 0; k < W; k++) fa[k] = end_at<DT, VEC>(w[k], at, bytes);
        multiply_step(fa, fb);
    }
    if constexpr (RUNS) {
#pragma unroll
        for (int k = 0; k < W; k++)
#pragma unroll
            for (int g = 0; g < G; g++) acc[k][g] += total[k][g];
    }
    if constexpr (PARTS == 2) {
#pragma unroll
        for (int k = 0; k < W; k++)
#pragma unroll
            for (int g = 0; g < G; g++)
#pragma unroll
                for (int e = 0; e < 4; e++) acc[k][g][e] += fabsf(acc[k][g][e]) < INFINITY ? rest[k][g][e] : 0.f;
    }
}
// Steps of share `i` of `n`, whole pairs of them (a pair is a line of the weights).
__device__ __forceinline__ void share_steps(uint32_t steps, uint32_t i, uint32_t n, uint32_t& lo, uint32_t& hi) {
    const uint32_t pairs = (steps + 1) / 2, each = pairs / n, more = pairs % n;
    lo = (i * each + (i < more ? i : more)) * 2;
    hi = lo + (each + (i < more ? 1 : 0)) * 2;
    if (lo > steps) lo = steps;
    if (hi > steps) hi = steps;
}

}  // namespace
}  // namespace dt
