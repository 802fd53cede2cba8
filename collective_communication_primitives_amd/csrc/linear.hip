// linear.hip -- matrix products of every rank's rows with bias, activation and
// residual in the epilogue, one weight matrix per run of rows: the experts'
// products between dispatch and combine, or a dense layer (one run).
//
//   z = W_e x + b_e        y = residual + act(z)
//   gated: z = [g; u],     y = residual + act(g) u
//   dz = dy act'(z); gated: dg = dy u act'(g), du = dy act(g)
//   dx = W_e^T dz          dW_e = sum over the run's rows of dz x^T,  db_e = sum of dz
//   relu: max(z, 0)   gelu: z Phi(z), Phi the normal distribution function   silu: z / (1 + exp(-z))
//
// The runs' ends are known on the device only (dt_moe_dispatch leaves them
// there), so a workgroup counts the tiles of all runs itself and walks over its
// share of them.  The host knows the buffers' rows only and takes them as the rows in
// use, evenly among the runs, when it picks a kernel: the results do not depend on
// that, the time does a little (64 runs of 4 to 30 bf16 rows of 4096 to 2 x 1024
// gated, 185 to 227 us in tight buffers, 185 to 212 in buffers 2 to 16 times as long),
// and more where the runs' lengths differ much.
//
// All sums are fp32.  z, y, dx, dW and db are rounded once; dz is rounded to the
// tensors' type before it enters its two products, as the matrix units take it.
//
// Many rows are bound by the matrix units: 52432 bf16 rows of 4096 in 64 runs to 2 x
// 2048 gated, pre kept, 1.87 ms (0.94 PFLOP/s; 8192 rows of 4096 to 11008 with gelu
// 0.74 ms, 1.0), dz 0.25 ms (memory), dx 1.65 (1.07), dweight 1.80 (0.98).  Tiles that
// runs end in are 15% of the work, weights that no neighbour has fetched yet cost 9%,
// pre's stores 7%.  Few rows are bound by the weights' bytes: 16 rows of 4096 in four
// runs to 4096 24 us, 5.6 TB/s.  fp32: 5444 ragged rows of 1001 from 509 backward 17 us
// for dz, 5 for the bias, 67 for dx and 69 for dweight, 80 TFLOP/s in tiles of 64 x 64.
#include "dt_act.h"
#include "dt_stream.h"

namespace dt {
namespace {

constexpr int kThreads = 256;     // workgroups of the kernels without a matrix tile
constexpr uint32_t kMaxRuns = DT_MAX_EXPERTS;

// Run g = rank * runs + run: its rank and its rows of the rank's, cut to the rows that are there.
struct Run {
    uint32_t rank, run, lo, count;
};
__device__ __forceinline__ Run run_at(const LinearArgs& a, uint32_t g) {
    const uint32_t q = g / a.runs, e = g % a.runs, rows = a.rows.start[q + 1] - a.rows.start[q];
    if (rows == 0 || a.offsets[q] == nullptr) return Run{q, e, 0, rows};
    const int32_t lo = a.offsets[q][e], hi = a.offsets[q][e + 1];
    const uint32_t from = lo < 0 ? 0 : uint32_t(lo) < rows ? uint32_t(lo) : rows;
    const uint32_t to = hi < 0 ? 0 : uint32_t(hi) < rows ? uint32_t(hi) : rows;
    return Run{q, e, from, to > from ? to - from : 0};
}
// The same run in every lane of the wave.
__device__ __forceinline__ Run same(const Run& r) {
    return Run{uint32_t(__builtin_amdgcn_readfirstlane(r.rank)), uint32_t(__builtin_amdgcn_readfirstlane(r.run)),
               uint32_t(__builtin_amdgcn_readfirstlane(r.lo)), uint32_t(__builtin_amdgcn_readfirstlane(r.count))};
}

// The runs' tiles of `per` rows, counted by the workgroup itself.
constexpr uint32_t kCachedRuns = 256;
struct Runs {
    uint32_t first[kMaxRuns + 1];                    // tiles of the runs before g; of all runs
    uint32_t lo[kCachedRuns], count[kCachedRuns];    // rows of the first runs
};
__device__ __forceinline__ void count_tiles(const LinearArgs& a, uint32_t per, Runs& t) {
    const uint32_t groups = a.runs * a.nranks;
    for (uint32_t g = threadIdx.x; g < groups; g += blockDim.x) {
        const Run r = run_at(a, g);
        t.first[g] = (r.count + per - 1) / per;
        if (g < kCachedRuns) {
            t.lo[g] = r.lo;
            t.count[g] = r.count;
        }
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        const uint32_t each = (groups + 63) / 64, lo = threadIdx.x * each, hi = lo + each < groups ? lo + each : groups;
        uint32_t sum = 0;
        for (uint32_t g = lo; g < hi; g++) sum += t.first[g];
        uint32_t before = sum;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const uint32_t o = uint32_t(__shfl_up(int(before), m));
            if (int(threadIdx.x) >= m) before += o;
        }
        before -= sum;
        for (uint32_t g = lo; g < hi; g++) {
            const uint32_t n = t.first[g];
            t.first[g] = before;
            before += n;
        }
        if (threadIdx.x == 63) t.first[groups] = before;
    }
    __syncthreads();
}
// Run g in scalar registers.
__device__ __forceinline__ Run run_of(const LinearArgs& a, const Runs& t, uint32_t g) {
    if (g >= kCachedRuns) return same(run_at(a, g));
    return Run{g / a.runs, g % a.runs, uint32_t(__builtin_amdgcn_readfirstlane(t.lo[g])), uint32_t(__builtin_amdgcn_readfirstlane(t.count[g]))};
}
// The run that tile t belongs to.
__device__ __forceinline__ uint32_t run_of_tile(const uint32_t* first, uint32_t groups, uint32_t t) {
    uint32_t lo = 0, hi = groups;  // first[lo] <= t < first[hi]
    while (lo + 1 < hi) {
        const uint32_t mid = (lo + hi) / 2;
        if (uint32_t(__builtin_amdgcn_readfirstlane(first[mid])) <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// A tile of a product: its run, its first feature (or column) m0 and row (or feature) n0.
struct LinearTile {
    Run r;
    uint32_t m0, n0, split;
};
// Of `terms` terms split s has those from part_of(..) * s on, whole steps of KR.
template <uint32_t KR>
__device__ __forceinline__ uint32_t part_of(uint32_t terms, uint32_t splits) {
    return ((terms + KR - 1) / KR + splits - 1) / splits * KR;
}
// The workgroup's tiles of products whose rows are the runs': every gridDim.x-th, run
// by run, so that neighbouring tiles meet the same weights; SPLIT: all of them for
// each split of the summed index.
template <uint32_t BM, uint32_t BN, bool SPLIT>
struct RowTiles {
    const LinearArgs& a;
    const Runs& runs;
    uint32_t mts, all, id;
    __device__ __forceinline__ RowTiles(const LinearArgs& args, Runs& t, uint32_t features)
        : a(args), runs(t), mts((features + BM - 1) / BM), id(blockIdx.x) {
        count_tiles(a, BN, t);
        all = mts * __builtin_amdgcn_readfirstlane(t.first[a.runs * a.nranks]);
    }
    __device__ __forceinline__ bool operator()(LinearTile& t) {
        if (id >= (SPLIT ? all * a.splits : all)) return false;
        const uint32_t split = SPLIT ? __builtin_amdgcn_readfirstlane(id / all) : 0;
        const uint32_t at = share_of(SPLIT ? id - split * all : id, all), g = run_of_tile(runs.first, a.runs * a.nranks, __builtin_amdgcn_readfirstlane(at / mts));
        const uint32_t from = __builtin_amdgcn_readfirstlane(runs.first[g]), to = __builtin_amdgcn_readfirstlane(runs.first[g + 1]);
        uint32_t mt, nt;
        band_tile(at - from * mts, mts, to - from, mt, nt);
        id += gridDim.x;
        t = LinearTile{run_of(a, runs, g), mt * BM, nt * BN, split};
        return true;
    }
};
// The same for the runs' weights: run by run, so that a run's rows are read while they are near.
template <uint32_t BM, uint32_t BN, bool SPLIT>
struct WeightTiles {
    const LinearArgs& a;
    const Runs& runs;
    uint32_t mts, nts;
    uint64_t id;
    __device__ __forceinline__ WeightTiles(const LinearArgs& args, Runs& t, uint32_t cols, uint32_t features)
        : a(args), runs(t), mts((cols + BM - 1) / BM), nts((features + BN - 1) / BN), id(blockIdx.x) {
        count_tiles(a, BN, t);
    }
    __device__ __forceinline__ bool operator()(LinearTile& t) {
        const uint32_t each = mts * nts, groups = a.runs * a.nranks;
        if (id >= uint64_t(each) * groups * (SPLIT ? a.splits : 1)) return false;
        uint32_t g = __builtin_amdgcn_readfirstlane(uint32_t(id / each)), split = 0;
        if constexpr (SPLIT) {
            split = g / groups;
            g -= split * groups;
        }
        uint32_t mt, nt;
        tile_of(__builtin_amdgcn_readfirstlane(uint32_t(id % each)), mts, nts, mt, nt);
        id += gridDim.x;
        t = LinearTile{run_of(a, runs, g), mt * BM, nt * BN, split};
        return true;
    }
};

// --------------------------------------------------------------- operands --
// A gated product's tile of weight rows: 16 rows of the gate and the 16 of the
// linear part that they meet, in turn, so that a lane has both of a feature.
template <bool TAIL>
struct GatedOperand : RowOperand<TAIL> {
    uint32_t half;   // bytes between a gate row and its linear row
    __device__ __forceinline__ uint32_t group_at(uint32_t group) const { return (group >> 1) * 16 * this->pitch + (group & 1) * half; }
};

// Operands whose rows start at any element: read at that alignment into
// registers and put into LDS in the order that the direct loads leave there.
struct LooseRows {
    const char* p;      // the tile's first row
    uint32_t rows, pitch;
    uint32_t half;      // gated: rows between a gate row and its linear row, otherwise 0
    template <int ES, int R>
    __device__ __forceinline__ u32x4 chunk(uint32_t group, uint32_t step) const {
        const uint32_t lane = threadIdx.x & 63, sub = lane >> 2;
        const uint32_t row = half != 0 ? (group >> 1) * 16 + sub : group * 16 + sub;
        if (row >= rows) return u32x4{0, 0, 0, 0};
        return read_loose<ES>(p + uint64_t(row + (group & 1) * half) * pitch, step * kStepBytes + ((lane & 3) ^ row_turn(sub)) * 16, pitch);
    }
};
struct LooseCols {
    const char* p;      // row 0 at the tile's first column
    uint32_t rows, pitch, bytes;   // bytes: of a row from the tile's first column on
    template <int ES, int R>
    __device__ __forceinline__ u32x4 chunk(uint32_t group, uint32_t step) const {
        typedef ColTile<ES == 2 ? kBF16 : kF32, R> C;
        constexpr uint32_t slots = C::row_bytes / 16, per_unit = C::unit_bytes / 16;
        const uint32_t lane = threadIdx.x & 63, k = group * C::per_load + lane / slots, slot = lane % slots, row = step * C::KR + k;
        if (row >= rows) return u32x4{0, 0, 0, 0};
        return read_loose<ES>(p + uint64_t(row) * pitch, ((slot / per_unit) ^ C::f(k)) * C::unit_bytes + slot % per_unit * 16, bytes);
    }
};

// matrix_tile for such operands: two stages of LDS, the next step's bytes on
// their way to registers while one is multiplied.
// Returns LDS of the wave's own, which the next tile may use again.
template <int DT, typename S, int MA, int MB, typename OA, typename OB>
__device__ __forceinline__ u32x4* loose_tile(const OA& A, const OB& B, uint32_t steps, f32x4 (&acc)[S::MI][S::NI]) {
    constexpr int ES = DT == kBF16 ? 2 : 4;
    __shared__ u32x4 stage[2][S::stage];
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < S::MI; i++)
#pragma unroll
        for (int j = 0; j < S::NI; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 ca[S::loads_a], cb[S::loads_b];
    auto read = [&](uint32_t step) {
#pragma unroll
        for (int i = 0; i < S::loads_a; i++) ca[i] = A.template chunk<ES, S::BM>(wave * S::loads_a + i, step);
#pragma unroll
        for (int i = 0; i < S::loads_b; i++) cb[i] = B.template chunk<ES, S::BN>(wave * S::loads_b + i, step);
    };
    const uint32_t wm = (wave % S::GM) * S::WM, wn = (wave / S::GM) * S::WN;
    const uint32_t ra = fragment_place<DT, MA, S::BM>(wm, lane), rb = fragment_place<DT, MB, S::BN>(wn, lane);
    if (steps > 0) read(0);
    __syncthreads();  // the waves have left the room of the tile before
    for (uint32_t step = 0; step < steps; step++) {
        u32x4* to = stage[step & 1];
#pragma unroll
        for (int i = 0; i < S::loads_a; i++) to[(wave * S::loads_a + i) * 64 + lane] = ca[i];
#pragma unroll
        for (int i = 0; i < S::loads_b; i++) to[S::BM * kChunks + (wave * S::loads_b + i) * 64 + lane] = cb[i];
        // The other stage was read before this barrier's predecessor by every wave, or is read behind it: it is
        // written again behind the next one only.
        __syncthreads();
        if (step + 1 < steps) read(step + 1);
        u32x4 fa, fb[S::NI];
#pragma unroll
        for (int j = 0; j < S::NI; j++) fb[j] = fragment<DT, MB, S::BN>(to + S::BM * kChunks, rb, j);
#pragma unroll
        for (int i = 0; i < S::MI; i++) {
            fa = fragment<DT, MA, S::BM>(to, ra, i);
#pragma unroll
            for (int j = 0; j < S::NI; j++) acc[i][j] = multiply<DT>(fa, fb[j], acc[i][j]);
        }
    }
    __syncthreads();
    return &stage[0][0] + wave * (S::stage / S::waves);
}

// Four neighbouring values at any element, `left` of them before the row's end.
template <int DT>
struct Four;
template <>
struct Four<kBF16> {
    typedef uint32_t type __attribute__((ext_vector_type(2), aligned(2)));
};
template <>
struct Four<kF32> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4)));
};
template <int DT>
__device__ __forceinline__ f32x4 load_four(const typename Elem<DT>::type* p, uint32_t left) {
    typedef typename Elem<DT>::type T;
    T t[4];
    if (left >= 4) {
        const typename Four<DT>::type v = *reinterpret_cast<const typename Four<DT>::type*>(p);
        __builtin_memcpy(t, &v, sizeof t);
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++) t[e] = uint32_t(e) < left ? p[e] : T(0);
    }
    return f32x4{Elem<DT>::get(t[0]), Elem<DT>::get(t[1]), Elem<DT>::get(t[2]), Elem<DT>::get(t[3])};
}
template <int DT>
__device__ __forceinline__ void store_four(typename Elem<DT>::type* p, f32x4 v, uint32_t left) {
    typedef typename Elem<DT>::type T;
    T t[4];
    store_quad<DT>(t, v, true);
    if (left >= 4) {
        typename Four<DT>::type o;
        __builtin_memcpy(&o, t, sizeof t);
        *reinterpret_cast<typename Four<DT>::type*>(p) = o;
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (uint32_t(e) < left) p[e] = t[e];
    }
}

// ---------------------------------------------------------------- forward --
// 16 bytes of a row at element m, `left` elements before the row's end, as floats.
template <int DT, int E>
__device__ __forceinline__ void add_some(float (&v)[E], const typename Elem<DT>::type* p, bool vec, uint32_t left) {
    typedef typename Elem<DT>::type T;
    T t[E];
    if (vec) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(p);
        __builtin_memcpy(t, &x, 16);
    } else {
#pragma unroll
        for (int e = 0; e < E; e++) t[e] = uint32_t(e) < left ? p[e] : T(0);
    }
#pragma unroll
    for (int e = 0; e < E; e++) v[e] += Elem<DT>::get(t[e]);
}
template <int DT, int E>
__device__ __forceinline__ void store_some(typename Elem<DT>::type* p, const float (&v)[E], bool vec, uint32_t left) {
    typedef typename Elem<DT>::type T;
    T t[E];
#pragma unroll
    for (int e = 0; e < E; e++) t[e] = Elem<DT>::put(v[e]);
    if (vec) {
        u32x4 x;
        __builtin_memcpy(&x, t, 16);
        *reinterpret_cast<u32x4*>(p) = x;
    } else {
#pragma unroll
        for (int e = 0; e < E; e++)
            if (uint32_t(e) < left) p[e] = t[e];
    }
}

// Bias, activation and residual of a tile.  The sums go through the wave's room in
// LDS, 16 rows of up to 64 features at a time, so that a lane has 16 bytes of
// neighbouring features of y, and whole lines are read and written.  One copy of
// the arithmetic for all of them: unrolled over the tile it did not fit the
// registers.
template <int DT, typename S, bool GATED>
__device__ __forceinline__ void epilogue(const LinearArgs& a, const LinearTile& t, const f32x4 (&acc)[S::MI][S::NI], u32x4* room) {
    typedef typename Elem<DT>::type T;
    constexpr int E = 16 / int(sizeof(T)), step = GATED ? 2 : 1;
    constexpr int F = S::WM < 64 ? S::WM : 64, passes = S::WM / F, chunks = F / 4;   // features of acc in a pass
    constexpr uint32_t per_row = F / step / E, all = 16 * per_row;
    const uint32_t lane = fresh_lane(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t nleft = t.r.count - t.n0, wide = step * a.outs;
    const uint64_t row0 = t.r.lo + t.n0;
    const bool vec = a.vecs;
    const T* bias = a.bias[t.r.rank] != nullptr ? static_cast<const T*>(a.bias[t.r.rank]) + uint64_t(t.r.run) * wide : nullptr;
    const T* residual = static_cast<const T*>(a.residual[t.r.rank]);
    T* pre = static_cast<T*>(a.pre[t.r.rank]);
    T* out = static_cast<T*>(a.y[t.r.rank]);
    // 16 bytes (four sums) c of row n of the room
    auto place = [&](uint32_t n, uint32_t c) { return n * chunks + (c ^ (n & (chunks - 1))); };
#pragma unroll 1
    for (int pass = 0; pass < S::NI * passes; pass++) {
        const int j = pass / passes, h = pass % passes;
#pragma unroll
        for (int jj = 0; jj < S::NI; jj++)
#pragma unroll
            for (int hh = 0; hh < passes; hh++)
                if (j == jj && h == hh) {
#pragma unroll
                    for (int q = 0; q < F / 16; q++) room[place(lane & 15, 4 * q + (lane >> 4))] = __builtin_bit_cast(u32x4, acc[hh * (F / 16) + q][jj]);
                }
#pragma unroll 1
        for (uint32_t i = lane; i < all; i += 64) {
            const uint32_t row = i / per_row, f = i % per_row * E;
            const uint32_t n = (wave / S::GM) * S::WN + j * 16 + row, m = t.m0 + ((wave % S::GM) * S::WM + h * F) / step + f;
            float z[E], u[E];
            // gated: 16 features' gates and their 16 linear parts lie in turn
            const uint32_t c = GATED ? (f / 16) * 8 + f % 16 / 4 : f / 4;
#pragma unroll
            for (int k = 0; k < E / 4; k++) {
                const f32x4 v = __builtin_bit_cast(f32x4, room[place(row, c + k)]);
                const f32x4 w = GATED ? __builtin_bit_cast(f32x4, room[place(row, c + 4 + k)]) : v;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    z[4 * k + e] = v[e];
                    u[4 * k + e] = w[e];
                }
            }
            if (n >= nleft || m >= a.outs) continue;
            const uint32_t left = a.outs - m;
            if (bias != nullptr) {
                add_some<DT, E>(z, bias + m, vec, left);
                if (GATED) add_some<DT, E>(u, bias + a.outs + m, vec, left);
            }
            const uint64_t at = row0 + n;
            if (pre != nullptr) {
                store_some<DT, E>(pre + at * wide + m, z, vec, left);
                if (GATED) store_some<DT, E>(pre + at * wide + a.outs + m, u, vec, left);
            }
            if (a.act == DT_ACT_GELU) {
#pragma unroll
                for (int e = 0; e < E; e++) z[e] = act(z[e], DT_ACT_GELU);
            } else if (a.act == DT_ACT_SILU) {
#pragma unroll
                for (int e = 0; e < E; e++) z[e] = act(z[e], DT_ACT_SILU);
            } else if (a.act == DT_ACT_RELU) {
#pragma unroll
                for (int e = 0; e < E; e++) z[e] = act(z[e], DT_ACT_RELU);
            }
            if (GATED) {
#pragma unroll
                for (int e = 0; e < E; e++) z[e] *= u[e];
            }
            if (residual != nullptr) add_some<DT, E>(z, residual + at * a.outs + m, vec, left);
            store_some<DT, E>(out + at * a.outs + m, z, vec, left);
        }
    }
}

// PATH: rows on 16-byte boundaries, on 4-byte boundaries, or on any.
enum { kWhole = 0, kTail = 1, kLoose = 2 };

template <int DT, typename S, int PATH, bool GATED>
__global__ __launch_bounds__(S::threads, 2) void k_linear(LinearArgs a) {
    typedef typename Elem<DT>::type T;
    constexpr uint32_t BM = GATED ? S::BM / 2 : S::BM;   // features of a tile
    __shared__ Runs runs;
    RowTiles<BM, S::BN, false> tiles(a, runs, a.outs);
    const uint32_t pitch = a.cols * uint32_t(sizeof(T)), steps = (pitch + kStepBytes - 1) / kStepBytes;
    auto weight_of = [&](const LinearTile& t) {
        return static_cast<const char*>(a.weight[t.r.rank]) + (uint64_t(t.r.run) * (GATED ? 2 : 1) * a.outs + t.m0) * pitch;
    };
    auto x_of = [&](const LinearTile& t) { return static_cast<const char*>(a.x[t.r.rank]) + uint64_t(t.r.lo + t.n0) * pitch; };
    auto features_of = [&](const LinearTile& t) { return a.outs - t.m0 < BM ? a.outs - t.m0 : BM; };
    auto rows_of = [&](const LinearTile& t) { return t.r.count - t.n0 < uint32_t(S::BN) ? t.r.count - t.n0 : uint32_t(S::BN); };
    auto done = [&](const LinearTile& t, f32x4 (&acc)[S::MI][S::NI], u32x4* room) { epilogue<DT, S, GATED>(a, t, acc, room); };
    if constexpr (PATH == kLoose) {
        for (LinearTile t; tiles(t);) {
            f32x4 acc[S::MI][S::NI];
            u32x4* room = loose_tile<DT, S, kRows, kRows>(LooseRows{weight_of(t), features_of(t), pitch, GATED ? a.outs : 0},
                                                          LooseRows{x_of(t), rows_of(t), pitch, 0}, steps, acc);
            done(t, acc, room);
        }
    } else {
        constexpr bool TAIL = PATH == kTail;
        typedef typename std::conditional<GATED, GatedOperand<TAIL>, RowOperand<TAIL>>::type OA;
        typedef RowOperand<TAIL> OB;
        const uint32_t whole = (pitch + 15) / 16 * 16;
        matrix_walk<DT, S, kRows, kRows, OA, OB, LinearTile>(tiles, [&](const LinearTile& t, OA& A, OB& B) {
            static_cast<RowOperand<TAIL>&>(A) = RowOperand<TAIL>{weight_of(t), (GATED ? a.outs : 0) + features_of(t), pitch, whole, pitch};
            if constexpr (GATED) A.half = a.outs * pitch;
            B = OB{x_of(t), rows_of(t), pitch, whole, pitch};
            return steps;
        }, rows_of, done);
    }
}

// Few rows to a run: 16 features of one run to a workgroup, whose NW waves share the
// summed index; weights go past LDS, read once for up to 16 GM rows.
template <int DT, bool VEC, bool GATED, int NW, int G>
__device__ __forceinline__ void few_rows(const LinearArgs& a, const Run& r, uint32_t base, f32x4 (*sums)[64]) {
    typedef typename Elem<DT>::type T;
    constexpr int W = GATED ? 2 : 1, P = G > 1 ? 1 : 2;
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t pitch = a.cols * uint32_t(sizeof(T)), m0 = blockIdx.x * 16, wide = W * a.outs;
    // the rows that the lane loads; behind the last one it is repeated
    const uint32_t m = m0 + (lane >> 2) < a.outs ? m0 + (lane >> 2) : a.outs - 1;
    const char *w[W], *x[1][G];
#pragma unroll
    for (int k = 0; k < W; k++) w[k] = static_cast<const char*>(a.weight[r.rank]) + (uint64_t(r.run) * wide + k * a.outs + m) * pitch;
#pragma unroll
    for (int g = 0; g < G; g++) {
        const uint32_t n = base + g * 16 + (lane >> 2);
        x[0][g] = static_cast<const char*>(a.x[r.rank]) + (uint64_t(r.lo) + (n < r.count ? n : r.count - 1)) * pitch;
    }
    f32x4 acc[W][G];
#pragma unroll
    for (int k = 0; k < W; k++)
#pragma unroll
        for (int g = 0; g < G; g++) acc[k][g] = f32x4{0.f, 0.f, 0.f, 0.f};
    uint32_t lo, hi;
    share_steps((pitch + kStepBytes - 1) / kStepBytes, wave, NW, lo, hi);
    stream_rows<DT, VEC, W, G, 1, P>(w, x, lo, hi, pitch, pitch, acc);
#pragma unroll
    for (int k = 0; k < W; k++)
#pragma unroll
        for (int g = 0; g < G; g++) sums[(wave * G + g) * W + k][lane] = acc[k][g];
    __syncthreads();
    // thread: 16 rows threadIdx.x / 64, the lane's four features of its row
    const uint32_t g = threadIdx.x >> 6, n = base + g * 16 + (lane & 15), f = m0 + (lane >> 4) * 4;
    if (g < uint32_t(G) && n < r.count && f < a.outs) {
        f32x4 z = {0.f, 0.f, 0.f, 0.f}, u = z;
#pragma unroll
        for (uint32_t k = 0; k < NW; k++) {
            z += sums[(k * G + g) * W][lane];
            if (GATED) u += sums[(k * G + g) * W + W - 1][lane];
        }
        const uint32_t left = a.outs - f;
        const uint64_t row = uint64_t(r.lo) + n;
        if (a.bias[r.rank] != nullptr) {
            const T* b = static_cast<const T*>(a.bias[r.rank]) + uint64_t(r.run) * wide + f;
            z += load_four<DT>(b, left);
            if (GATED) u += load_four<DT>(b + a.outs, left);
        }
        if (a.pre[r.rank] != nullptr) {
            T* to = static_cast<T*>(a.pre[r.rank]) + row * wide + f;
            store_four<DT>(to, z, left);
            if (GATED) store_four<DT>(to + a.outs, u, left);
        }
        f32x4 y;
#pragma unroll
        for (int e = 0; e < 4; e++) y[e] = act(z[e], a.act) * (GATED ? u[e] : 1.f);
        if (a.residual[r.rank] != nullptr) y += load_four<DT>(static_cast<const T*>(a.residual[r.rank]) + row * a.outs + f, left);
        store_four<DT>(static_cast<T*>(a.y[r.rank]) + row * a.outs + f, y, left);
    }
    __syncthreads();  // the next rows' sums
}
template <int DT, bool VEC, bool GATED, int NW, int GM>
__global__ __launch_bounds__(NW * 64) void k_linear_few(LinearArgs a) {
    __shared__ f32x4 sums[NW * GM * (GATED ? 2 : 1)][64];
    const Run r = same(run_at(a, blockIdx.y));
    uint32_t base = 0;
    if constexpr (GM > 1)
        for (; base < r.count && r.count - base > 16; base += 16 * GM) few_rows<DT, VEC, GATED, NW, GM>(a, r, base, sums);
    for (; base < r.count; base += 16) few_rows<DT, VEC, GATED, NW, 1>(a, r, base, sums);
}

// --------------------------------------------------------------- backward --
// dz of the runs' rows, dz_rows of them and 1024 columns to a workgroup, and its
// columns' sums over those rows.  A thread has four neighbouring columns, and four
// rows' loads go out together.  Bound by memory: 52432 rows of 2048 gated, bf16, 236 us, 4.5 TB/s.
template <int DT, bool GATED>
__global__ __launch_bounds__(kThreads) void k_linear_dz(LinearArgs a) {
    typedef typename Elem<DT>::type T;
    __shared__ Runs runs;
    count_tiles(a, a.dz_rows, runs);
    const uint32_t groups = a.runs * a.nranks, m = (blockIdx.x * kThreads + threadIdx.x) * 4;
    // offsets that decrease, which are not allowed, could make the runs longer than all rows
    const uint32_t tiles = runs.first[groups] < a.dz_tiles ? runs.first[groups] : a.dz_tiles;
    const uint32_t wide = GATED ? 2 * a.outs : a.outs;
    const uint64_t ldz = a.zpitch / sizeof(T);
    if (m >= a.outs) return;
    const uint32_t left = a.outs - m;
    for (uint32_t t = blockIdx.y; t < tiles; t += gridDim.y) {
        const uint32_t g = run_of_tile(runs.first, groups, t);
        const Run r = run_of(a, runs, g);
        const uint32_t n0 = (t - runs.first[g]) * a.dz_rows, rows = r.count - n0 < a.dz_rows ? r.count - n0 : a.dz_rows;
        const uint64_t row0 = r.lo + n0;
        const T* dy = static_cast<const T*>(a.dy[r.rank]) + row0 * a.outs + m;
        const T* pre = a.need_dz ? static_cast<const T*>(a.saved[r.rank]) + row0 * wide + m : nullptr;
        T* dz = a.need_dz ? reinterpret_cast<T*>(a.dz) + (a.rows.start[r.rank] + row0) * ldz : nullptr;
        f32x4 sum = {0.f, 0.f, 0.f, 0.f}, sumu = sum;
        for (uint32_t n = 0; n < rows; n += 4) {
            f32x4 d[4], z[4], u[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint32_t row = n + i < rows ? n + i : rows - 1;   // the last row again, and nothing of it is used
                d[i] = load_four<DT>(dy + uint64_t(row) * a.outs, left);
                if (a.need_dz) z[i] = load_four<DT>(pre + uint64_t(row) * wide, left);
                if (GATED) u[i] = load_four<DT>(pre + uint64_t(row) * wide + a.outs, left);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if (n + i >= rows) break;
                f32x4 du = {0.f, 0.f, 0.f, 0.f};
                if (a.need_dz) {
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        float value, slope;
                        act_and_slope(z[i][e], a.act, value, slope);
                        if (GATED) du[e] = d[i][e] * value;
                        d[i][e] *= GATED ? u[i][e] * slope : slope;
                    }
                    T* to = dz + (n + i) * ldz;
                    store_four<DT>(to + m, d[i], left);
                    if (GATED) store_four<DT>(to + a.outs + m, du, left);
                    if (left <= 4)  // what lies between the row's end and its pitch
                        for (uint64_t c = wide; c < ldz; c++) to[c] = T(0);
                }
                sum += d[i];
                if (GATED) sumu += du;
            }
        }
        if (a.partial != nullptr) {
            float* to = a.partial + uint64_t(t) * wide + m;
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (uint32_t(e) < left) {
                    to[e] = sum[e];
                    if (GATED) to[a.outs + e] = sumu[e];
                }
        }
    }
}

// db of run blockIdx.y: its tiles' sums in a fixed order, 64 columns to a workgroup,
// of whose 16 waves each takes every 16th tile.
template <int DT>
__global__ __launch_bounds__(1024) void k_linear_dbias(LinearArgs a) {
    typedef typename Elem<DT>::type T;
    __shared__ Runs runs;
    __shared__ float sums[16][64];
    count_tiles(a, a.dz_rows, runs);
    const uint32_t wide = (a.gated ? 2 : 1) * a.outs, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane, g = blockIdx.y;
    const uint32_t end = runs.first[g + 1] < a.dz_tiles ? runs.first[g + 1] : a.dz_tiles;
    float s = 0.f;
    if (c < wide)
        for (uint32_t t = runs.first[g] + wave; t < end; t += 16 * 4) {
            float v[4];  // four tiles' loads go out before the first is added
#pragma unroll
            for (int k = 0; k < 4; k++) v[k] = t + 16 * k < end ? a.partial[uint64_t(t + 16 * k) * wide + c] : 0.f;
#pragma unroll
            for (int k = 0; k < 4; k++) s += v[k];
        }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c >= wide) return;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 16; k++) s += sums[k][lane];
    static_cast<T*>(a.dbias[g / a.runs])[uint64_t(g % a.runs) * wide + c] = Elem<DT>::put(s);
}

// Rows of dz: in the workspace, or dy itself where dz is dy.
template <typename T>
__device__ __forceinline__ const char* dz_row(const LinearArgs& a, const Run& r, uint32_t row) {
    return a.need_dz ? a.dz + (uint64_t(a.rows.start[r.rank]) + r.lo + row) * a.zpitch
                     : static_cast<const char*>(a.dy[r.rank]) + uint64_t(r.lo + row) * a.zpitch;
}

// A tile's sums to rows of `cols` elements from `out` on, row n0, column m0.
template <int DT, typename S, bool ROOM>
__device__ __forceinline__ void store_tile(const LinearArgs& a, typename Elem<DT>::type* out, uint32_t m0, uint32_t n0, uint32_t nleft,
                                           const f32x4 (&acc)[S::MI][S::NI], u32x4* room) {
    const uint32_t lane = fresh_lane(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t mw = m0 + (wave % S::GM) * S::WM, nw = (wave / S::GM) * S::WN, cols = a.cols;
#pragma unroll
    for (int j = 0; j < S::NI; j++) {
        if (ROOM && a.col_vecs) {
            f32x4 v[S::MI];
#pragma unroll
            for (int i = 0; i < S::MI; i++) v[i] = acc[i][j];
            turn_rows<DT, S::WM>(room, v, [&](uint32_t row, uint32_t m, u32x4 x) {
                const uint32_t n = nw + j * 16 + row;
                if (n < nleft && mw + m < cols) *reinterpret_cast<u32x4*>(out + uint64_t(n0 + n) * cols + mw + m) = x;
            });
            continue;
        }
        const uint32_t n = nw + j * 16 + (lane & 15);
        if (n >= nleft) continue;
#pragma unroll
        for (int i = 0; i < S::MI; i++) {
            const uint32_t m = mw + i * 16 + (lane >> 4) * 4;
            if (m >= cols) continue;
            store_four<DT>(out + uint64_t(n0 + n) * cols + m, acc[i][j], cols - m);
        }
    }
}

// dx[t][k] = sum over the features of dz[t][m] W[m][k].  SPLIT: the sum over one
// part of the features, left for k_linear_join.
template <int DT, typename S, int PATH, bool SPLIT>
__global__ __launch_bounds__(S::threads, 2) void k_linear_dx(LinearArgs a) {
    typedef typename Elem<DT>::type T;
    constexpr uint32_t es = sizeof(T), KR = kStepBytes / es;
    static_assert(!SPLIT || PATH != kLoose, "");
    __shared__ Runs runs;
    RowTiles<S::BM, S::BN, SPLIT> tiles(a, runs, a.cols);
    const uint32_t wide = (a.gated ? 2 : 1) * a.outs, pitch = a.cols * es, part = SPLIT ? part_of<KR>(wide, a.splits) : wide;
    auto weight_of = [&](const LinearTile& t) {
        return static_cast<const char*>(a.weight[t.r.rank]) + uint64_t(t.r.run) * wide * pitch + t.m0 * es;
    };
    auto rows_of = [&](const LinearTile& t) { return t.r.count - t.n0 < uint32_t(S::BN) ? t.r.count - t.n0 : uint32_t(S::BN); };
    auto done = [&](const LinearTile& t, f32x4 (&acc)[S::MI][S::NI], u32x4* room) {
        if constexpr (SPLIT)
            store_tile<kF32, S, true>(a, a.sums + ((uint64_t(t.split) * a.rows.start[a.nranks] + a.rows.start[t.r.rank]) + t.r.lo) * a.cols,
                                      t.m0, t.n0, t.r.count - t.n0, acc, room);
        else store_tile<DT, S, PATH != kLoose>(a, static_cast<T*>(a.dx[t.r.rank]) + uint64_t(t.r.lo) * a.cols, t.m0, t.n0, t.r.count - t.n0, acc, room);
    };
    if constexpr (PATH == kLoose) {
        for (LinearTile t; tiles(t);) {
            f32x4 acc[S::MI][S::NI];
            loose_tile<DT, S, kCols, kRows>(LooseCols{weight_of(t), wide, pitch, pitch - t.m0 * es}, LooseRows{dz_row<T>(a, t.r, t.n0), rows_of(t), a.zpitch, 0},
                                            (wide + KR - 1) / KR, acc);
            done(t, acc, nullptr);
        }
    } else {
        typedef ColOperand<KR, 1> OA;
        typedef RowOperand<PATH == kTail> OB;
        matrix_walk<DT, S, kCols, kRows, OA, OB, LinearTile>(tiles, [&](const LinearTile& t, OA& A, OB& B) {
            const uint32_t from = t.split * part, terms = from >= wide ? 0 : wide - from < part ? wide - from : part;
            A = OA{weight_of(t) + uint64_t(from) * pitch, terms, pitch, t.m0 * es, 0};
            B = OB{dz_row<T>(a, t.r, t.n0) + from * es, rows_of(t), a.zpitch, (a.zpitch + 15) / 16 * 16 - from * es, terms * es, from * es};
            return (terms + KR - 1) / KR;
        }, rows_of, done);
    }
}

// dW[m][k] = sum over the run's rows of dz[t][m] x[t][k]; zeros for a run without
// rows.  SPLIT: the sum over one part of the rows, left for k_linear_join.
template <int DT, typename S, int PATH, bool SPLIT>
__global__ __launch_bounds__(S::threads, 2) void k_linear_dweight(LinearArgs a) {
    typedef typename Elem<DT>::type T;
    constexpr uint32_t es = sizeof(T), KR = kStepBytes / es;
    static_assert(!SPLIT || PATH != kLoose, "");
    __shared__ Runs runs;
    const uint32_t wide = (a.gated ? 2 : 1) * a.outs, pitch = a.cols * es;
    WeightTiles<S::BM, S::BN, SPLIT> tiles(a, runs, a.cols, wide);
    auto x_of = [&](const LinearTile& t, uint32_t from) { return static_cast<const char*>(a.x[t.r.rank]) + uint64_t(t.r.lo + from) * pitch + t.m0 * es; };
    auto dz_of = [&](const LinearTile& t, uint32_t from) { return dz_row<T>(a, t.r, from) + t.n0 * es; };
    auto done = [&](const LinearTile& t, f32x4 (&acc)[S::MI][S::NI], u32x4* room) {
        if constexpr (SPLIT)
            store_tile<kF32, S, true>(a, a.sums + ((uint64_t(t.split) * a.nranks + t.r.rank) * a.runs + t.r.run) * wide * a.cols, t.m0, t.n0, wide - t.n0,
                                      acc, room);
        else store_tile<DT, S, PATH != kLoose>(a, static_cast<T*>(a.dweight[t.r.rank]) + uint64_t(t.r.run) * wide * a.cols, t.m0, t.n0, wide - t.n0, acc, room);
    };
    if constexpr (PATH == kLoose) {
        for (LinearTile t; tiles(t);) {
            f32x4 acc[S::MI][S::NI];
            loose_tile<DT, S, kCols, kCols>(LooseCols{x_of(t, 0), t.r.count, pitch, pitch - t.m0 * es},
                                            LooseCols{dz_of(t, 0), t.r.count, a.zpitch, (wide - t.n0) * es}, (t.r.count + KR - 1) / KR, acc);
            done(t, acc, nullptr);
        }
    } else {
        typedef ColOperand<KR, 1> OP;
        matrix_walk<DT, S, kCols, kCols, OP, OP, LinearTile>(tiles, [&](const LinearTile& t, OP& A, OP& B) {
            const uint32_t part = SPLIT ? part_of<KR>(t.r.count, a.splits) : t.r.count, from = SPLIT && t.split * part < t.r.count ? t.split * part : 0;
            const uint32_t terms = !SPLIT || t.split == 0 || from > 0 ? (t.r.count - from < part ? t.r.count - from : part) : 0;
            A = OP{x_of(t, from), terms, pitch, t.m0 * es, 0};
            B = OP{dz_of(t, from), terms, a.zpitch, t.n0 * es, 0};
            return (terms + KR - 1) / KR;
        }, [&](const LinearTile& t) { return wide - t.n0; }, done);
    }
}

// dx's rows, or dweight, from the sums over the parts, in their order: a run's
// values lie side by side in both.
template <int DT, bool WEIGHT>
__global__ __launch_bounds__(kThreads) void k_linear_join(LinearArgs a) {
    typedef typename Elem<DT>::type T;
    const Run r = same(run_at(a, blockIdx.y));
    const uint32_t wide = (a.gated ? 2 : 1) * a.outs;
    const uint64_t count = uint64_t(WEIGHT ? wide : r.count) * a.cols, apart = uint64_t(WEIGHT ? a.nranks * a.runs * wide : a.rows.start[a.nranks]) * a.cols;
    const float* from = a.sums + (WEIGHT ? uint64_t(blockIdx.y) * wide : uint64_t(a.rows.start[r.rank]) + r.lo) * a.cols;
    T* to = WEIGHT ? static_cast<T*>(a.dweight[r.rank]) + uint64_t(r.run) * wide * a.cols : static_cast<T*>(a.dx[r.rank]) + uint64_t(r.lo) * a.cols;
    for (uint64_t i = uint64_t(blockIdx.x) * kThreads + threadIdx.x; i < count; i += uint64_t(gridDim.x) * kThreads) {
        float s = 0.f;
        uint32_t k = 0;
        for (; k + 8 <= a.splits; k += 8) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = from[(k + j) * apart + i];
#pragma unroll
            for (int j = 0; j < 8; j++) s += v[j];
        }
        for (; k < a.splits; k++) s += from[k * apart + i];
        to[i] = Elem<DT>::put(s);
    }
}

// -------------------------------------------------------------------- host --
uint64_t ceil_div(uint64_t n, uint64_t by) { return (n + by - 1) / by; }

typedef Shape<256, 256, 2, 4> Wide;
typedef Shape<128, 128, 2, 2> Square;
typedef Shape<64, 64, 2, 2> Small;
typedef Shape<64, 16, 1, 1> Tiny;
enum Tile { kWide, kSquare, kSmall, kTiny };
constexpr uint32_t kTileM[] = {256, 128, 64, 64}, kTileN[] = {256, 128, 64, 16};

// The tile for products of m features with runs of `mean` rows each.
Tile pick_tile(int dtype, uint64_t m, uint64_t mean, uint64_t groups, int path, bool tiny) {
    if (tiny && mean <= 16) return kTiny;
    auto tiles = [&](uint64_t by) { return ceil_div(m, by) * ceil_div(mean, by) * groups; };
    if (path == kLoose || dtype == kF32) return tiles(128) >= 1024 ? kSquare : kSmall;
    if (mean > 128 && tiles(256) >= 224) return kWide;
    return mean > 32 && tiles(128) >= 192 ? kSquare : kSmall;
}
// launch(Shape) with the shape of `t`; TINY: where pick_tile may say so.
template <int DT, int PATH, bool TINY, typename F>
void with_tile(Tile t, F&& launch) {
    if constexpr (TINY) {
        if (t == kTiny) return launch(Tiny());
    }
    if constexpr (DT == kBF16 && PATH != kLoose) {
        if (t == kWide) return launch(Wide());
    }
    if (t == kSquare) launch(Square());
    else launch(Small());
}
// launch(path).  fp32 rows always start on 4-byte boundaries.
template <int DT, typename F>
void with_path(int path, F&& launch) {
    if (path == kWhole) launch(std::integral_constant<int, kWhole>());
    else if (DT == kF32 || path == kTail) launch(std::integral_constant<int, kTail>());
    else if constexpr (DT == kBF16) launch(std::integral_constant<int, kLoose>());
}
// Workgroups that walk over at most `tiles` tiles.  The widest ones: as many as run
// at a time, one to a CU, whose loads run on from tile to tile.  Of smaller ones
// several share a CU and fill each other's gaps: one to a tile, as far as that goes.
uint32_t walkers(uint64_t tiles, Tile t) {
    const uint64_t most = t == kWide ? 256 : 1 << 14;
    return uint32_t(tiles < 1 ? 1 : tiles < most ? tiles : most);
}

bool on(const void* const* list, int n, uintptr_t boundary) {
    for (int r = 0; r < n; r++)
        if (reinterpret_cast<uintptr_t>(list[r]) % boundary != 0) return false;
    return true;
}
int path_of(uint64_t pitch, bool on4) { return !on4 || pitch % 4 != 0 ? kLoose : pitch % 16 != 0 ? kTail : kWhole; }

// Whether the weights are streamed past LDS: for up to 32 rows of a run on average
// (64 runs of 4096 x 4096 bf16: 434 us with 32 rows, tiles 491), and for up to 64
// where the tiles of 128 would leave CUs idle (4 x 4096 x 4096 bf16, 33 rows: 45 us,
// tiles 51; 8 x 1000 x 1000 fp32, 64 rows: 19, 26; but 64 runs with 64 rows: 553, 427).
bool few_rows_to_run(int dtype, uint64_t features, uint64_t mean, uint64_t groups) {
    return mean <= 32 || (mean <= 64 && (dtype == kF32 || ceil_div(features, 128) * groups < 192));
}
// 16 waves to a workgroup where there are few of them: a wave's way through the summed index is shorter.
template <int DT, bool VEC, bool GATED>
void few(const LinearArgs& a, hipStream_t s) {
    const dim3 grid((a.outs + 15) / 16, a.runs * a.nranks);
    const uint64_t rows = a.rows.start[a.nranks];
    if (rows > 32 * uint64_t(grid.y)) hipLaunchKernelGGL((k_linear_few<DT, VEC, GATED, 4, 4>), grid, dim3(4 * 64), 0, s, a);
    else if (rows > 16 * uint64_t(grid.y)) hipLaunchKernelGGL((k_linear_few<DT, VEC, GATED, 4, 2>), grid, dim3(4 * 64), 0, s, a);
    else if (uint64_t(grid.x) * grid.y <= 512) hipLaunchKernelGGL((k_linear_few<DT, VEC, GATED, 16, 1>), grid, dim3(16 * 64), 0, s, a);
    else hipLaunchKernelGGL((k_linear_few<DT, VEC, GATED, 4, 1>), grid, dim3(4 * 64), 0, s, a);
}

template <int DT>
hipError_t forward(LinearArgs a, hipStream_t s) {
    constexpr uint64_t es = sizeof(typename Elem<DT>::type);
    const uint64_t rows = a.rows.start[a.nranks], groups = uint64_t(a.runs) * a.nranks;
    a.vecs = a.outs * es % 16 == 0 && on(a.y, a.nranks, 16) && on(a.pre, a.nranks, 16) && on(a.bias, a.nranks, 16) && on(a.residual, a.nranks, 16);
    const uint64_t features = uint64_t(a.outs) * (a.gated ? 2 : 1);
    if (few_rows_to_run(DT, features, ceil_div(rows, groups), groups)) {
        const bool vec = a.cols * es % 16 == 0 && on(a.x, a.nranks, 16) && on(a.weight, a.nranks, 16);
        if (a.gated) vec ? few<DT, true, true>(a, s) : few<DT, false, true>(a, s);
        else vec ? few<DT, true, false>(a, s) : few<DT, false, false>(a, s);
        return hipGetLastError();
    }
    with_path<DT>(path_of(a.cols * es, on(a.x, a.nranks, 4) && on(a.weight, a.nranks, 4)), [&](auto path) {
        constexpr int P = decltype(path)::value;
        const Tile t = pick_tile(DT, features, ceil_div(rows, groups), groups, P, false);
        // a run ends inside a tile, so there are up to one tile more than its rows fill
        const uint64_t tiles = ceil_div(features, kTileM[t]) * (rows / kTileN[t] + (groups < rows ? groups : rows));
        with_tile<DT, P, false>(t, [&](auto shape) {
            typedef decltype(shape) S;
            if (a.gated) hipLaunchKernelGGL((k_linear<DT, S, P, true>), dim3(walkers(tiles, t)), dim3(S::threads), 0, s, a);
            else hipLaunchKernelGGL((k_linear<DT, S, P, false>), dim3(walkers(tiles, t)), dim3(S::threads), 0, s, a);
        });
    });
    return hipGetLastError();
}

uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }
// Rows of a workgroup that forms dz: 32, or 8 where those would be too few
// workgroups (6048 rows of 509 fp32 with gelu: 41 us with 32).
uint32_t dz_rows(uint64_t rows, uint64_t wide) { return rows / 32 * ceil_div(wide, 4 * kThreads) >= 1024 ? 32 : 8; }
uint64_t dz_tiles(const RowTable& rows, int nranks, uint32_t runs, uint64_t wide) {
    const uint64_t n = rows.start[nranks], groups = uint64_t(runs) * nranks;
    return n / dz_rows(n, wide) + (groups < n ? groups : n);
}
// Where a product has too few tiles for the CUs, its sum is split among workgroups:
// into as many parts as bring the tiles to kSplitTiles of 64 x 64, whose fp32 sums
// fill kSplitBytes (tiny ones: as many bytes), of 16 steps or more each.  The sums'
// way through memory and one launch more are worth it from four parts on (dx and
// dweight in us, split and not: 17 rows of 33 fp32 from 2 x 7808 gated 42, 384; 8192
// rows of 2048 fp32 from 128 107, 238; 128 rows of 4096 bf16 from 4096 37, 45; but in
// two parts 1024 rows of 1024 bf16 from 1024 37, 24, and fp32 66, 58).
constexpr uint64_t kSplitTiles = 512, kSplitBytes = kSplitTiles * 64 * 64 * 4, kFewestParts = 4;
uint64_t part_terms(int dtype) { return 16 * kStepBytes / (dtype == kBF16 ? 2 : 4); }
uint32_t splits_of(uint64_t tiles, bool tiny, uint64_t terms, int dtype) {
    const uint64_t by_tiles = kSplitTiles * (tiny ? 4 : 1) / tiles, by_terms = terms / part_terms(dtype);
    const uint64_t n = by_tiles < by_terms ? by_tiles : by_terms;
    return n < kFewestParts ? 1 : uint32_t(n);
}
struct BackwardParts {
    uint64_t dz, partial, sums, bytes;
};
BackwardParts backward_parts(const RowTable& rows, int nranks, uint32_t runs, uint64_t wide, bool need_dz, bool dbias, int dtype) {
    const uint64_t es = dtype == kBF16 ? 2 : 4, n = rows.start[nranks], groups = uint64_t(runs) * nranks;
    BackwardParts b;
    b.dz = 0;
    b.partial = need_dz ? up(n * up(wide * es, 16), 256) : 0;
    b.sums = b.partial + (dbias ? up(dz_tiles(rows, nranks, runs, wide) * wide * 4, 256) : 0);
    const bool may_split = wide >= kFewestParts * part_terms(dtype) || ceil_div(n, groups) >= kFewestParts * part_terms(dtype);
    b.bytes = b.sums + (may_split ? kSplitBytes : 0);
    return b;
}

template <int DT, bool WEIGHT>
void join(const LinearArgs& a, uint64_t each, hipStream_t s) {
    const uint64_t need = ceil_div(each, kThreads);
    hipLaunchKernelGGL((k_linear_join<DT, WEIGHT>), dim3(uint32_t(need < 1024 ? need : 1024), a.runs * a.nranks), dim3(kThreads), 0, s, a);
}

template <int DT>
hipError_t backward(LinearArgs a, char* workspace, hipStream_t s) {
    constexpr uint64_t es = sizeof(typename Elem<DT>::type);
    const uint64_t rows = a.rows.start[a.nranks], groups = uint64_t(a.runs) * a.nranks, wide = uint64_t(a.outs) * (a.gated ? 2 : 1);
    const bool dbias = a.dbias[0] != nullptr;
    const BackwardParts b = backward_parts(a.rows, a.nranks, a.runs, wide, a.need_dz, dbias, DT);
    a.dz = workspace + b.dz;
    a.zpitch = uint32_t(a.need_dz ? up(wide * es, 16) : wide * es);
    a.dz_rows = dz_rows(rows, wide);
    a.dz_tiles = uint32_t(dz_tiles(a.rows, a.nranks, a.runs, wide));
    a.partial = dbias ? reinterpret_cast<float*>(workspace + b.partial) : nullptr;
    a.sums = reinterpret_cast<float*>(workspace + b.sums);
    a.col_vecs = a.cols * es % 16 == 0 && on(a.dx, a.nranks, 16) && on(a.dweight, a.nranks, 16);
    if (rows > 0 && (a.need_dz || dbias)) {
        const uint64_t tiles = dz_tiles(a.rows, a.nranks, a.runs, wide), across = ceil_div(a.outs, 4 * kThreads), most = ceil_div(4096, across);
        const dim3 grid(uint32_t(across), uint32_t(tiles < most ? tiles : most));
        if (a.gated) hipLaunchKernelGGL((k_linear_dz<DT, true>), grid, dim3(kThreads), 0, s, a);
        else hipLaunchKernelGGL((k_linear_dz<DT, false>), grid, dim3(kThreads), 0, s, a);
    }
    if (dbias) hipLaunchKernelGGL(k_linear_dbias<DT>, dim3(uint32_t(ceil_div(wide, 64)), uint32_t(groups)), dim3(1024), 0, s, a);
    const bool dz4 = a.need_dz || on(a.dy, a.nranks, 4), x4 = on(a.x, a.nranks, 4), w4 = on(a.weight, a.nranks, 4);
    if (rows > 0) {
        // dx: only dz' rows can end inside 16 bytes that count
        const int zp = path_of(a.zpitch, dz4), wp = path_of(a.cols * es, w4);
        with_path<DT>(zp == kLoose || wp == kLoose ? kLoose : zp, [&](auto path) {
            constexpr int P = decltype(path)::value;
            const uint64_t mean = ceil_div(rows, groups);
            if constexpr (P != kLoose) {
                const bool tiny = mean <= kTileN[kTiny];
                const uint64_t filled = ceil_div(a.cols, kTileM[kTiny]) * ceil_div(mean, kTileN[tiny ? kTiny : kSmall]) * groups;
                a.splits = splits_of(filled, tiny, wide, DT);
                if (a.splits > 1) {
                    const uint64_t tiles = ceil_div(a.cols, kTileM[kTiny]) * (rows / kTileN[tiny ? kTiny : kSmall] + (groups < rows ? groups : rows)) * a.splits;
                    if (tiny) hipLaunchKernelGGL((k_linear_dx<DT, Tiny, P, true>), dim3(walkers(tiles, kTiny)), dim3(Tiny::threads), 0, s, a);
                    else hipLaunchKernelGGL((k_linear_dx<DT, Small, P, true>), dim3(walkers(tiles, kSmall)), dim3(Small::threads), 0, s, a);
                    join<DT, false>(a, mean * a.cols, s);
                    return;
                }
            }
            const Tile t = pick_tile(DT, a.cols, mean, groups, P, true);
            const uint64_t tiles = ceil_div(a.cols, kTileM[t]) * (rows / kTileN[t] + (groups < rows ? groups : rows));
            with_tile<DT, P, true>(t, [&](auto shape) {
                typedef decltype(shape) S;
                hipLaunchKernelGGL((k_linear_dx<DT, S, P, false>), dim3(walkers(tiles, t)), dim3(S::threads), 0, s, a);
            });
        });
    }
    const bool loose = path_of(a.zpitch, dz4) == kLoose || path_of(a.cols * es, x4) == kLoose;
    auto dweight = [&](auto path) {
        constexpr int P = decltype(path)::value;
        if constexpr (P != kLoose) {
            const uint64_t filled = ceil_div(a.cols, kTileM[kSmall]) * ceil_div(wide, kTileN[kSmall]) * groups;
            a.splits = splits_of(filled, false, ceil_div(rows, groups), DT);
            if (a.splits > 1) {
                hipLaunchKernelGGL((k_linear_dweight<DT, Small, P, true>), dim3(walkers(filled * a.splits, kSmall)), dim3(Small::threads), 0, s, a);
                join<DT, true>(a, wide * a.cols, s);
                return;
            }
        }
        const Tile t = pick_tile(DT, a.cols, wide, groups, P, false);
        with_tile<DT, P, false>(t, [&](auto shape) {
            typedef decltype(shape) S;
            hipLaunchKernelGGL((k_linear_dweight<DT, S, P, false>), dim3(walkers(ceil_div(a.cols, S::BM) * ceil_div(wide, S::BN) * groups, t)), dim3(S::threads), 0, s, a);
        });
    };
    if constexpr (DT == kBF16) {
        if (loose) {
            dweight(std::integral_constant<int, kLoose>());
            return hipGetLastError();
        }
    }
    dweight(std::integral_constant<int, kWhole>());
    return hipGetLastError();
}

}  // namespace

uint64_t linear_backward_workspace(const RowTable& rows, int nranks, uint32_t runs, uint64_t outs, int act, int gated, bool dbias, int dtype) {
    return backward_parts(rows, nranks, runs, outs * (gated ? 2 : 1), gated || act != DT_ACT_NONE, dbias, dtype).bytes;
}
hipError_t launch_linear(const LinearArgs& a, int dtype, hipStream_t s) { return dtype == kBF16 ? forward<kBF16>(a, s) : forward<kF32>(a, s); }
hipError_t launch_linear_backward(const LinearArgs& a, void* workspace, int dtype, hipStream_t s) {
    char* ws = static_cast<char*>(workspace);
    return dtype == kBF16 ? backward<kBF16>(a, ws, s) : backward<kF32>(a, ws, s);
}

}  // namespace dt
