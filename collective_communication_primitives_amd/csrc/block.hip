// block.hip -- the norms after and before a block, with its gate, the residual
// scale and the residual, over the rows of all ranks, forward and backward.
//
//   p = N1(z)  (without a norm after the block p = z)
//   h = x + scale gate p
//   y = N2(h)
//   N(v) = (v - m) r w + b,  m = mean(v) (RMS norm: 0),  r = 1 / sqrt(mean((v - m)^2) + eps)
// backward, with n the normalised row, from dy and dh (h's gradient past the norm):
//   dx = dh + r2 (a - mean(a) - n2 mean(a n2)),  a = dy w2      (RMS norm: without mean(a))
//   du = scale gate dx,   dz = r1 (b - mean(b) - n1 mean(b n1)),  b = du w1
//   dw2 = sum dy n2, db2 = sum dy, dw1 = sum du n1, db1 = sum du over all ranks' rows,
//   dgate = scale dx p, summed over all ranks' rows for a gate that they share
//
// Bound by memory: 8 x 4096 rows of 8192 bf16 forward 367 us (5.8 TB/s), 8 x 4096 of
// 4096 backward 331 us (5.0 TB/s, 10 us of it the strips' fold), 2831 ragged rows of
// 1001 fp32 backward 29 + 6 us, few rows by the launch (one row per rank 5 us).
//
// A row lives in the registers of its waves through both norms, so each tensor is
// read and written once; the variance is that of the centred values, and y is
// taken from h before it is rounded.  All sums are fp32; results are rounded once.
// The gradients of what the rows share are summed in registers over a workgroup's
// rows, written as one strip per workgroup and folded in a fixed order into every
// rank's buffer.
#include <type_traits>

#include "dt_rows.h"

namespace dt {
namespace {

enum { kNoGate = 0, kChannelGate = 1, kRowGate = 2 };

// A row is shared by L lanes: 8 or 16 (several rows to a wave), a wave, or several
// waves, then the workgroup's all.
template <int L>
struct Share {
    static constexpr int waves = L <= 64 ? 4 : L / 64, threads = waves * 64, rows = threads / L;
};

// Rows of a wave or more are buffer resources; narrower ones are plain addresses.
struct NarrowRow {
    char* p;
    uint32_t bytes;
};
template <int DT, bool VEC, int POL>
__device__ __forceinline__ Unit<DT> load_unit(const NarrowRow& row, uint32_t u) {
    Unit<DT> x;
    u32x4 v = {0, 0, 0, 0};
    if constexpr (VEC) {
        if (u * 16 < row.bytes) v = load16_h<POL != 0>(row.p + u * 16);
    } else {
        v = load_loose<int(sizeof(typename Unit<DT>::T))>(row.p, u, row.bytes);
    }
    __builtin_memcpy(x.v, &v, 16);
    return x;
}
template <int DT, bool VEC>
__device__ __forceinline__ void store_unit(const NarrowRow& row, uint32_t u, const Unit<DT>& x) {
    u32x4 v;
    __builtin_memcpy(&v, x.v, 16);
    if constexpr (VEC) {
        if (u * 16 < row.bytes) store16(row.p + u * 16, v);
    } else {
        store_loose<int(sizeof(typename Unit<DT>::T))>(row.p, u, row.bytes, v);
    }
}
template <int L>
__device__ __forceinline__ auto shared_row(const void* base, uint64_t row, uint32_t pitch) {
    if constexpr (L < 64) return NarrowRow{const_cast<char*>(static_cast<const char*>(base)) + row * pitch, pitch};
    else return row_at(base, row, pitch);
}

// A unit's values rounded to the type, two to an instruction.
template <int DT>
__device__ __forceinline__ Unit<DT> rounded(const float (&v)[Unit<DT>::elems]) {
    Unit<DT> o;
    if constexpr (DT == kBF16) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        bf16x2 t[Unit<DT>::elems / 2];
#pragma unroll
        for (int e = 0; e < Unit<DT>::elems / 2; e++) t[e] = bf16x2{__bf16(v[2 * e]), __bf16(v[2 * e + 1])};
        __builtin_memcpy(o.v, t, 16);
    } else {
        __builtin_memcpy(o.v, v, 16);
    }
    return o;
}

// Sums over a row's lanes, the same in all of them.
template <int L>
__device__ __forceinline__ float row_total(float v, float* cell) {
    if constexpr (L == 8) {
        v += dpp<kSwap1>(v);
        v += dpp<kSwap2>(v);
        return v + dpp<kHalfMirror>(v);
    } else if constexpr (L == 16) {
        return sum16(v);
    } else {
        return row_sum<L / 64>(v, cell);
    }
}
template <int L>
__device__ __forceinline__ void row_totals(float& u, float& v, float (*cells)[Share<L>::waves]) {
    if constexpr (L <= 64) {
        u = row_total<L>(u, nullptr);
        v = row_total<L>(v, nullptr);
    } else {
        u = wave_sum(u);
        v = wave_sum(v);
        if ((threadIdx.x & 63) == 0) {
            cells[0][threadIdx.x >> 6] = u;
            cells[1][threadIdx.x >> 6] = v;
        }
        __syncthreads();
        u = v = 0.f;
#pragma unroll
        for (int k = 0; k < L / 64; k++) {
            u += cells[0][k];
            v += cells[1][k];
        }
    }
}
template <int L>
__device__ __forceinline__ uint32_t first_row() {
    const uint32_t mine = threadIdx.x / L;   // 0 where the workgroup shares a row
    return blockIdx.x * Share<L>::rows + (L < 64 ? mine : uint32_t(__builtin_amdgcn_readfirstlane(mine)));
}

// The rank of a row, which narrow rows' lanes do not share: counted against all
// ranks' first rows, whose addresses they do.
template <int L>
__device__ __forceinline__ int rank_for(const RowTable& t, int nranks, uint32_t row) {
    if constexpr (L >= 64) return rank_of_row(t, nranks, row);
    int r = 0;
    for (int k = 1; k < nranks; k++) r += row >= t.start[k] ? 1 : 0;
    return r;
}

// Rank r's pointer of a list in the kernel's arguments.  Narrow rows' lanes may be in
// several ranks, mostly in one: an index of their own would make the lanes fetch the
// pointer from the arguments' memory, microseconds away.
template <int L>
__device__ __forceinline__ uint32_t start_of(const RowTable& t, int nranks, int r) {
    if constexpr (L >= 64) return t.start[r];
    const int r0 = __builtin_amdgcn_readfirstlane(r);
    uint32_t at = t.start[r0];
    if (!__all(r == r0))
        for (int k = 0; k <= nranks; k++) at = r == k ? t.start[k] : at;
    return at;
}
template <int L, typename P>
__device__ __forceinline__ P of_rank(P const (&list)[kMaxRanksHost], int nranks, int r) {
    if constexpr (L >= 64) return list[r];
    const int r0 = __builtin_amdgcn_readfirstlane(r);
    P p = list[r0];
    if (!__all(r == r0))
        for (int k = 0; k < nranks; k++) p = r == k ? list[k] : p;
    return p;
}

template <int DT, bool VEC, int NV>
struct Units {
    Unit<DT> v[NV];
    // the lane's units of a row, L lanes apart; `there` false: untouched
    template <int L, int POL>
    __device__ __forceinline__ void load(bool there, const void* base, uint64_t row, uint32_t pitch, uint32_t lane) {
        if (!there) return;
        const auto r = shared_row<L>(base, row, pitch);
#pragma unroll
        for (int i = 0; i < NV; i++) v[i] = load_unit<DT, VEC, POL>(r, lane + i * L);
    }
    // The same of row `row` of `rows`.  AHEAD: for the next row; a unit that the row
    // ends in is loaded whole then where the rows behind it have its bytes, as picking
    // its values one by one would wait for them in the middle of the loads (backward of
    // 8 x 8192 rows of 1999 bf16 666 us, 456 this way), and cut() clears what lies
    // behind the row.
    template <int L, bool AHEAD>
    __device__ __forceinline__ void load_row(bool there, const void* base, uint64_t row, uint64_t rows, uint32_t pitch, uint32_t lane) {
        if constexpr (VEC || !AHEAD) {
            load<L, kPolNT>(there, base, row, pitch, lane);
        } else {
            if (!there) return;
            const char* p = static_cast<const char*>(base) + row * pitch;
            const uint64_t left = (rows - row) * pitch;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const uint32_t at = (lane + i * L) * 16;
                constexpr int ES = 16 / Unit<DT>::elems;
                u32x4 x = {0, 0, 0, 0};
                if (at < pitch) {
                    if (at + 16 <= left) x = __builtin_nontemporal_load(reinterpret_cast<const typename Loose<ES>::type*>(p + at));
                    else x = load_loose<ES>(p, lane + i * L, pitch);
                }
                __builtin_memcpy(v[i].v, &x, 16);
            }
        }
    }
    template <int L, bool AHEAD>
    __device__ __forceinline__ void cut(uint32_t pitch, uint32_t lane) {
        if constexpr (!VEC && AHEAD) {
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int32_t bytes = int32_t(pitch) - int32_t((lane + i * L) * 16);
                u32x4 x;
                __builtin_memcpy(&x, v[i].v, 16);
#pragma unroll
                for (int e = 0; e < 4; e++) x[e] &= bytes >= 4 * e + 4 ? ~0u : bytes == 4 * e + 2 ? 0xFFFFu : 0u;
                __builtin_memcpy(v[i].v, &x, 16);
            }
        }
    }
};
// Rows of rank r, for load_row.
template <int L, bool UNUSED>
__device__ __forceinline__ uint64_t rows_in(const RowTable& t, int nranks, int r) {
    return UNUSED ? 0 : start_of<L>(t, nranks, r + 1) - start_of<L>(t, nranks, r);
}

// ---------------------------------------------------------------- forward --
// More than one unit per lane of a full workgroup leaves no registers for the next
// row's loads and the weights: those are read again for every row, from the cache.
template <int DT, bool VEC, int NV, int L>
__global__ __launch_bounds__(Share<L>::threads) void k_block(BlockArgs a) {
    typedef Unit<DT> U;
    constexpr int E = U::elems;
    __shared__ float cells[2][4][Share<L>::waves];
    const uint32_t lane = threadIdx.x % L, step = gridDim.x * Share<L>::rows;
    const uint32_t total = a.rows.start[a.nranks], pitch = a.cols * uint32_t(sizeof(typename U::T));
    uint32_t row = first_row<L>();
    if (row >= total) return;
    int r = rank_for<L>(a.rows, a.nranks, row);
    const bool post = of_rank<L>(a.post_weight, a.nranks, r) != nullptr, pre = of_rank<L>(a.pre_weight, a.nranks, r) != nullptr, b1 = of_rank<L>(a.post_bias, a.nranks, r) != nullptr, b2 = of_rank<L>(a.pre_bias, a.nranks, r) != nullptr;
    const bool rms = a.rms, shared_gate = a.gate_kind == kChannelGate, row_gate = a.gate_kind == kRowGate;
    constexpr bool HELD = NV == 1 || L < 1024;
    const void *w1_at = of_rank<L>(a.post_weight, a.nranks, r), *c1_at = of_rank<L>(a.post_bias, a.nranks, r), *w2_at = of_rank<L>(a.pre_weight, a.nranks, r), *c2_at = of_rank<L>(a.pre_bias, a.nranks, r), *gate_at = of_rank<L>(a.gate, a.nranks, r);
    Units<DT, VEC, NV> w1, c1, w2, c2, gate, z, x;
    if constexpr (HELD) {
        w1.template load<L, 0>(post, w1_at, 0, pitch, lane);
        c1.template load<L, 0>(b1, c1_at, 0, pitch, lane);
        w2.template load<L, 0>(pre, w2_at, 0, pitch, lane);
        c2.template load<L, 0>(b2, c2_at, 0, pitch, lane);
        gate.template load<L, 0>(shared_gate, gate_at, 0, pitch, lane);
    }
    auto fetch = [&](uint64_t at) {
        const uint64_t rows = rows_in<L, VEC || !HELD>(a.rows, a.nranks, r);
        z.template load_row<L, HELD>(true, of_rank<L>(a.z, a.nranks, r), at, rows, pitch, lane);
        x.template load_row<L, HELD>(true, of_rank<L>(a.x, a.nranks, r), at, rows, pitch, lane);
        gate.template load_row<L, HELD>(row_gate, of_rank<L>(a.gate, a.nranks, r), at, rows, pitch, lane);
    };
    if constexpr (HELD) fetch(row - start_of<L>(a.rows, a.nranks, r));
    const float inv = 1.f / float(a.cols), scale = a.scale;
    // whole units are inside a row that is one of them, or outside
    auto inside = [&](int i, int e) { return (lane + i * L) * E + (VEC ? 0 : e) < a.cols; };
    for (int parity = 0; row < total; parity ^= 1) {
        if constexpr (!HELD) {
            while (row >= a.rows.start[r + 1]) r++;
            fetch(row - start_of<L>(a.rows, a.nranks, r));
            gate.template load<L, 0>(shared_gate, gate_at, 0, pitch, lane);
        }
        z.template cut<L, HELD>(pitch, lane);
        x.template cut<L, HELD>(pitch, lane);
        if (row_gate) gate.template cut<L, HELD>(pitch, lane);
        float v[NV][E], h[NV][E], f[NV][E];
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int e = 0; e < E; e++) {
                v[i][e] = z.v[i].get(e);
                h[i][e] = x.v[i].get(e);
                f[i][e] = shared_gate || row_gate ? scale * gate.v[i].get(e) : scale;
            }
        const int now = r;
        const uint64_t local = row - start_of<L>(a.rows, a.nranks, now);
        const uint32_t next = row + step;
        if (HELD && next < total) {
            if constexpr (L < 64) r = rank_for<L>(a.rows, a.nranks, next);
            else while (next >= a.rows.start[r + 1]) r++;
            fetch(next - start_of<L>(a.rows, a.nranks, r));
        }
        float stats[4] = {0.f, 0.f, 0.f, 0.f};
        // (v - mean) and 1 / deviation
        auto moments = [&](float (&t)[NV][E], int cell, float& mean, float& rstd) {
            mean = 0.f;
            if (!rms) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < NV; i++)
#pragma unroll
                    for (int e = 0; e < E; e++) s += t[i][e];   // zeros past the row's end
                mean = row_total<L>(s, cells[parity][cell]) * inv;
            }
            float q = 0.f;
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int e = 0; e < E; e++) {
                    t[i][e] = inside(i, e) ? t[i][e] - mean : 0.f;
                    q += t[i][e] * t[i][e];
                }
            rstd = 1.f / sqrtf(row_total<L>(q, cells[parity][cell + 1]) * inv + a.eps);
        };
        if (post) {
            float mean, rstd;
            moments(v, 0, mean, rstd);
            stats[0] = mean;
            stats[1] = rstd;
            if constexpr (!HELD) {
                w1.template load<L, 0>(true, w1_at, 0, pitch, lane);
                c1.template load<L, 0>(b1, c1_at, 0, pitch, lane);
            }
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int e = 0; e < E; e++) {
                    v[i][e] *= rstd * w1.v[i].get(e);
                    if (b1) v[i][e] += c1.v[i].get(e);
                }
        }
        const auto to = shared_row<L>(of_rank<L>(a.h, a.nranks, now), local, pitch);
#pragma unroll
        for (int i = 0; i < NV; i++) {
#pragma unroll
            for (int e = 0; e < E; e++) h[i][e] += f[i][e] * v[i][e];
            store_unit<DT, VEC>(to, lane + i * L, rounded<DT>(h[i]));
        }
        if (pre) {
            float mean, rstd;
            moments(h, 2, mean, rstd);
            stats[2] = mean;
            stats[3] = rstd;
            if constexpr (!HELD) {
                w2.template load<L, 0>(true, w2_at, 0, pitch, lane);
                c2.template load<L, 0>(b2, c2_at, 0, pitch, lane);
            }
            const auto out = shared_row<L>(of_rank<L>(a.y, a.nranks, now), local, pitch);
#pragma unroll
            for (int i = 0; i < NV; i++) {
                float y[E];
#pragma unroll
                for (int e = 0; e < E; e++) {
                    y[e] = h[i][e] * rstd * w2.v[i].get(e);
                    if (b2) y[e] += c2.v[i].get(e);
                }
                store_unit<DT, VEC>(out, lane + i * L, rounded<DT>(y));
            }
        }
        if (lane == 0 && of_rank<L>(a.stats, a.nranks, now) != nullptr) {
#pragma unroll
            for (int k = 0; k < 4; k++) of_rank<L>(a.stats, a.nranks, now)[local * 4 + k] = stats[k];
        }
        row = next;
    }
}

// --------------------------------------------------------------- backward --
// What a gradient of all rows is summed into, in the strips' order.
enum { kPostWeight, kPostBias, kPreWeight, kPreBias, kGate, kSums };

// SUM: the sums over the rows too; without, two sums of each row are left for
// k_block_columns.  BIAS: biases, or sums for them, are among the arguments, and
// take registers that others then do without.
template <int DT, bool VEC, int NV, int L, bool SUM, bool BIAS>
__global__ __launch_bounds__(Share<L>::threads) void k_block_backward(BlockBackArgs a) {
    typedef Unit<DT> U;
    constexpr int E = U::elems;
    __shared__ float cells[2][4][Share<L>::waves];
    const uint32_t lane = threadIdx.x % L, step = gridDim.x * Share<L>::rows;
    const uint32_t total = a.rows.start[a.nranks], pitch = a.cols * uint32_t(sizeof(typename U::T));
    uint32_t row = first_row<L>();
    float sums[SUM ? kSums : 1][NV][E];
#pragma unroll
    for (int k = 0; k < (SUM ? kSums : 1); k++)
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int e = 0; e < E; e++) sums[k][i][e] = 0.f;
    auto add = [&](int k, int i, int e, float v) {
        if constexpr (SUM) {
            if (BIAS || (k != kPostBias && k != kPreBias)) sums[k][i][e] += v;
        }
    };
    if (row < total) {
        int r = rank_for<L>(a.rows, a.nranks, row);
        const bool post = of_rank<L>(a.post_weight, a.nranks, r) != nullptr, pre = of_rank<L>(a.pre_weight, a.nranks, r) != nullptr, b1 = BIAS && of_rank<L>(a.post_bias, a.nranks, r) != nullptr;
        const bool rms = a.rms, shared_gate = a.gate_kind == kChannelGate, row_gate = a.gate_kind == kRowGate, gated = shared_gate || row_gate;
        const bool past = of_rank<L>(a.dh, a.nranks, r) != nullptr, need_z = of_rank<L>(a.z, a.nranks, r) != nullptr;
        Units<DT, VEC, NV> w1, c1, w2, gate, z, h, dy, dh;
        constexpr bool HELD = NV == 1 || L < (BIAS ? 512 : 1024);   // as in k_block
        const void *w1_at = of_rank<L>(a.post_weight, a.nranks, r), *c1_at = of_rank<L>(a.post_bias, a.nranks, r), *w2_at = of_rank<L>(a.pre_weight, a.nranks, r), *gate_at = of_rank<L>(a.gate, a.nranks, r);
        if constexpr (HELD) {
            w1.template load<L, 0>(post, w1_at, 0, pitch, lane);
            c1.template load<L, 0>(b1, c1_at, 0, pitch, lane);
            w2.template load<L, 0>(pre, w2_at, 0, pitch, lane);
            gate.template load<L, 0>(shared_gate, gate_at, 0, pitch, lane);
        }
        float m1, r1, m2, r2;
        auto fetch = [&](uint64_t at) {
            const uint64_t rows = rows_in<L, VEC || !HELD>(a.rows, a.nranks, r);
            dy.template load_row<L, HELD>(pre, of_rank<L>(a.dy, a.nranks, r), at, rows, pitch, lane);
            h.template load_row<L, HELD>(pre, of_rank<L>(a.h, a.nranks, r), at, rows, pitch, lane);
            dh.template load_row<L, HELD>(past, of_rank<L>(a.dh, a.nranks, r), at, rows, pitch, lane);
            z.template load_row<L, HELD>(need_z, of_rank<L>(a.z, a.nranks, r), at, rows, pitch, lane);
            gate.template load_row<L, HELD>(row_gate, of_rank<L>(a.gate, a.nranks, r), at, rows, pitch, lane);
            const float* s = of_rank<L>(a.stats, a.nranks, r) + at * 4;
            m1 = s[0];
            r1 = s[1];
            m2 = s[2];
            r2 = s[3];
        };
        uint64_t local = row - start_of<L>(a.rows, a.nranks, r);
        if constexpr (HELD) fetch(local);
        const float inv = 1.f / float(a.cols), scale = a.scale;
        for (int parity = 0; row < total; parity ^= 1) {
            if constexpr (!HELD) {
                while (row >= a.rows.start[r + 1]) r++;
                local = row - start_of<L>(a.rows, a.nranks, r);
                fetch(local);
                w2.template load<L, 0>(pre, w2_at, 0, pitch, lane);
            }
            if (pre) {
                dy.template cut<L, HELD>(pitch, lane);
                h.template cut<L, HELD>(pitch, lane);
            }
            if (past) dh.template cut<L, HELD>(pitch, lane);
            if (need_z) z.template cut<L, HELD>(pitch, lane);
            if (row_gate) gate.template cut<L, HELD>(pitch, lane);
            float d[NV][E], n[NV][E], g[NV][E];
            // dx
            if (pre) {
                float s1 = 0.f, s2 = 0.f;
#pragma unroll
                for (int i = 0; i < NV; i++)
#pragma unroll
                    for (int e = 0; e < E; e++) {
                        // past the row's end dy and the weights are 0: nothing is added to a row's sums
                        const float dye = dy.v[i].get(e);
                        n[i][e] = (h.v[i].get(e) - m2) * r2;
                        g[i][e] = dye * w2.v[i].get(e);
                        s1 += g[i][e];
                        s2 += g[i][e] * n[i][e];
                        add(kPreWeight, i, e, dye * n[i][e]);
                        add(kPreBias, i, e, dye);
                    }
                row_totals<L>(s1, s2, &cells[parity][0]);
                const float mean = rms ? 0.f : s1 * inv, along = s2 * inv;
                if (!SUM && lane == 0) {
                    a.row_sums[uint64_t(row) * 2] = mean;
                    a.row_sums[uint64_t(row) * 2 + 1] = along;
                }
#pragma unroll
                for (int i = 0; i < NV; i++)
#pragma unroll
                    for (int e = 0; e < E; e++) d[i][e] = (past ? dh.v[i].get(e) : 0.f) + r2 * (g[i][e] - mean - n[i][e] * along);
            } else {
#pragma unroll
                for (int i = 0; i < NV; i++)
#pragma unroll
                    for (int e = 0; e < E; e++) d[i][e] = past ? dh.v[i].get(e) : 0.f;
            }
            const auto to = shared_row<L>(of_rank<L>(a.dx, a.nranks, r), local, pitch);
#pragma unroll
            for (int i = 0; i < NV; i++) store_unit<DT, VEC>(to, lane + i * L, rounded<DT>(d[i]));
            // dz, and the gate's
            const int now = r;
            const uint64_t at = local;
            float t1 = 0.f, t2 = 0.f;
            if constexpr (!HELD) {
                w1.template load<L, 0>(post, w1_at, 0, pitch, lane);
                c1.template load<L, 0>(b1, c1_at, 0, pitch, lane);
                gate.template load<L, 0>(shared_gate, gate_at, 0, pitch, lane);
            }
#pragma unroll
            for (int i = 0; i < NV; i++) {
                float o[E];
#pragma unroll
                for (int e = 0; e < E; e++) {
                    n[i][e] = need_z ? z.v[i].get(e) : 0.f;
                    if (post) n[i][e] = (n[i][e] - m1) * r1;
                    float p = n[i][e];
                    if (post) p *= w1.v[i].get(e);
                    if (b1) p += c1.v[i].get(e);
                    const float dg = d[i][e] * p * scale, du = d[i][e] * (gated ? scale * gate.v[i].get(e) : scale);
                    if (shared_gate) add(kGate, i, e, dg);
                    o[e] = dg;
                    g[i][e] = post ? du * w1.v[i].get(e) : du;
                    add(kPostWeight, i, e, du * n[i][e]);
                    add(kPostBias, i, e, du);
                    t1 += g[i][e];
                    t2 += g[i][e] * n[i][e];
                }
                if (row_gate && of_rank<L>(a.dgate, a.nranks, now) != nullptr) store_unit<DT, VEC>(shared_row<L>(of_rank<L>(a.dgate, a.nranks, now), at, pitch), lane + i * L, rounded<DT>(o));
            }
            const float rstd = r1;
            const uint32_t next = row + step;
            if (HELD && next < total) {
                if constexpr (L < 64) r = rank_for<L>(a.rows, a.nranks, next);
                else while (next >= a.rows.start[r + 1]) r++;
                local = next - start_of<L>(a.rows, a.nranks, r);
                fetch(local);
            }
            const auto zto = shared_row<L>(of_rank<L>(a.dz, a.nranks, now), at, pitch);
            if (post) {
                row_totals<L>(t1, t2, &cells[parity][2]);
                const float mean = rms ? 0.f : t1 * inv, along = t2 * inv;
#pragma unroll
                for (int i = 0; i < NV; i++)
#pragma unroll
                    for (int e = 0; e < E; e++) g[i][e] = rstd * (g[i][e] - mean - n[i][e] * along);
            }
#pragma unroll
            for (int i = 0; i < NV; i++) store_unit<DT, VEC>(zto, lane + i * L, rounded<DT>(g[i]));
            row = next;
        }
    }
    if constexpr (SUM) {
        // the workgroup's strip of each sum that is wanted
        float* strip = a.partial + uint64_t(blockIdx.x) * a.wanted * a.cols;
        if constexpr (L <= 64) {
            // the rows that a wave holds side by side, then the waves one after the other
            __shared__ float joined[kSums][NV * E * L];
#pragma unroll
            for (int k = 0; k < kSums; k++) {
                if (!(a.sums >> k & 1)) continue;
#pragma unroll
                for (int i = 0; i < NV; i++)
#pragma unroll
                    for (int e = 0; e < E; e++)
#pragma unroll
                        for (int m = L; m < 64; m <<= 1) sums[k][i][e] += __shfl_xor(sums[k][i][e], m);
            }
            for (int w = 0; w < Share<L>::waves; w++) {
                if (int(threadIdx.x >> 6) == w && (threadIdx.x & 63) < uint32_t(L)) {
#pragma unroll
                    for (int k = 0; k < kSums; k++)
#pragma unroll
                        for (int i = 0; i < NV; i++)
#pragma unroll
                            for (int e = 0; e < E; e++) {
                                float* at = &joined[k][(lane + i * L) * E + e];
                                *at = w == 0 ? sums[k][i][e] : *at + sums[k][i][e];
                            }
                }
                __syncthreads();
            }
            uint32_t at = 0;
            for (int k = 0; k < kSums; k++) {
                if (!(a.sums >> k & 1)) continue;
                for (uint32_t c = threadIdx.x; c < a.cols; c += Share<L>::threads) strip[uint64_t(at) * a.cols + c] = joined[k][c];
                at++;
            }
        } else {
            uint32_t at = 0;
#pragma unroll
            for (int k = 0; k < kSums; k++) {
                if (!(a.sums >> k & 1)) continue;
                float* to = strip + uint64_t(at++) * a.cols;
#pragma unroll
                for (int i = 0; i < NV; i++)
#pragma unroll
                    for (int e = 0; e < E; e++) {
                        const uint32_t c = (lane + i * L) * E + e;
                        if (c < a.cols) to[c] = sums[k][i][e];
                    }
            }
        }
    }
}

// The sums over the rows from what k_block_backward left of each: strip
// blockIdx.y of the rows, 16 bytes of columns per thread.
template <int DT, bool VEC>
__global__ __launch_bounds__(kBlock) void k_block_columns(BlockBackArgs a) {
    typedef Unit<DT> U;
    constexpr int E = U::elems;
    const uint32_t u = blockIdx.x * kBlock + threadIdx.x, pitch = a.cols * uint32_t(sizeof(typename U::T));
    if (u * 16 >= pitch) return;
    const uint64_t total = a.rows.start[a.nranks];
    const uint32_t lo = uint32_t(total * blockIdx.y / a.strips), hi = uint32_t(total * (blockIdx.y + 1) / a.strips);
    float sums[kSums][E] = {};
    int r = rank_of_row(a.rows, a.nranks, lo);
    const bool post = a.post_weight[r] != nullptr, pre = a.pre_weight[r] != nullptr, b1 = a.post_bias[r] != nullptr;
    const bool shared_gate = a.gate_kind == kChannelGate, row_gate = a.gate_kind == kRowGate, gated = shared_gate || row_gate;
    const bool past = a.dh[r] != nullptr, need_z = a.z[r] != nullptr;
    auto some = [&](bool there, const void* base, uint64_t row) {
        U x = {};
        if (there) x = load_unit<DT, VEC, kPolNT>(row_at(base, row, pitch), u);
        return x;
    };
    const U w1 = some(post, a.post_weight[r], 0), c1 = some(b1, a.post_bias[r], 0), w2 = some(pre, a.pre_weight[r], 0);
    U gate = some(shared_gate, a.gate[r], 0);
    for (uint32_t row = lo; row < hi; row++) {
        while (row >= a.rows.start[r + 1]) r++;
        const uint64_t local = row - a.rows.start[r];
        const U dy = some(pre, a.dy[r], local), h = some(pre, a.h[r], local), dh = some(past, a.dh[r], local), z = some(need_z, a.z[r], local);
        if (row_gate) gate = some(true, a.gate[r], local);
        const float* s = a.stats[r] + local * 4;
        const float m1 = s[0], r1 = s[1], m2 = s[2], r2 = s[3];
        const float mean = pre ? a.row_sums[uint64_t(row) * 2] : 0.f, along = pre ? a.row_sums[uint64_t(row) * 2 + 1] : 0.f;
#pragma unroll
        for (int e = 0; e < E; e++) {
            float d = past ? dh.get(e) : 0.f;
            if (pre) {
                const float n = (h.get(e) - m2) * r2;
                d += r2 * (dy.get(e) * w2.get(e) - mean - n * along);
                sums[kPreWeight][e] += dy.get(e) * n;
                sums[kPreBias][e] += dy.get(e);
            }
            float n = z.get(e);
            if (post) n = (n - m1) * r1;
            float p = n;
            if (post) p *= w1.get(e);
            if (b1) p += c1.get(e);
            const float du = d * (gated ? a.scale * gate.get(e) : a.scale);
            sums[kPostWeight][e] += du * n;
            sums[kPostBias][e] += du;
            sums[kGate][e] += d * p * a.scale;
        }
    }
    uint32_t at = 0;
#pragma unroll
    for (int k = 0; k < kSums; k++) {
        if (!(a.sums >> k & 1)) continue;
        float* to = a.partial + (uint64_t(blockIdx.y) * a.wanted + at++) * a.cols + u * E;
#pragma unroll
        for (int e = 0; e < E; e++)
            if (u * E + e < a.cols) to[e] = sums[k][e];
    }
}

// ------------------------------------------------------------- wide rows --
// Rows too wide for the registers: a workgroup per row, which reads it again for
// each sum, and the columns' sums strip by strip.
template <int DT>
struct WideRow {
    typedef typename Elem<DT>::type T;
    static __device__ __forceinline__ float at(const void* base, uint64_t row, uint32_t cols, uint32_t c) {
        return Elem<DT>::get(static_cast<const T*>(base)[row * cols + c]);
    }
};

template <int DT>
__global__ __launch_bounds__(kBlock) void k_block_wide(BlockArgs a) {
    typedef typename Elem<DT>::type T;
    typedef WideRow<DT> W;
    __shared__ float tmp[4][kBlock / 64];
    const uint32_t row = blockIdx.x, C = a.cols;
    const int r = rank_of_row(a.rows, a.nranks, row);
    const uint64_t local = row - a.rows.start[r];
    const bool post = a.post_weight[r] != nullptr, pre = a.pre_weight[r] != nullptr;
    float m1 = 0.f, r1 = 0.f, m2 = 0.f, r2 = 0.f;
    auto p_of = [&](uint32_t c) {
        float v = W::at(a.z[r], local, C, c);
        if (post) v = (v - m1) * (r1 * W::at(a.post_weight[r], 0, C, c));
        if (a.post_bias[r] != nullptr) v += W::at(a.post_bias[r], 0, C, c);
        return v;
    };
    auto h_of = [&](uint32_t c) {
        const float f = a.gate_kind == kNoGate ? a.scale : a.scale * W::at(a.gate[r], a.gate_kind == kRowGate ? local : 0, C, c);
        return W::at(a.x[r], local, C, c) + f * p_of(c);
    };
    auto moments = [&](auto value, int cell, float& mean, float& rstd) {
        if (!a.rms) {
            float s = 0.f;
            for (uint32_t c = threadIdx.x; c < C; c += kBlock) s += value(c);
            mean = block_sum<kBlock / 64>(s, tmp[cell]) / float(C);
        }
        float q = 0.f;
        for (uint32_t c = threadIdx.x; c < C; c += kBlock) {
            const float d = value(c) - mean;
            q += d * d;
        }
        rstd = 1.f / sqrtf(block_sum<kBlock / 64>(q, tmp[cell + 1]) / float(C) + a.eps);
    };
    if (post) moments([&](uint32_t c) { return W::at(a.z[r], local, C, c); }, 0, m1, r1);
    if (pre) moments(h_of, 2, m2, r2);
    for (uint32_t c = threadIdx.x; c < C; c += kBlock) {
        const float h = h_of(c);
        static_cast<T*>(a.h[r])[local * C + c] = Elem<DT>::put(h);
        if (!pre) continue;
        float y = (h - m2) * r2 * W::at(a.pre_weight[r], 0, C, c);
        if (a.pre_bias[r] != nullptr) y += W::at(a.pre_bias[r], 0, C, c);
        static_cast<T*>(a.y[r])[local * C + c] = Elem<DT>::put(y);
    }
    if (threadIdx.x == 0 && a.stats[r] != nullptr) {
        float* s = a.stats[r] + local * 4;
        s[0] = m1;
        s[1] = r1;
        s[2] = m2;
        s[3] = r2;
    }
}

// One element of a wide row's backward pass; mean and along are those of dx's row.
template <int DT>
struct WideBack {
    typedef WideRow<DT> W;
    const BlockBackArgs& a;
    int r;
    uint64_t local;
    float m1, r1, m2, r2;
    __device__ __forceinline__ WideBack(const BlockBackArgs& args, int rank, uint64_t row) : a(args), r(rank), local(row) {
        const float* s = a.stats[r] + local * 4;
        m1 = s[0];
        r1 = s[1];
        m2 = s[2];
        r2 = s[3];
    }
    __device__ __forceinline__ float dy(uint32_t c) const { return W::at(a.dy[r], local, a.cols, c); }
    __device__ __forceinline__ float n2(uint32_t c) const { return (W::at(a.h[r], local, a.cols, c) - m2) * r2; }
    __device__ __forceinline__ float dx(uint32_t c, float mean, float along) const {
        float d = a.dh[r] != nullptr ? W::at(a.dh[r], local, a.cols, c) : 0.f;
        if (a.pre_weight[r] != nullptr) d += r2 * (dy(c) * W::at(a.pre_weight[r], 0, a.cols, c) - mean - n2(c) * along);
        return d;
    }
    __device__ __forceinline__ float n1(uint32_t c) const {
        const float v = a.z[r] != nullptr ? W::at(a.z[r], local, a.cols, c) : 0.f;
        return a.post_weight[r] != nullptr ? (v - m1) * r1 : v;
    }
    __device__ __forceinline__ float p(uint32_t c) const {
        float v = n1(c);
        if (a.post_weight[r] != nullptr) v *= W::at(a.post_weight[r], 0, a.cols, c);
        if (a.post_bias[r] != nullptr) v += W::at(a.post_bias[r], 0, a.cols, c);
        return v;
    }
    __device__ __forceinline__ float factor(uint32_t c) const {
        return a.gate_kind == kNoGate ? a.scale : a.scale * W::at(a.gate[r], a.gate_kind == kRowGate ? local : 0, a.cols, c);
    }
};

template <int DT>
__global__ __launch_bounds__(kBlock) void k_block_rows_wide(BlockBackArgs a) {
    typedef typename Elem<DT>::type T;
    typedef WideRow<DT> W;
    __shared__ float tmp[4][kBlock / 64];
    const uint32_t row = blockIdx.x, C = a.cols;
    const int r = rank_of_row(a.rows, a.nranks, row);
    const uint64_t local = row - a.rows.start[r];
    const WideBack<DT> v(a, r, local);
    const bool post = a.post_weight[r] != nullptr, pre = a.pre_weight[r] != nullptr;
    float mean = 0.f, along = 0.f, mean1 = 0.f, along1 = 0.f;
    if (pre) {
        float s1 = 0.f, s2 = 0.f;
        for (uint32_t c = threadIdx.x; c < C; c += kBlock) {
            const float g = v.dy(c) * W::at(a.pre_weight[r], 0, C, c);
            s1 += g;
            s2 += g * v.n2(c);
        }
        s1 = block_sum<kBlock / 64>(s1, tmp[0]);
        mean = a.rms ? 0.f : s1 / float(C);
        along = block_sum<kBlock / 64>(s2, tmp[1]) / float(C);
    }
    if (post) {
        float s1 = 0.f, s2 = 0.f;
        for (uint32_t c = threadIdx.x; c < C; c += kBlock) {
            const float g = v.dx(c, mean, along) * v.factor(c) * W::at(a.post_weight[r], 0, C, c);
            s1 += g;
            s2 += g * v.n1(c);
        }
        s1 = block_sum<kBlock / 64>(s1, tmp[2]);
        mean1 = a.rms ? 0.f : s1 / float(C);
        along1 = block_sum<kBlock / 64>(s2, tmp[3]) / float(C);
    }
    if (threadIdx.x == 0) {
        a.row_sums[uint64_t(row) * 2] = mean;
        a.row_sums[uint64_t(row) * 2 + 1] = along;
    }
    for (uint32_t c = threadIdx.x; c < C; c += kBlock) {
        const float d = v.dx(c, mean, along), du = d * v.factor(c);
        static_cast<T*>(a.dx[r])[local * C + c] = Elem<DT>::put(d);
        const float dz = post ? v.r1 * (du * W::at(a.post_weight[r], 0, C, c) - mean1 - v.n1(c) * along1) : du;
        static_cast<T*>(a.dz[r])[local * C + c] = Elem<DT>::put(dz);
        if (a.gate_kind == kRowGate && a.dgate[r] != nullptr) static_cast<T*>(a.dgate[r])[local * C + c] = Elem<DT>::put(d * v.p(c) * a.scale);
    }
}

// Sum blockIdx.y of those that are wanted, the strips folded in order: 64 columns
// per workgroup, each of its 16 waves takes every 16th strip, then the waves in
// order; every rank gets it.
template <int DT>
__global__ __launch_bounds__(1024) void k_block_fold(BlockBackArgs a) {
    typedef typename Elem<DT>::type T;
    __shared__ float sums[16][64];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    float s = 0.f;
    if (c < a.cols)
        for (uint32_t s0 = wave; s0 < a.strips; s0 += 16 * 8) {
            float v[8];  // eight strips' loads go out before the first is added
#pragma unroll
            for (int k = 0; k < 8; k++) v[k] = s0 + 16 * k < a.strips ? a.partial[(uint64_t(s0 + 16 * k) * a.wanted + blockIdx.y) * a.cols + c] : 0.f;
#pragma unroll
            for (int k = 0; k < 8; k++) s += v[k];
        }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c >= a.cols) return;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 16; k++) s += sums[k][lane];
    int which = 0;   // the blockIdx.y-th bit of those that are wanted
    for (uint32_t left = blockIdx.y; ; which++)
        if (a.sums >> which & 1) {
            if (left == 0) break;
            left--;
        }
    void* const* out = which == kPostWeight ? a.dpost_weight : which == kPostBias ? a.dpost_bias : which == kPreWeight ? a.dpre_weight :
                       which == kPreBias ? a.dpre_bias : a.dgate;
    for (int r = 0; r < a.nranks; r++) static_cast<T*>(out[r])[c] = Elem<DT>::put(s);
}

// -------------------------------------------------------------------- host --
// How a row is held: L lanes with NV units each; l 0: too wide.  One unit per lane
// as far as a workgroup goes: more waves hide more of the memory's latency than a
// second unit does (32768 x 4096 bf16 backward 393 us with two units in 256 lanes).
struct Hold {
    int nv, l;
};
Hold hold(uint32_t units, int dtype) {
    if (units <= 8) return {1, 8};
    if (units <= 16) return {1, 16};
    if (units <= 64) return {1, 64};
    if (units <= 128) return {2, 64};
    if (units <= 256) return {1, 256};
    if (units <= 512) return {1, 512};
    if (units <= 1024) return {2, 512};
    if (units <= 2048) return {2, 1024};
    if (units <= 4096 && dtype == kF32) return {4, 1024};
    return {0, 0};
}
// The backward pass keeps the sums over the rows in registers where a row is shared
// by fewer than 1024 lanes, up to two units in each; 1024 lanes have 128 registers
// each, where the sums do not fit.
bool sums_along(Hold h) { return h.l < 1024 && h.l != 0; }
template <int DT, typename F>
void with_hold(Hold h, F&& run) {
    typedef std::integral_constant<int, 1> one;
    if (h.l == 8) run(one(), std::integral_constant<int, 8>());
    else if (h.l == 16) run(one(), std::integral_constant<int, 16>());
    else if (h.l == 64 && h.nv == 1) run(one(), std::integral_constant<int, 64>());
    else if (h.l == 64) run(std::integral_constant<int, 2>(), std::integral_constant<int, 64>());
    else if (h.l == 256) run(one(), std::integral_constant<int, 256>());
    else if (h.l == 512 && h.nv == 1) run(one(), std::integral_constant<int, 512>());
    else if (h.l == 512) run(std::integral_constant<int, 2>(), std::integral_constant<int, 512>());
    else if (DT == kBF16 || h.nv == 2) run(std::integral_constant<int, 2>(), std::integral_constant<int, 1024>());
    else if constexpr (DT == kF32) run(std::integral_constant<int, 4>(), std::integral_constant<int, 1024>());
}
uint32_t units_of(uint32_t cols, int dtype) { return (cols + (dtype == kBF16 ? 8 : 4) - 1) / (dtype == kBF16 ? 8 : 4); }
bool rows16(uint32_t cols, int dtype) { return cols * uint64_t(dtype == kBF16 ? 2 : 4) % 16 == 0; }
// Workgroups of the backward pass, each of which leaves a strip: two to a CU, with
// four rows or more each.  Rows that are not whole 16 bytes wait longer for their
// loads and get as many workgroups as the registers let run, where a lane holds one
// unit (fp32: 8 x 4001 rows of 1001 274 us with 512 workgroups, 213 with 768, 185 with
// 1024; bf16: 8 x 8192 of 1999 861, 666, 899, as 768 run at a time; whole 16 bytes,
// fp32: 8 x 8192 of 1024 293, 305, 320).
uint32_t strips_of(uint32_t rows, uint32_t cols, int dtype) {
    const Hold h = hold(units_of(cols, dtype), dtype);
    if (!sums_along(h)) return rows < 256 ? rows : 256;
    const uint32_t per = h.l <= 64 ? 256 / h.l : 1, need = (rows + per - 1) / per;
    const bool more = h.l <= 256 && h.nv == 1 && !rows16(cols, dtype);
    uint32_t most = !more ? 512 : dtype == kBF16 ? 768 : 1024;
    if (need > 256 && need < 4 * most) most = (need + 3) / 4;  // at least four rows, but for very few
    return need < most ? need : most;
}
bool on16(const void* const* list, int n) {
    for (int r = 0; r < n; r++)
        if (reinterpret_cast<uintptr_t>(list[r]) % 16 != 0) return false;
    return true;
}
// Whether a list that is read is there: a rank without rows may list NULL.
bool given(const void* const* list, int n) {
    for (int r = 0; r < n; r++)
        if (list[r] != nullptr) return true;
    return false;
}

template <int DT, bool VEC>
hipError_t forward(const BlockArgs& a, hipStream_t s) {
    const uint32_t rows = a.rows.start[a.nranks];
    const Hold h = hold(units_of(a.cols, DT), DT);
    if (h.l == 0) {
        hipLaunchKernelGGL(k_block_wide<DT>, dim3(rows), dim3(kBlock), 0, s, a);
        return hipGetLastError();
    }
    with_hold<DT>(h, [&](auto nv, auto lanes) {
        constexpr int L = decltype(lanes)::value;
        const uint32_t need = (rows + Share<L>::rows - 1) / Share<L>::rows, most = 2048;
        hipLaunchKernelGGL((k_block<DT, VEC, decltype(nv)::value, L>), dim3(need < most ? need : most), dim3(Share<L>::threads), 0, s, a);
    });
    return hipGetLastError();
}

template <int DT, bool VEC>
hipError_t backward(const BlockBackArgs& a, hipStream_t s) {
    const uint32_t rows = a.rows.start[a.nranks];
    const Hold h = hold(units_of(a.cols, DT), DT);
    if (rows > 0) {
        if (h.l == 0) {
            hipLaunchKernelGGL(k_block_rows_wide<DT>, dim3(rows), dim3(kBlock), 0, s, a);
        } else {
            with_hold<DT>(h, [&](auto nv, auto lanes) {
                constexpr int NV = decltype(nv)::value, L = decltype(lanes)::value;
                const uint32_t groups = sums_along(h) ? a.strips : rows < 2048 ? rows : 2048;
                if (given(a.post_bias, a.nranks) || (a.sums & (1u << kPostBias | 1u << kPreBias)) != 0)
                    hipLaunchKernelGGL((k_block_backward<DT, VEC, NV, L, (L < 1024), true>), dim3(groups), dim3(Share<L>::threads), 0, s, a);
                else
                    hipLaunchKernelGGL((k_block_backward<DT, VEC, NV, L, (L < 1024), false>), dim3(groups), dim3(Share<L>::threads), 0, s, a);
            });
        }
        if (!sums_along(h) && a.wanted > 0)
            hipLaunchKernelGGL((k_block_columns<DT, VEC>), dim3((units_of(a.cols, DT) + kBlock - 1) / kBlock, a.strips), dim3(kBlock), 0, s, a);
    }
    if (a.wanted > 0) hipLaunchKernelGGL(k_block_fold<DT>, dim3((a.cols + 63) / 64, a.wanted), dim3(1024), 0, s, a);
    return hipGetLastError();
}

uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

}  // namespace

hipError_t launch_block(const BlockArgs& a, int dtype, hipStream_t s) {
    const int n = a.nranks;
    const bool vec = rows16(a.cols, dtype) && on16(a.z, n) && on16(a.x, n) && on16(a.gate, n) && on16(a.post_weight, n) && on16(a.post_bias, n) &&
                     on16(a.pre_weight, n) && on16(a.pre_bias, n) && on16(a.h, n) && on16(a.y, n);
    if (dtype == kBF16) return vec ? forward<kBF16, true>(a, s) : forward<kBF16, false>(a, s);
    return vec ? forward<kF32, true>(a, s) : forward<kF32, false>(a, s);
}

// The strips, and where they are formed in a launch of their own two sums of each row.
uint64_t block_workspace(uint32_t rows, uint32_t cols, int dtype) {
    return up(uint64_t(strips_of(rows, cols, dtype)) * kSums * cols * 4, 256) + (sums_along(hold(units_of(cols, dtype), dtype)) ? 0 : up(uint64_t(rows) * 8, 256));
}

hipError_t launch_block_backward(BlockBackArgs a, void* workspace, int dtype, hipStream_t s) {
    const int n = a.nranks;
    a.strips = strips_of(a.rows.start[n], a.cols, dtype);
    a.partial = static_cast<float*>(workspace);
    a.row_sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + up(uint64_t(a.strips) * kSums * a.cols * 4, 256));
    void* const* of[kSums] = {a.dpost_weight, a.dpost_bias, a.dpre_weight, a.dpre_bias, a.dgate};
    a.sums = a.wanted = 0;
    for (int k = 0; k < kSums; k++)
        if (of[k][0] != nullptr && (k != kGate || a.gate_kind == kChannelGate)) {
            a.sums |= 1u << k;
            a.wanted++;
        }
    const bool vec = rows16(a.cols, dtype) && on16(a.dy, n) && on16(a.dh, n) && on16(a.z, n) && on16(a.h, n) && on16(a.gate, n) &&
                     on16(a.post_weight, n) && on16(a.post_bias, n) && on16(a.pre_weight, n) && on16(a.dz, n) && on16(a.dx, n) && on16(a.dgate, n);
    if (dtype == kBF16) return vec ? backward<kBF16, true>(a, s) : backward<kBF16, false>(a, s);
    return vec ? backward<kF32, true>(a, s) : backward<kF32, false>(a, s);
}

}  // namespace dt
