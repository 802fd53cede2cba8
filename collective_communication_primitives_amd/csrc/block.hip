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

// Sums of two values over the WPR waves that hold a row.
template <int WPR>
__device__ __forceinline__ void row_sums(float& u, float& v, float (*cells)[Group<WPR>::waves]) {
    u = wave_sum(u);
    v = wave_sum(v);
    if constexpr (WPR > 1) {
        if ((threadIdx.x & 63) == 0) {
            cells[0][threadIdx.x >> 6] = u;
            cells[1][threadIdx.x >> 6] = v;
        }
        __syncthreads();
        u = v = 0.f;
#pragma unroll
        for (int k = 0; k < WPR; k++) {
            u += cells[0][k];
            v += cells[1][k];
        }
    }
}

template <int DT, bool VEC, int NV>
struct Units {
    Unit<DT> v[NV];
    // the lane's units of a row, L lanes apart; `there` false: untouched
    template <int L, int POL>
    __device__ __forceinline__ void load(bool there, const void* base, uint64_t row, uint32_t pitch, uint32_t lane) {
        if (!there) return;
        const Row r = row_at(base, row, pitch);
#pragma unroll
        for (int i = 0; i < NV; i++) v[i] = load_unit<DT, VEC, POL>(r, lane + i * L);
    }
};

// ---------------------------------------------------------------- forward --
template <int DT, bool VEC, int NV, int WPR>
__global__ __launch_bounds__(Group<WPR>::threads) void k_block(BlockArgs a) {
    typedef Unit<DT> U;
    constexpr int E = U::elems, L = Group<WPR>::lanes;
    __shared__ float cells[2][4][Group<WPR>::waves];
    const uint32_t lane = threadIdx.x % L, step = gridDim.x * Group<WPR>::rows;
    const uint32_t total = a.rows.start[a.nranks], pitch = a.cols * uint32_t(sizeof(typename U::T));
    uint32_t row = blockIdx.x * Group<WPR>::rows + (WPR == 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0);
    if (row >= total) return;
    int r = rank_of_row(a.rows, a.nranks, row);
    const bool post = a.post_weight[r] != nullptr, pre = a.pre_weight[r] != nullptr, b1 = a.post_bias[r] != nullptr, b2 = a.pre_bias[r] != nullptr;
    const bool rms = a.rms, shared_gate = a.gate_kind == kChannelGate, row_gate = a.gate_kind == kRowGate;
    Units<DT, VEC, NV> w1, c1, w2, c2, gate, z, x;
    w1.template load<L, 0>(post, a.post_weight[r], 0, pitch, lane);
    c1.template load<L, 0>(b1, a.post_bias[r], 0, pitch, lane);
    w2.template load<L, 0>(pre, a.pre_weight[r], 0, pitch, lane);
    c2.template load<L, 0>(b2, a.pre_bias[r], 0, pitch, lane);
    gate.template load<L, 0>(shared_gate, a.gate[r], 0, pitch, lane);
    auto fetch = [&](uint64_t at) {
        z.template load<L, kPolNT>(true, a.z[r], at, pitch, lane);
        x.template load<L, kPolNT>(true, a.x[r], at, pitch, lane);
        gate.template load<L, kPolNT>(row_gate, a.gate[r], at, pitch, lane);
    };
    fetch(row - a.rows.start[r]);
    const float inv = 1.f / float(a.cols), scale = a.scale;
    auto inside = [&](int i, int e) { return (lane + i * L) * E + e < a.cols; };
    for (int parity = 0; row < total; parity ^= 1) {
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
        const uint64_t local = row - a.rows.start[now];
        const uint32_t next = row + step;
        if (next < total) {
            while (next >= a.rows.start[r + 1]) r++;
            fetch(next - a.rows.start[r]);
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
                    for (int e = 0; e < E; e++) s += inside(i, e) ? t[i][e] : 0.f;
                mean = row_sum<WPR>(s, cells[parity][cell]) * inv;
            }
            float q = 0.f;
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int e = 0; e < E; e++) {
                    t[i][e] -= mean;
                    q += inside(i, e) ? t[i][e] * t[i][e] : 0.f;
                }
            rstd = 1.f / sqrtf(row_sum<WPR>(q, cells[parity][cell + 1]) * inv + a.eps);
        };
        if (post) {
            float mean, rstd;
            moments(v, 0, mean, rstd);
            stats[0] = mean;
            stats[1] = rstd;
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int e = 0; e < E; e++) {
                    v[i][e] *= rstd * w1.v[i].get(e);
                    if (b1) v[i][e] += c1.v[i].get(e);
                }
        }
        const Row to = row_at(a.h[now], local, pitch);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            U o;
#pragma unroll
            for (int e = 0; e < E; e++) {
                h[i][e] += f[i][e] * v[i][e];
                o.put(e, h[i][e]);
            }
            store_unit<DT, VEC>(to, lane + i * L, o);
        }
        if (pre) {
            float mean, rstd;
            moments(h, 2, mean, rstd);
            stats[2] = mean;
            stats[3] = rstd;
            const Row out = row_at(a.y[now], local, pitch);
#pragma unroll
            for (int i = 0; i < NV; i++) {
                U o;
#pragma unroll
                for (int e = 0; e < E; e++) {
                    const float n = h[i][e] * rstd * w2.v[i].get(e);
                    o.put(e, b2 ? n + c2.v[i].get(e) : n);
                }
                store_unit<DT, VEC>(out, lane + i * L, o);
            }
        }
        if (lane == 0 && a.stats[now] != nullptr) {
#pragma unroll
            for (int k = 0; k < 4; k++) a.stats[now][local * 4 + k] = stats[k];
        }
        row = next;
    }
}

// --------------------------------------------------------------- backward --
// What a gradient of all rows is summed into, in the strips' order.
enum { kPostWeight, kPostBias, kPreWeight, kPreBias, kGate, kSums };

template <int DT, bool VEC, int NV, int WPR>
__global__ __launch_bounds__(Group<WPR>::threads) void k_block_backward(BlockBackArgs a) {
    typedef Unit<DT> U;
    constexpr int E = U::elems, L = Group<WPR>::lanes;
    __shared__ float cells[2][4][Group<WPR>::waves];
    const uint32_t lane = threadIdx.x % L, step = gridDim.x * Group<WPR>::rows;
    const uint32_t total = a.rows.start[a.nranks], pitch = a.cols * uint32_t(sizeof(typename U::T));
    uint32_t row = blockIdx.x * Group<WPR>::rows + (WPR == 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0);
    float sums[kSums][NV][E];
#pragma unroll
    for (int k = 0; k < kSums; k++)
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int e = 0; e < E; e++) sums[k][i][e] = 0.f;
    if (row < total) {
        int r = rank_of_row(a.rows, a.nranks, row);
        const bool post = a.post_weight[r] != nullptr, pre = a.pre_weight[r] != nullptr, b1 = a.post_bias[r] != nullptr;
        const bool rms = a.rms, shared_gate = a.gate_kind == kChannelGate, row_gate = a.gate_kind == kRowGate, gated = shared_gate || row_gate;
        const bool past = a.dh[r] != nullptr, need_z = a.z[r] != nullptr;
        Units<DT, VEC, NV> w1, c1, w2, gate, z, h, dy, dh;
        w1.template load<L, 0>(post, a.post_weight[r], 0, pitch, lane);
        c1.template load<L, 0>(b1, a.post_bias[r], 0, pitch, lane);
        w2.template load<L, 0>(pre, a.pre_weight[r], 0, pitch, lane);
        gate.template load<L, 0>(shared_gate, a.gate[r], 0, pitch, lane);
        float m1, r1, m2, r2;
        auto fetch = [&](uint64_t at) {
            dy.template load<L, kPolNT>(pre, a.dy[r], at, pitch, lane);
            h.template load<L, kPolNT>(pre, a.h[r], at, pitch, lane);
            dh.template load<L, kPolNT>(past, a.dh[r], at, pitch, lane);
            z.template load<L, kPolNT>(need_z, a.z[r], at, pitch, lane);
            gate.template load<L, kPolNT>(row_gate, a.gate[r], at, pitch, lane);
            const float* s = a.stats[r] + at * 4;
            m1 = s[0];
            r1 = s[1];
            m2 = s[2];
            r2 = s[3];
        };
        uint64_t local = row - a.rows.start[r];
        fetch(local);
        const float inv = 1.f / float(a.cols), scale = a.scale;
        for (int parity = 0; row < total; parity ^= 1) {
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
                        sums[kPreWeight][i][e] += dye * n[i][e];
                        sums[kPreBias][i][e] += dye;
                    }
                row_sums<WPR>(s1, s2, &cells[parity][0]);
                const float mean = rms ? 0.f : s1 * inv, along = s2 * inv;
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
            const Row to = row_at(a.dx[r], local, pitch);
#pragma unroll
            for (int i = 0; i < NV; i++) {
                U o;
#pragma unroll
                for (int e = 0; e < E; e++) o.put(e, d[i][e]);
                store_unit<DT, VEC>(to, lane + i * L, o);
            }
            // dz, and the gate's
            const int now = r;
            const uint64_t at = local;
            float t1 = 0.f, t2 = 0.f;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                U o;
#pragma unroll
                for (int e = 0; e < E; e++) {
                    n[i][e] = need_z ? z.v[i].get(e) : 0.f;
                    if (post) n[i][e] = (n[i][e] - m1) * r1;
                    float p = n[i][e];
                    if (post) p *= w1.v[i].get(e);
                    if (b1) p += c1.v[i].get(e);
                    const float dg = d[i][e] * p * scale, du = d[i][e] * (gated ? scale * gate.v[i].get(e) : scale);
                    if (shared_gate) sums[kGate][i][e] += dg;
                    o.put(e, dg);
                    g[i][e] = post ? du * w1.v[i].get(e) : du;
                    sums[kPostWeight][i][e] += du * n[i][e];
                    sums[kPostBias][i][e] += du;
                    t1 += g[i][e];
                    t2 += g[i][e] * n[i][e];
                }
                if (row_gate && a.dgate[now] != nullptr) store_unit<DT, VEC>(row_at(a.dgate[now], at, pitch), lane + i * L, o);
            }
            const float rstd = r1;
            const uint32_t next = row + step;
            if (next < total) {
                while (next >= a.rows.start[r + 1]) r++;
                local = next - a.rows.start[r];
                fetch(local);
            }
            const Row zto = row_at(a.dz[now], at, pitch);
            if (post) {
                row_sums<WPR>(t1, t2, &cells[parity][2]);
                const float mean = rms ? 0.f : t1 * inv, along = t2 * inv;
#pragma unroll
                for (int i = 0; i < NV; i++)
#pragma unroll
                    for (int e = 0; e < E; e++) g[i][e] = rstd * (g[i][e] - mean - n[i][e] * along);
            }
#pragma unroll
            for (int i = 0; i < NV; i++) {
                U o;
#pragma unroll
                for (int e = 0; e < E; e++) o.put(e, g[i][e]);
                store_unit<DT, VEC>(zto, lane + i * L, o);
            }
            row = next;
        }
    }
    // the workgroup's strip of each sum that is wanted
    float* strip = a.partial + uint64_t(blockIdx.x) * a.wanted * a.cols;
    uint32_t at = 0;
#pragma unroll
    for (int k = 0; k < kSums; k++) {
        if (!(a.sums >> k & 1)) continue;
        float* to = strip + uint64_t(at++) * a.cols;
        if constexpr (WPR == 1) {
            // the waves' sums one after the other, in a fixed order
            __shared__ float joined[NV * E * 64];
            __syncthreads();
            for (int w = 0; w < Group<WPR>::waves; w++) {
                if (int(threadIdx.x >> 6) == w) {
#pragma unroll
                    for (int i = 0; i < NV; i++)
#pragma unroll
                        for (int e = 0; e < E; e++) {
                            const uint32_t c = (lane + i * L) * E + e;
                            joined[c] = w == 0 ? sums[k][i][e] : joined[c] + sums[k][i][e];
                        }
                }
                __syncthreads();
            }
            for (uint32_t c = threadIdx.x; c < a.cols; c += Group<WPR>::threads) to[c] = joined[c];
        } else {
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

// Strip blockIdx.y of the rows, one column per thread.
template <int DT>
__global__ __launch_bounds__(kBlock) void k_block_columns_wide(BlockBackArgs a) {
    const uint32_t c = blockIdx.x * kBlock + threadIdx.x;
    if (c >= a.cols) return;
    const uint64_t total = a.rows.start[a.nranks];
    const uint32_t lo = uint32_t(total * blockIdx.y / a.strips), hi = uint32_t(total * (blockIdx.y + 1) / a.strips);
    float sums[kSums] = {};
    int r = rank_of_row(a.rows, a.nranks, lo);
    for (uint32_t row = lo; row < hi; row++) {
        while (row >= a.rows.start[r + 1]) r++;
        const WideBack<DT> v(a, r, row - a.rows.start[r]);
        const float d = v.dx(c, a.row_sums[uint64_t(row) * 2], a.row_sums[uint64_t(row) * 2 + 1]), du = d * v.factor(c);
        if (a.pre_weight[r] != nullptr) {
            const float dy = v.dy(c);
            sums[kPreWeight] += dy * v.n2(c);
            sums[kPreBias] += dy;
        }
        sums[kPostWeight] += du * v.n1(c);
        sums[kPostBias] += du;
        sums[kGate] += d * v.p(c) * a.scale;
    }
    uint32_t at = 0;
#pragma unroll
    for (int k = 0; k < kSums; k++)
        if (a.sums >> k & 1) a.partial[(uint64_t(blockIdx.y) * a.wanted + at++) * a.cols + c] = sums[k];
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
// How a row is held: WPR waves with NV units per lane each; wpr 0: too wide.
struct Hold {
    int nv, wpr;
};
Hold hold(uint32_t units) {
    if (units <= 64) return {1, 1};
    if (units <= 128) return {2, 1};
    if (units <= 256) return {1, 4};
    if (units <= 512) return {2, 4};
    if (units <= 1024) return {2, 8};
    return {0, 0};
}
template <typename F>
void with_hold(Hold h, F&& run) {
    if (h.wpr == 1 && h.nv == 1) run(std::integral_constant<int, 1>(), std::integral_constant<int, 1>());
    else if (h.wpr == 1) run(std::integral_constant<int, 2>(), std::integral_constant<int, 1>());
    else if (h.wpr == 4 && h.nv == 1) run(std::integral_constant<int, 1>(), std::integral_constant<int, 4>());
    else if (h.wpr == 4) run(std::integral_constant<int, 2>(), std::integral_constant<int, 4>());
    else run(std::integral_constant<int, 2>(), std::integral_constant<int, 8>());
}
uint32_t units_of(uint32_t cols, int dtype) { return (cols + (dtype == kBF16 ? 8 : 4) - 1) / (dtype == kBF16 ? 8 : 4); }
// Workgroups of the backward pass, each of which leaves a strip.
uint32_t strips_of(uint32_t rows, uint32_t cols, int dtype) {
    const Hold h = hold(units_of(cols, dtype));
    if (h.wpr == 0) return rows < 256 ? rows : 256;
    const uint32_t need = h.wpr == 1 ? (rows + 3) / 4 : rows;
    uint32_t most = 512;
    if (need < 4 * most) most = (need + 3) / 4;  // at least four rows
    return need < most ? need : most;
}
bool on16(const void* const* list, int n) {
    for (int r = 0; r < n; r++)
        if (reinterpret_cast<uintptr_t>(list[r]) % 16 != 0) return false;
    return true;
}
bool rows16(uint32_t cols, int dtype) { return cols * uint64_t(dtype == kBF16 ? 2 : 4) % 16 == 0; }

template <int DT, bool VEC>
hipError_t forward(const BlockArgs& a, hipStream_t s) {
    const uint32_t rows = a.rows.start[a.nranks];
    const Hold h = hold(units_of(a.cols, DT));
    if (h.wpr == 0) {
        hipLaunchKernelGGL(k_block_wide<DT>, dim3(rows), dim3(kBlock), 0, s, a);
        return hipGetLastError();
    }
    with_hold(h, [&](auto nv, auto wpr) {
        constexpr int W = decltype(wpr)::value;
        const uint32_t need = (rows + Group<W>::rows - 1) / Group<W>::rows, most = 2048;
        hipLaunchKernelGGL((k_block<DT, VEC, decltype(nv)::value, W>), dim3(need < most ? need : most), dim3(Group<W>::threads), 0, s, a);
    });
    return hipGetLastError();
}

template <int DT, bool VEC>
hipError_t backward(const BlockBackArgs& a, hipStream_t s) {
    const uint32_t rows = a.rows.start[a.nranks];
    const Hold h = hold(units_of(a.cols, DT));
    if (rows > 0 && h.wpr == 0) {
        hipLaunchKernelGGL(k_block_rows_wide<DT>, dim3(rows), dim3(kBlock), 0, s, a);
        if (a.wanted > 0) hipLaunchKernelGGL(k_block_columns_wide<DT>, dim3((a.cols + kBlock - 1) / kBlock, a.strips), dim3(kBlock), 0, s, a);
    } else if (rows > 0) {
        with_hold(h, [&](auto nv, auto wpr) {
            constexpr int W = decltype(wpr)::value;
            hipLaunchKernelGGL((k_block_backward<DT, VEC, decltype(nv)::value, W>), dim3(a.strips), dim3(Group<W>::threads), 0, s, a);
        });
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

// The strips, and for rows that no registers hold two sums of each row.
uint64_t block_workspace(uint32_t rows, uint32_t cols, int dtype) {
    return up(uint64_t(strips_of(rows, cols, dtype)) * kSums * cols * 4, 256) + (hold(units_of(cols, dtype)).wpr == 0 ? up(uint64_t(rows) * 8, 256) : 0);
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
