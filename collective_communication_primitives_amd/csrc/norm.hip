// norm.hip -- layer norm over the rows of all ranks, forward and backward.
//
//   mu = sum_i x_i / C      v = sum_i (x_i - mu)^2 / C      r = 1 / sqrt(v + eps)
//   n_i = (x_i - mu) r      y_i = n_i w_i + b_i
//   dx_i = r (g_i - mean(g) - n_i mean(g n)),   g_i = dy_i w_i
//   dw_i = sum over all rows of dy_i n_i,       db_i = sum over all rows of dy_i
//
// The variance is taken from the centred values (not from sums of squares),
// so a large mean costs the digits of its own rounding, not of its square's.  All sums are fp32; y, dx, dw and db are
// rounded once.  The weight's gradient is the sum over the rows of every
// rank, folded in a fixed order, and goes to every rank: the AllReduce of
// the ranks' partial gradients in the same pass.
//
// Both passes read each row once: a row lives in the registers of WPR waves,
// and a workgroup walks over rows with its share of the weight (and, in the
// backward pass, of dw and db) in registers too.  The next row's loads go
// out before the current row is reduced.  Both are bound by memory: 32768 rows
// of 8192 bf16 forward 195 us, 5.5 TB/s; 32768 of 4096 backward 146 us, 5.6 TB/s
// with the fold of the weight's gradients (6.8 us).
//
// Rows of more than 1024 units of 16 bytes take 16 waves, whose 1024 threads leave
// each lane 128 registers.  What does not fit is spilled (the second number: rows off
// 16-byte boundaries): forward bf16 above 16384 elements 28 / 44 registers; backward
// bf16 above 8192 3 / 34, above 16384 180 / 195, fp32 above 8192 28 / 58.  128 MiB of
// bf16 rows, forward and backward: rows of 8192 58 and 93 us, of 16384 55 and 104, of
// 32768 89 and 424; of 65536, which no registers hold, 244 and 453.
#include <type_traits>

#include "dt_rows.h"

namespace dt {
namespace {

template <int DT, bool VEC, int NV, int WPR>
__global__ __launch_bounds__(Group<WPR>::threads) void k_norm(NormArgs a) {
    typedef Unit<DT> U;
    typedef typename Elem<DT>::type T;
    constexpr int E = U::elems, L = Group<WPR>::lanes;
    __shared__ float cells[2][2][Group<WPR>::waves];
    const uint32_t lane = threadIdx.x % L, step = gridDim.x * Group<WPR>::rows;
    const uint32_t total = a.rows.start[a.nranks];
    uint32_t row = blockIdx.x * Group<WPR>::rows + (WPR == 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0);
    if (row >= total) return;
    int r = rank_of_row(a.rows, a.nranks, row);
    U w[NV], b[NV], x[NV];
    const bool biased = a.bias[r] != nullptr;
    const uint32_t pitch = a.cols * sizeof(T);
    {
        const Row wr = row_at(a.weight[r], 0, pitch), br = row_at(biased ? a.bias[r] : a.weight[r], 0, pitch);
        const Row xr = row_at(a.x[r], row - a.rows.start[r], pitch);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            w[i] = load_unit<DT, VEC, 0>(wr, lane + i * L);
            b[i] = load_unit<DT, VEC, 0>(br, lane + i * L);
            x[i] = load_unit<DT, VEC, kPolNT>(xr, lane + i * L);
        }
    }
    const float inv = 1.f / float(a.cols);
    for (int parity = 0; row < total; parity ^= 1) {
        float v[NV][E];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
#pragma unroll
            for (int e = 0; e < E; e++) {
                v[i][e] = x[i].get(e);
                s += v[i][e];
            }
        }
        const int now = r;
        const uint64_t local = row - a.rows.start[now];
        const uint32_t next = row + step;
        if (next < total) {
            while (next >= a.rows.start[r + 1]) r++;
            const Row xr = row_at(a.x[r], next - a.rows.start[r], pitch);
#pragma unroll
            for (int i = 0; i < NV; i++) x[i] = load_unit<DT, VEC, kPolNT>(xr, lane + i * L);
        }
        const float mean = row_sum<WPR>(s, cells[parity][0]) * inv;
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
#pragma unroll
            for (int e = 0; e < E; e++) {
                v[i][e] -= mean;
                q += (lane + i * L) * E + e < a.cols ? v[i][e] * v[i][e] : 0.f;
            }
        }
        const float rstd = 1.f / sqrtf(row_sum<WPR>(q, cells[parity][1]) * inv + a.eps);
        const Row to = row_at(a.y[now], local, pitch);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            U y;
#pragma unroll
            for (int e = 0; e < E; e++) {
                const float n = v[i][e] * rstd * w[i].get(e);
                y.put(e, biased ? n + b[i].get(e) : n);
            }
            store_unit<DT, VEC>(to, lane + i * L, y);
        }
        if (lane == 0 && a.mean[now] != nullptr) {
            a.mean[now][local] = mean;
            a.rstd[now][local] = rstd;
        }
        row = next;
    }
}

template <int DT, bool VEC, int NV, int WPR>
__global__ __launch_bounds__(Group<WPR>::threads) void k_norm_backward(NormBackArgs a) {
    typedef Unit<DT> U;
    typedef typename Elem<DT>::type T;
    constexpr int E = U::elems, L = Group<WPR>::lanes;
    __shared__ float cells[2][2][Group<WPR>::waves];
    const uint32_t lane = threadIdx.x % L, step = gridDim.x * Group<WPR>::rows;
    const uint32_t total = a.rows.start[a.nranks];
    uint32_t row = blockIdx.x * Group<WPR>::rows + (WPR == 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0);
    float dw[NV][E], db[NV][E];
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int e = 0; e < E; e++) dw[i][e] = db[i][e] = 0.f;
    if (row < total) {
        int r = rank_of_row(a.rows, a.nranks, row);
        U w[NV], x[NV], d[NV];
        const uint32_t pitch = a.cols * sizeof(T);
        uint64_t local = row - a.rows.start[r];
        float mean = a.mean[r][local], rstd = a.rstd[r][local];
        {
            const Row wr = row_at(a.weight[r], 0, pitch), xr = row_at(a.x[r], local, pitch), dr = row_at(a.dy[r], local, pitch);
#pragma unroll
            for (int i = 0; i < NV; i++) {
                w[i] = load_unit<DT, VEC, 0>(wr, lane + i * L);
                x[i] = load_unit<DT, VEC, kPolNT>(xr, lane + i * L);
                d[i] = load_unit<DT, VEC, kPolNT>(dr, lane + i * L);
            }
        }
        const float inv = 1.f / float(a.cols);
        for (int parity = 0; row < total; parity ^= 1) {
            float n[NV][E], g[NV][E];
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < NV; i++) {
#pragma unroll
                for (int e = 0; e < E; e++) {
                    // past the row's end dy is 0, and nothing is added to any sum
                    const float dy = d[i].get(e);
                    n[i][e] = (x[i].get(e) - mean) * rstd;
                    g[i][e] = dy * w[i].get(e);
                    s1 += g[i][e];
                    s2 += g[i][e] * n[i][e];
                    dw[i][e] += dy * n[i][e];
                    db[i][e] += dy;
                }
            }
            const int now = r;
            const float scale = rstd;
            const Row to = row_at(a.dx[now], local, pitch);
            const uint32_t next = row + step;
            if (next < total) {
                while (next >= a.rows.start[r + 1]) r++;
                local = next - a.rows.start[r];
                mean = a.mean[r][local];
                rstd = a.rstd[r][local];
                const Row xr = row_at(a.x[r], local, pitch), dr = row_at(a.dy[r], local, pitch);
#pragma unroll
                for (int i = 0; i < NV; i++) {
                    x[i] = load_unit<DT, VEC, kPolNT>(xr, lane + i * L);
                    d[i] = load_unit<DT, VEC, kPolNT>(dr, lane + i * L);
                }
            }
            s1 = wave_sum(s1);
            s2 = wave_sum(s2);
            if constexpr (WPR > 1) {
                if ((threadIdx.x & 63) == 0) {
                    cells[parity][0][threadIdx.x >> 6] = s1;
                    cells[parity][1][threadIdx.x >> 6] = s2;
                }
                __syncthreads();
                s1 = s2 = 0.f;
#pragma unroll
                for (int k = 0; k < WPR; k++) {
                    s1 += cells[parity][0][k];
                    s2 += cells[parity][1][k];
                }
            }
            const float m1 = s1 * inv, m2 = s2 * inv;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                U o;
#pragma unroll
                for (int e = 0; e < E; e++) o.put(e, scale * (g[i][e] - m1 - n[i][e] * m2));
                store_unit<DT, VEC>(to, lane + i * L, o);
            }
            row = next;
        }
    }
    // the workgroup's strip of the partial sums
    float* strip = a.partial + uint64_t(blockIdx.x) * 2 * a.cols;
    if constexpr (WPR == 1) {
        // its waves' sums one after the other, in a fixed order
        __shared__ float sums[2][NV * E * 64];
        for (int k = 0; k < Group<WPR>::waves; k++) {
            if (int(threadIdx.x >> 6) == k) {
#pragma unroll
                for (int i = 0; i < NV; i++)
#pragma unroll
                    for (int e = 0; e < E; e++) {
                        const uint32_t c = (lane + i * L) * E + e;
                        sums[0][c] = k == 0 ? dw[i][e] : sums[0][c] + dw[i][e];
                        sums[1][c] = k == 0 ? db[i][e] : sums[1][c] + db[i][e];
                    }
            }
            __syncthreads();
        }
        for (uint32_t c = threadIdx.x; c < a.cols; c += Group<WPR>::threads) {
            strip[c] = sums[0][c];
            strip[a.cols + c] = sums[1][c];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; i++) {
#pragma unroll
            for (int e = 0; e < E; e++) {
                const uint32_t c = (lane + i * L) * E + e;
                if (c >= a.cols) continue;
                strip[c] = dw[i][e];
                strip[a.cols + c] = db[i][e];
            }
        }
    }
}

// Rows of at most 16 units: 16 lanes per row, four rows to a wave.
constexpr uint32_t kNarrowRows = kBlock / 16;  // rows in flight in a workgroup

template <int DT, bool VEC>
__device__ __forceinline__ Unit<DT> narrow_unit(const void* base, uint64_t row, uint32_t pitch, uint32_t u) {
    Unit<DT> x;
    u32x4 v = {0, 0, 0, 0};
    const char* p = static_cast<const char*>(base) + row * pitch;
    if constexpr (VEC) {
        if (u * 16 < pitch) v = load16(p + u * 16);
    } else {
        v = load_loose<int(sizeof(typename Unit<DT>::T))>(p, u, pitch);
    }
    __builtin_memcpy(x.v, &v, 16);
    return x;
}
template <int DT, bool VEC>
__device__ __forceinline__ void narrow_store(void* base, uint64_t row, uint32_t pitch, uint32_t u, const Unit<DT>& x) {
    u32x4 v;
    __builtin_memcpy(&v, x.v, 16);
    char* p = static_cast<char*>(base) + row * pitch;
    if constexpr (VEC) {
        if (u * 16 < pitch) store16(p + u * 16, v);
    } else {
        store_loose<int(sizeof(typename Unit<DT>::T))>(p, u, pitch, v);
    }
}

template <int DT, bool VEC>
__global__ __launch_bounds__(kBlock) void k_norm_narrow(NormArgs a) {
    typedef Unit<DT> U;
    constexpr int E = U::elems;
    const uint32_t u = threadIdx.x & 15, total = a.rows.start[a.nranks], step = gridDim.x * kNarrowRows;
    const uint32_t pitch = a.cols * uint32_t(sizeof(typename U::T));
    uint32_t row = blockIdx.x * kNarrowRows + (threadIdx.x >> 4);
    int r = 0;
    while (r + 1 < a.nranks && row >= a.rows.start[r + 1]) r++;
    if (row >= total) return;  // whole rows of lanes leave together
    const U w = narrow_unit<DT, VEC>(a.weight[r], 0, pitch, u);
    const bool biased = a.bias[r] != nullptr;
    const U b = narrow_unit<DT, VEC>(biased ? a.bias[r] : a.weight[r], 0, pitch, u);
    U x = narrow_unit<DT, VEC>(a.x[r], row - a.rows.start[r], pitch, u);
    const float inv = 1.f / float(a.cols);
    while (row < total) {
        float v[E], s = 0.f;
#pragma unroll
        for (int e = 0; e < E; e++) {
            v[e] = x.get(e);
            s += v[e];
        }
        const int now = r;
        const uint64_t local = row - a.rows.start[now];
        row += step;
        if (row < total) {
            while (row >= a.rows.start[r + 1]) r++;
            x = narrow_unit<DT, VEC>(a.x[r], row - a.rows.start[r], pitch, u);
        }
        const float mean = sum16(s) * inv;
        float q = 0.f;
#pragma unroll
        for (int e = 0; e < E; e++) {
            v[e] -= mean;
            q += u * E + e < a.cols ? v[e] * v[e] : 0.f;
        }
        const float rstd = 1.f / sqrtf(sum16(q) * inv + a.eps);
        U y;
#pragma unroll
        for (int e = 0; e < E; e++) {
            const float n = v[e] * rstd * w.get(e);
            y.put(e, biased ? n + b.get(e) : n);
        }
        narrow_store<DT, VEC>(a.y[now], local, pitch, u, y);
        if (u == 0 && a.mean[now] != nullptr) {
            a.mean[now][local] = mean;
            a.rstd[now][local] = rstd;
        }
    }
}

template <int DT, bool VEC>
__global__ __launch_bounds__(kBlock) void k_norm_backward_narrow(NormBackArgs a) {
    typedef Unit<DT> U;
    constexpr int E = U::elems;
    __shared__ float sums[2][kNarrowRows][16 * E];
    const uint32_t u = threadIdx.x & 15, total = a.rows.start[a.nranks], step = gridDim.x * kNarrowRows;
    const uint32_t pitch = a.cols * uint32_t(sizeof(typename U::T));
    uint32_t row = blockIdx.x * kNarrowRows + (threadIdx.x >> 4);
    int r = 0;
    while (r + 1 < a.nranks && row >= a.rows.start[r + 1]) r++;
    float dw[E], db[E];
#pragma unroll
    for (int e = 0; e < E; e++) dw[e] = db[e] = 0.f;
    if (row < total) {
        const U w = narrow_unit<DT, VEC>(a.weight[r], 0, pitch, u);
        uint64_t local = row - a.rows.start[r];
        U x = narrow_unit<DT, VEC>(a.x[r], local, pitch, u), d = narrow_unit<DT, VEC>(a.dy[r], local, pitch, u);
        float mean = a.mean[r][local], rstd = a.rstd[r][local];
        const float inv = 1.f / float(a.cols);
        while (row < total) {
            float n[E], g[E], s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int e = 0; e < E; e++) {
                // past the row's end dy is 0, and nothing is added to any sum
                const float dy = d.get(e);
                n[e] = (x.get(e) - mean) * rstd;
                g[e] = dy * w.get(e);
                s1 += g[e];
                s2 += g[e] * n[e];
                dw[e] += dy * n[e];
                db[e] += dy;
            }
            const int now = r;
            const uint64_t at = local;
            const float scale = rstd;
            row += step;
            if (row < total) {
                while (row >= a.rows.start[r + 1]) r++;
                local = row - a.rows.start[r];
                x = narrow_unit<DT, VEC>(a.x[r], local, pitch, u);
                d = narrow_unit<DT, VEC>(a.dy[r], local, pitch, u);
                mean = a.mean[r][local];
                rstd = a.rstd[r][local];
            }
            const float m1 = sum16(s1) * inv, m2 = sum16(s2) * inv;
            U o;
#pragma unroll
            for (int e = 0; e < E; e++) o.put(e, scale * (g[e] - m1 - n[e] * m2));
            narrow_store<DT, VEC>(a.dx[now], at, pitch, u, o);
        }
    }
    // the workgroup's strip: its 16 groups' sums in order
#pragma unroll
    for (int e = 0; e < E; e++) {
        sums[0][threadIdx.x >> 4][u * E + e] = dw[e];
        sums[1][threadIdx.x >> 4][u * E + e] = db[e];
    }
    __syncthreads();
    float* strip = a.partial + uint64_t(blockIdx.x) * 2 * a.cols;
    for (uint32_t c = threadIdx.x; c < 2 * 16 * E; c += kBlock) {
        const uint32_t which = c / (16 * E), col = c % (16 * E);
        float s = 0.f;
#pragma unroll
        for (uint32_t k = 0; k < kNarrowRows; k++) s += sums[which][k][col];
        if (col < a.cols) strip[which * a.cols + col] = s;
    }
}

// Rows too wide for the registers: a workgroup per row that reads it again for
// each sum, and the columns' sums strip by strip.
template <int DT>
__global__ __launch_bounds__(kBlock) void k_norm_wide(NormArgs a) {
    typedef typename Elem<DT>::type T;
    __shared__ float tmp[2][kBlock / 64];
    const uint32_t row = blockIdx.x;
    const int r = rank_of_row(a.rows, a.nranks, row);
    const uint64_t local = row - a.rows.start[r];
    const uint32_t C = a.cols;
    const T* x = static_cast<const T*>(a.x[r]) + local * C;
    const T* w = static_cast<const T*>(a.weight[r]);
    const T* b = static_cast<const T*>(a.bias[r]);
    T* y = static_cast<T*>(a.y[r]) + local * C;
    float s = 0.f;
    for (uint32_t c = threadIdx.x; c < C; c += kBlock) s += Elem<DT>::get(x[c]);
    const float mean = block_sum<kBlock / 64>(s, tmp[0]) / float(C);
    float q = 0.f;
    for (uint32_t c = threadIdx.x; c < C; c += kBlock) {
        const float d = Elem<DT>::get(x[c]) - mean;
        q += d * d;
    }
    const float var = block_sum<kBlock / 64>(q, tmp[1]) / float(C);
    const float rstd = 1.f / sqrtf(var + a.eps);
    for (uint32_t c = threadIdx.x; c < C; c += kBlock) {
        float v = (Elem<DT>::get(x[c]) - mean) * rstd * Elem<DT>::get(w[c]);
        if (b != nullptr) v += Elem<DT>::get(b[c]);
        y[c] = Elem<DT>::put(v);
    }
    if (threadIdx.x == 0 && a.mean[r] != nullptr) {
        a.mean[r][local] = mean;
        a.rstd[r][local] = rstd;
    }
}

template <int DT>
__global__ __launch_bounds__(kBlock) void k_norm_dx_wide(NormBackArgs a) {
    typedef typename Elem<DT>::type T;
    __shared__ float tmp[2][kBlock / 64];
    const uint32_t row = blockIdx.x;
    const int r = rank_of_row(a.rows, a.nranks, row);
    const uint64_t local = row - a.rows.start[r];
    const uint32_t C = a.cols;
    const T* x = static_cast<const T*>(a.x[r]) + local * C;
    const T* dy = static_cast<const T*>(a.dy[r]) + local * C;
    const T* w = static_cast<const T*>(a.weight[r]);
    T* dx = static_cast<T*>(a.dx[r]) + local * C;
    const float mean = a.mean[r][local], rstd = a.rstd[r][local];
    float s1 = 0.f, s2 = 0.f;
    for (uint32_t c = threadIdx.x; c < C; c += kBlock) {
        const float g = Elem<DT>::get(dy[c]) * Elem<DT>::get(w[c]);
        s1 += g;
        s2 += g * ((Elem<DT>::get(x[c]) - mean) * rstd);
    }
    const float m1 = block_sum<kBlock / 64>(s1, tmp[0]) / float(C);
    const float m2 = block_sum<kBlock / 64>(s2, tmp[1]) / float(C);
    for (uint32_t c = threadIdx.x; c < C; c += kBlock) {
        const float g = Elem<DT>::get(dy[c]) * Elem<DT>::get(w[c]);
        const float n = (Elem<DT>::get(x[c]) - mean) * rstd;
        dx[c] = Elem<DT>::put(rstd * (g - m1 - n * m2));
    }
}

// Strip blockIdx.y of the rows, one column per thread: the strip's share of
// dw and db.
template <int DT>
__global__ __launch_bounds__(kBlock) void k_norm_dw_wide(NormBackArgs a) {
    typedef typename Elem<DT>::type T;
    const uint32_t c = blockIdx.x * kBlock + threadIdx.x;
    if (c >= a.cols) return;
    const uint64_t total = a.rows.start[a.nranks];
    const uint32_t lo = uint32_t(total * blockIdx.y / a.strips);
    const uint32_t hi = uint32_t(total * (blockIdx.y + 1) / a.strips);
    float dw = 0.f, db = 0.f;
    int r = rank_of_row(a.rows, a.nranks, lo);
    for (uint32_t row = lo; row < hi; row++) {
        while (row >= a.rows.start[r + 1]) r++;
        const uint64_t local = row - a.rows.start[r];
        const float g = Elem<DT>::get(static_cast<const T*>(a.dy[r])[local * a.cols + c]);
        const float v = Elem<DT>::get(static_cast<const T*>(a.x[r])[local * a.cols + c]);
        dw += g * ((v - a.mean[r][local]) * a.rstd[r][local]);
        db += g;
    }
    a.partial[(uint64_t(blockIdx.y) * 2) * a.cols + c] = dw;
    a.partial[(uint64_t(blockIdx.y) * 2 + 1) * a.cols + c] = db;
}

// The strips folded in order: 64 columns per workgroup, each of its 16 waves
// takes every 16th strip, then the waves in order; every rank gets the sums.
template <int DT>
__global__ __launch_bounds__(1024) void k_norm_fold(NormBackArgs a) {
    typedef typename Elem<DT>::type T;
    __shared__ float sums[2][16][64];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    float dw = 0.f, db = 0.f;
    if (c < a.cols)
        for (uint32_t s0 = wave; s0 < a.strips; s0 += 16 * 8) {
            float u[8], v[8];  // eight strips' loads go out before the first is added
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const uint32_t s = s0 + 16 * k;
                u[k] = s < a.strips ? a.partial[(uint64_t(s) * 2) * a.cols + c] : 0.f;
                v[k] = s < a.strips ? a.partial[(uint64_t(s) * 2 + 1) * a.cols + c] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 8; k++) {
                dw += u[k];
                db += v[k];
            }
        }
    sums[0][wave][lane] = dw;
    sums[1][wave][lane] = db;
    __syncthreads();
    if (wave >= 2 || c >= a.cols) return;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 16; k++) s += sums[wave][k][lane];
    void* const* out = wave == 0 ? a.dweight : a.dbias;
    for (int r = 0; r < a.nranks; r++)
        if (out[r] != nullptr) static_cast<T*>(out[r])[c] = Elem<DT>::put(s);
}

// How a row of `cols` elements is held: WPR waves with up to NV units per
// lane.  NV stays small, so that several workgroups share a CU: a row of up to
// 1024 (bf16) or 512 (fp32) elements fits one wave, which then needs no
// exchange between waves at all.
struct Hold {
    int nv, wpr;   // wpr 0: too wide
};
Hold hold(uint32_t units) {
    if (units <= 64) return {1, 1};
    if (units <= 128) return {2, 1};
    if (units <= 256) return {1, 4};
    if (units <= 512) return {2, 4};
    if (units <= 1024) return {4, 4};
    if (units <= 2048) return {2, 16};
    if (units <= 4096) return {4, 16};
    return {0, 0};
}
// run(constant NV, constant WPR)
template <typename F>
void with_hold(Hold h, F&& run) {
#define DT_HOLD(n, w) \
    if (h.nv == n && h.wpr == w) return run(std::integral_constant<int, n>(), std::integral_constant<int, w>())
    DT_HOLD(1, 1);
    DT_HOLD(2, 1);
    DT_HOLD(1, 4);
    DT_HOLD(2, 4);
    DT_HOLD(4, 4);
    DT_HOLD(2, 16);
    DT_HOLD(4, 16);
#undef DT_HOLD
}

// Workgroups that walk over the rows, from sweeps on 16 MiB .. 512 MiB of data.
// Forward: rows held in up to two units per lane run best with many
// workgroups (32768 x 4096 bf16: 512 workgroups 136 us, 2048 111, 4096 101);
// larger holds with two per CU, all resident at once (8 x 4096 rows of 8192
// bf16: 512 191 us, 768 199, 1024 222).
uint32_t forward_workgroups(uint32_t rows, Hold h) {
    const uint32_t need = h.wpr == 1 ? (rows + 3) / 4 : rows, most = h.nv <= 2 && h.wpr <= 4 ? 4096 : 512;
    return need < most ? need : most;
}
// Backward: every workgroup costs a strip of partial sums, written and read
// again.  Two workgroups per CU (32768 x 4096 bf16: 512 146 us, 768 159, 256
// 191), four where the strips are short and the rows many (262144 x 512: 1024
// 139 us, 512 150), one where they are long.
uint32_t backward_workgroups(uint32_t rows, Hold h) {
    const uint32_t need = h.wpr == 1 ? (rows + 3) / 4 : rows;
    uint32_t most = h.wpr == 16 ? 256 : 512;
    if (h.wpr <= 4 && h.nv == 1 && need >= 16 * 1024) most = 1024;
    if (need < 4 * most) most = (need + 3) / 4;  // at least four rows (2000 x 1001 fp32: 19 us; two 20, eight 22)
    return need < most ? need : most;
}
constexpr uint32_t kMostStrips = 1024;

bool aligned(const void* const* list, int n) {
    for (int r = 0; r < n; r++)
        if (reinterpret_cast<uintptr_t>(list[r]) % 16 != 0) return false;
    return true;
}

template <int DT, bool VEC>
hipError_t norm(const NormArgs& a, hipStream_t s) {
    const uint32_t rows = a.rows.start[a.nranks];
    const uint32_t units = (a.cols + Unit<DT>::elems - 1) / Unit<DT>::elems;
    const Hold h = hold(units);
    if (units <= 16) {
        const uint32_t need = (rows + kNarrowRows - 1) / kNarrowRows;
        hipLaunchKernelGGL((k_norm_narrow<DT, VEC>), dim3(need < 4096 ? need : 4096), dim3(kBlock), 0, s, a);
    } else if (h.wpr == 0) {
        hipLaunchKernelGGL(k_norm_wide<DT>, dim3(rows), dim3(kBlock), 0, s, a);
    } else {
        with_hold(h, [&](auto nv, auto wpr) {
            constexpr int W = decltype(wpr)::value;
            hipLaunchKernelGGL((k_norm<DT, VEC, decltype(nv)::value, W>), dim3(forward_workgroups(rows, h)), dim3(Group<W>::threads), 0, s, a);
        });
    }
    return hipGetLastError();
}

template <int DT, bool VEC>
hipError_t norm_backward(NormBackArgs a, hipStream_t s) {
    const uint32_t rows = a.rows.start[a.nranks];
    const uint32_t units = (a.cols + Unit<DT>::elems - 1) / Unit<DT>::elems;
    const Hold h = hold(units);
    a.strips = 0;
    if (rows > 0 && units <= 16) {
        const uint32_t need = (rows + kNarrowRows - 1) / kNarrowRows;
        a.strips = need < kMostStrips ? need : kMostStrips;
        hipLaunchKernelGGL((k_norm_backward_narrow<DT, VEC>), dim3(a.strips), dim3(kBlock), 0, s, a);
    } else if (rows > 0 && h.wpr == 0) {
        a.strips = rows < 256 ? rows : 256;
        hipLaunchKernelGGL(k_norm_dx_wide<DT>, dim3(rows), dim3(kBlock), 0, s, a);
        hipLaunchKernelGGL(k_norm_dw_wide<DT>, dim3((a.cols + kBlock - 1) / kBlock, a.strips), dim3(kBlock), 0, s, a);
    } else if (rows > 0) {
        with_hold(h, [&](auto nv, auto wpr) {
            constexpr int W = decltype(wpr)::value;
            a.strips = backward_workgroups(rows, h);
            hipLaunchKernelGGL((k_norm_backward<DT, VEC, decltype(nv)::value, W>), dim3(a.strips), dim3(Group<W>::threads), 0, s, a);
        });
    }
    hipLaunchKernelGGL(k_norm_fold<DT>, dim3((a.cols + 63) / 64), dim3(1024), 0, s, a);
    return hipGetLastError();
}

bool rows_aligned(uint32_t cols, int dtype) { return cols * uint64_t(dtype == kBF16 ? 2 : 4) % 16 == 0; }

}  // namespace

hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s) {
    const bool vec = rows_aligned(a.cols, dtype) && aligned(a.x, a.nranks) && aligned(a.y, a.nranks) &&
                     aligned(a.weight, a.nranks) && aligned(a.bias, a.nranks);
    if (dtype == kBF16) return vec ? norm<kBF16, true>(a, s) : norm<kBF16, false>(a, s);
    return vec ? norm<kF32, true>(a, s) : norm<kF32, false>(a, s);
}

uint32_t norm_strips(uint32_t rows, uint32_t) { return rows < kMostStrips ? rows : kMostStrips; }

hipError_t launch_norm_backward(const NormBackArgs& a, int dtype, hipStream_t s) {
    const bool vec = rows_aligned(a.cols, dtype) && aligned(a.x, a.nranks) && aligned(a.dy, a.nranks) &&
                     aligned(a.dx, a.nranks) && aligned(a.weight, a.nranks);
    if (dtype == kBF16) return vec ? norm_backward<kBF16, true>(a, s) : norm_backward<kBF16, false>(a, s);
    return vec ? norm_backward<kF32, true>(a, s) : norm_backward<kF32, false>(a, s);
}

}  // namespace dt
