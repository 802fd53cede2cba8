// norm.hip -- layer norm over the rows of all ranks, forward and backward.
//
//   mu = sum_i x_i / C      v = sum_i (x_i - mu)^2 / C      r = 1 / sqrt(v + eps)
//   n_i = (x_i - mu) r      y_i = n_i w_i + b_i
//   dx_i = r (g_i - mean(g) - n_i mean(g n)),   g_i = dy_i w_i
//   dw_i = sum over all rows of dy_i n_i,       db_i = sum over all rows of dy_i
//
// The variance is taken from the centred values (not from sums of squares),
// so a large mean costs no digits.  All sums are fp32; y, dx, dw and db are
// rounded once.  The weight's gradient is the sum over the rows of every
// rank, folded in a fixed order, and goes to every rank: the AllReduce of
// the ranks' partial gradients in the same pass.
#include "dt_step_device.h"

namespace dt {
namespace {

constexpr int kNormWaves = kBlock / 64;

template <int DT>
__global__ __launch_bounds__(kBlock) void k_norm(NormArgs a) {
    typedef typename Elem<DT>::type T;
    __shared__ float tmp[2][kNormWaves];
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
    const float mean = block_sum<kNormWaves>(s, tmp[0]) / float(C);
    float q = 0.f;
    for (uint32_t c = threadIdx.x; c < C; c += kBlock) {
        const float d = Elem<DT>::get(x[c]) - mean;
        q += d * d;
    }
    const float var = block_sum<kNormWaves>(q, tmp[1]) / float(C);
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
__global__ __launch_bounds__(kBlock) void k_norm_dx(NormBackArgs a) {
    typedef typename Elem<DT>::type T;
    __shared__ float tmp[2][kNormWaves];
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
    const float m1 = block_sum<kNormWaves>(s1, tmp[0]) / float(C);
    const float m2 = block_sum<kNormWaves>(s2, tmp[1]) / float(C);
    for (uint32_t c = threadIdx.x; c < C; c += kBlock) {
        const float g = Elem<DT>::get(dy[c]) * Elem<DT>::get(w[c]);
        const float n = (Elem<DT>::get(x[c]) - mean) * rstd;
        dx[c] = Elem<DT>::put(rstd * (g - m1 - n * m2));
    }
}

// Strip blockIdx.y of the rows, one column per thread: the strip's share of
// dw and db.
template <int DT>
__global__ __launch_bounds__(kBlock) void k_norm_dw(NormBackArgs a) {
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

// The strips folded in order; every rank gets the sum.
template <int DT>
__global__ __launch_bounds__(kBlock) void k_norm_fold(NormBackArgs a) {
    typedef typename Elem<DT>::type T;
    const uint32_t c = blockIdx.x * kBlock + threadIdx.x;
    if (c >= a.cols) return;
    float dw = 0.f, db = 0.f;
    for (uint32_t s = 0; s < a.strips; s++) {
        dw += a.partial[(uint64_t(s) * 2) * a.cols + c];
        db += a.partial[(uint64_t(s) * 2 + 1) * a.cols + c];
    }
    for (int r = 0; r < a.nranks; r++) {
        static_cast<T*>(a.dweight[r])[c] = Elem<DT>::put(dw);
        if (a.dbias[r] != nullptr) static_cast<T*>(a.dbias[r])[c] = Elem<DT>::put(db);
    }
}

template <int DT>
hipError_t norm_backward(const NormBackArgs& a, hipStream_t s) {
    const uint32_t rows = a.rows.start[a.nranks];
    const uint32_t colblocks = (a.cols + kBlock - 1) / kBlock;
    if (rows > 0) {
        hipLaunchKernelGGL(k_norm_dx<DT>, dim3(rows), dim3(kBlock), 0, s, a);
        hipLaunchKernelGGL(k_norm_dw<DT>, dim3(colblocks, a.strips), dim3(kBlock), 0, s, a);
    }
    hipLaunchKernelGGL(k_norm_fold<DT>, dim3(colblocks), dim3(kBlock), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s) {
    const uint32_t rows = a.rows.start[a.nranks];
    if (dtype == kBF16) hipLaunchKernelGGL(k_norm<kBF16>, dim3(rows), dim3(kBlock), 0, s, a);
    else hipLaunchKernelGGL(k_norm<kF32>, dim3(rows), dim3(kBlock), 0, s, a);
    return hipGetLastError();
}

uint32_t norm_strips(uint32_t rows, uint32_t) { return rows < 256 ? rows : 256; }

hipError_t launch_norm_backward(const NormBackArgs& a, int dtype, hipStream_t s) {
    return dtype == kBF16 ? norm_backward<kBF16>(a, s) : norm_backward<kF32>(a, s);
}

}  // namespace dt
