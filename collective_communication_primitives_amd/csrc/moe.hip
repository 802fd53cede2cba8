// moe.hip -- routing of tokens to experts and the token exchange between the
// ranks' tokens and the experts' ranks, forward and backward.
//
// Routing, per token with logits x_e:
//   s_e = softmax(x)_e or 1 / (1 + exp(-x_e));   c_e = s_e + bias_e
//   a group's score is the sum of its two largest c; the topk_groups best
//   groups stay; the topk largest c in them are chosen, in descending order,
//   the lowest index first among equals;   w_j = scale * s_j (/ sum of the
//   chosen s when renormalised).
// A logit (or bias) of -inf or NaN takes its expert out; +inf counts as the
// largest finite value.  Slots that no expert is left for hold expert -1 and
// weight 0.
//
// The choice has to be that of the exact scores: candidates are ordered by
// the logits themselves where there is no bias (both scores are strictly
// monotone), and by 64-bit scores where there is one.
#include "dt_step_device.h"

namespace dt {
namespace {

__device__ __forceinline__ double shfl_xor_d(double v, int m) {
    const uint64_t u = __double_as_longlong(v);
    const uint32_t lo = __shfl_xor(uint32_t(u), m), hi = __shfl_xor(uint32_t(u >> 32), m);
    return __longlong_as_double(int64_t(uint64_t(hi) << 32 | lo));
}

// The largest key over the wave and the lowest index among equals; a lane
// without a candidate passes index UINT32_MAX.
__device__ __forceinline__ void wave_argmax(double& key, uint32_t& idx) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
        const double k2 = shfl_xor_d(key, m);
        const uint32_t i2 = __shfl_xor(idx, m);
        const bool take = idx == UINT32_MAX || (i2 != UINT32_MAX && (k2 > key || (k2 == key && i2 < idx)));
        if (i2 != UINT32_MAX && take) {
            key = k2;
            idx = i2;
        }
    }
}

// One wave per token; lane l holds experts l, l + 64, ...
template <int DT, int NV>
__global__ __launch_bounds__(kBlock) void k_route(RouteArgs a, int nranks) {
    typedef typename Elem<DT>::type T;
    const uint32_t row = blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6);
    if (row >= a.rows.start[nranks]) return;
    const uint32_t lane = threadIdx.x & 63;
    const int r = rank_of_row(a.rows, nranks, row);
    const uint64_t local = row - a.rows.start[r];
    const T* x = static_cast<const T*>(a.logits[r]) + local * a.nexperts;
    float v[NV];
    double c[NV];
    bool live[NV];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const uint32_t e = lane + 64 * i;
        v[i] = e < a.nexperts ? Elem<DT>::get(x[e]) : -INFINITY;
        live[i] = v[i] > -INFINITY;  // false for NaN
        v[i] = live[i] ? fminf(v[i], 3.402823466e38f) : -INFINITY;
        if (live[i] && a.bias != nullptr) live[i] = a.bias[e] > -INFINITY;
        top = fmaxf(top, v[i]);
    }
    top = wave_max(top);
    float total = 0.f;
    double totald = 0.;
    if (!a.sigmoid) {
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (v[i] > -INFINITY) {
                total += expf(v[i] - top);
                totald += exp(double(v[i]) - double(top));
            }
        total = wave_sum(total);
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) totald += shfl_xor_d(totald, m);
    }
    const bool scored = a.bias != nullptr || a.groups > 1;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const uint32_t e = lane + 64 * i;
        c[i] = double(v[i]);
        if (scored && live[i]) {
            c[i] = a.sigmoid ? 1. / (1. + exp(-double(v[i]))) : exp(double(v[i]) - double(top)) / totald;
            if (a.bias != nullptr) c[i] += double(a.bias[e]);
        }
    }
    if (a.groups > 1) {
        const uint32_t per = a.nexperts / a.groups;
        // lane g keeps group g's score and whether it stays
        double score = 0.;
        bool any = false;
        for (uint32_t g = 0; g < a.groups; g++) {
            double sum = 0.;
            uint32_t first = UINT32_MAX;
            bool got = false;
            for (int k = 0; k < 2; k++) {
                double key = 0.;
                uint32_t idx = UINT32_MAX;
#pragma unroll
                for (int i = 0; i < NV; i++) {
                    const uint32_t e = lane + 64 * i;
                    if (live[i] && e / per == g && e != first && (idx == UINT32_MAX || c[i] > key)) {
                        key = c[i];
                        idx = e;
                    }
                }
                wave_argmax(key, idx);
                if (idx != UINT32_MAX) {
                    sum += key;
                    got = true;
                }
                first = idx;
            }
            if (lane == g) {
                score = sum;
                any = got;
            }
        }
        uint64_t stay = 0;
        for (uint32_t k = 0; k < a.topk_groups; k++) {
            double key = score;
            uint32_t idx = lane < a.groups && any && !(stay >> lane & 1) ? lane : UINT32_MAX;
            wave_argmax(key, idx);
            if (idx == UINT32_MAX) break;
            stay |= 1ull << idx;
        }
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const uint32_t e = lane + 64 * i;
            if (live[i] && !(stay >> (e / per) & 1)) live[i] = false;
            if (a.bias == nullptr) c[i] = double(v[i]);  // the logits' own order within the groups that stay
        }
    }
    // lane j keeps choice j
    uint32_t mine = UINT32_MAX;
    float mylogit = 0.f;
    for (uint32_t k = 0; k < a.topk; k++) {
        double key = 0.;
        uint32_t idx = UINT32_MAX;
        float logit = 0.f;
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (live[i] && (idx == UINT32_MAX || c[i] > key)) {
                key = c[i];
                idx = lane + 64 * i;
            }
        wave_argmax(key, idx);
        if (idx == UINT32_MAX) break;
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (idx == lane + 64 * i) {
                live[i] = false;
                logit = v[i];
            }
        logit = __shfl(logit, int(idx & 63));
        if (lane == k) {
            mine = idx;
            mylogit = logit;
        }
    }
    const bool has = mine != UINT32_MAX;
    float s;
    if (a.renormalize) {
        // softmax: exp(x - max) over the chosen, the normaliser cancels; sigmoid: s over
        // their sum, and exp(x - max) too where the scores underflow
        const float ctop = wave_max(has ? mylogit : -INFINITY);
        s = has ? expf(mylogit - ctop) : 0.f;
        if (a.sigmoid && ctop > -60.f) s = has ? 1.f / (1.f + expf(-mylogit)) : 0.f;
        const float sum = wave_sum(s);
        s = has ? s / sum : 0.f;
    } else {
        s = !has ? 0.f : a.sigmoid ? 1.f / (1.f + expf(-mylogit)) : expf(mylogit - top) / total;
    }
    if (lane < a.topk) {
        a.experts[r][local * a.topk + lane] = has ? int32_t(mine) : -1;
        a.weights[r][local * a.topk + lane] = s * a.scale;
    }
}

// dlogits of the weights' gradient g_j = dL/dw_j, with a_j the weight before
// the scale and g'_j = scale g_j:
//   renormalised: t_j = a_j (g'_j - sum_i g'_i a_i); softmax: dx_{e_j} += t_j
//                 (the normaliser cancels), sigmoid: dx_{e_j} += t_j (1 - s_j)
//   otherwise:    softmax: dx_e = s_e (sum_{j: e_j = e} g'_j - sum_i g'_i s_i),
//                 sigmoid: dx_{e_j} += g'_j s_j (1 - s_j)
template <int DT, int NV>
__global__ __launch_bounds__(kBlock) void k_route_backward(RouteBackArgs a, int nranks) {
    typedef typename Elem<DT>::type T;
    const uint32_t row = blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6);
    if (row >= a.rows.start[nranks]) return;
    const uint32_t lane = threadIdx.x & 63;
    const int r = rank_of_row(a.rows, nranks, row);
    const uint64_t local = row - a.rows.start[r];
    const T* x = static_cast<const T*>(a.logits[r]) + local * a.nexperts;
    T* dx = static_cast<T*>(a.dlogits[r]) + local * a.nexperts;
    float v[NV];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const uint32_t e = lane + 64 * i;
        v[i] = e < a.nexperts ? Elem<DT>::get(x[e]) : -INFINITY;
        v[i] = v[i] > -INFINITY ? fminf(v[i], 3.402823466e38f) : -INFINITY;
        top = fmaxf(top, v[i]);
    }
    top = wave_max(top);
    float total = 0.f;
    if (!a.sigmoid && !a.renormalize) {
#pragma unroll
        for (int i = 0; i < NV; i++) total += v[i] > -INFINITY ? expf(v[i] - top) : 0.f;
        total = wave_sum(total);
    }
    // lane j: choice j's logit and gradient
    int32_t e = lane < a.topk ? a.experts[r][local * a.topk + lane] : -1;
    float g = 0.f, logit = -INFINITY;
    if (e >= 0 && uint32_t(e) < a.nexperts) {
        g = a.dweights[r][local * a.topk + lane] * a.scale;
        const float l = Elem<DT>::get(x[e]);
        logit = l > -INFINITY ? fminf(l, 3.402823466e38f) : -INFINITY;
    }
    const bool has = logit > -INFINITY;
    if (!has) {
        g = 0.f;
        e = -1;
    }
    float t;  // what choice j adds to its expert
    float all = 0.f;
    if (a.renormalize) {
        const float ctop = wave_max(logit);
        float s = has ? expf(logit - ctop) : 0.f;
        if (a.sigmoid && ctop > -60.f) s = has ? 1.f / (1.f + expf(-logit)) : 0.f;
        const float sum = wave_sum(s);
        const float w = has ? s / sum : 0.f;
        t = w * (g - wave_sum(g * w));
        if (a.sigmoid && has) t *= 1.f / (1.f + expf(logit));
    } else if (a.sigmoid) {
        t = has ? g / (1.f + expf(-logit)) / (1.f + expf(logit)) : 0.f;
    } else {
        const float s = has ? expf(logit - top) / total : 0.f;
        all = wave_sum(g * s);
        t = g;
    }
    float d[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) d[i] = 0.f;
    for (uint32_t k = 0; k < a.topk; k++) {
        const int32_t ek = __shfl(e, int(k));
        const float tk = __shfl(t, int(k));
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (ek == int32_t(lane + 64 * i)) d[i] += tk;
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const uint32_t c = lane + 64 * i;
        if (c >= a.nexperts) continue;
        if (!a.sigmoid && !a.renormalize) d[i] = v[i] > -INFINITY ? expf(v[i] - top) / total * (d[i] - all) : 0.f;
        dx[c] = Elem<DT>::put(d[i]);
    }
}

// --------------------------------------------------------------- exchange --
// The plan is a stable counting sort of the slots by expert, over all ranks:
// count per workgroup, scan, place.  Slot order (rank, token, choice) is kept
// within an expert, so the rows' order does not depend on timing.
__device__ __forceinline__ int32_t slot_expert(const PlanArgs& a, uint64_t slot, uint64_t slots) {
    if (slot >= slots) return -1;
    const uint32_t row = uint32_t(slot / a.topk);
    const int r = rank_of_row(a.rows, a.nranks, row);
    const int32_t e = a.experts[r][slot - uint64_t(a.rows.start[r]) * a.topk];
    return e >= 0 && uint32_t(e) < a.nexperts ? e : -1;
}

__global__ __launch_bounds__(kBlock) void k_plan_count(PlanArgs a) {
    __shared__ uint32_t hist[DT_MAX_EXPERTS];
    const uint64_t slots = uint64_t(a.rows.start[a.nranks]) * a.topk;
    for (uint32_t e = threadIdx.x; e < a.nexperts; e += kBlock) hist[e] = 0;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < kPlanSlots; i += kBlock) {
        const int32_t e = slot_expert(a, uint64_t(blockIdx.x) * kPlanSlots + i, slots);
        if (e >= 0) atomicAdd(&hist[e], 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.nexperts; e += kBlock) a.counts[uint64_t(blockIdx.x) * a.nexperts + e] = hist[e];
}

// One workgroup: counts[b][e] becomes the row, in the expert's rank, of the
// first slot of workgroup b for expert e; offsets get the experts' first rows.
__global__ __launch_bounds__(1024) void k_plan_scan(PlanArgs a, uint32_t blocks) {
    __shared__ uint32_t total[DT_MAX_EXPERTS];
    const uint32_t e = threadIdx.x;
    uint32_t sum = 0;
    if (e < a.nexperts)
        for (uint32_t b = 0; b < blocks; b++) sum += a.counts[uint64_t(b) * a.nexperts + e];
    total[e] = sum;
    __syncthreads();
    if (e >= a.nexperts) return;
    const uint32_t q = e / a.per_rank;
    uint32_t base = 0;
    for (uint32_t f = q * a.per_rank; f < e; f++) base += total[f];
    const uint32_t cap = a.capacity[q];
    a.offsets[q][e - q * a.per_rank] = int32_t(base < cap ? base : cap);
    if (e + 1 == (q + 1) * a.per_rank) a.offsets[q][a.per_rank] = int32_t(base + sum < cap ? base + sum : cap);
    for (uint32_t b = 0; b < blocks; b++) {
        const uint64_t at = uint64_t(b) * a.nexperts + e;
        const uint32_t n = a.counts[at];
        a.counts[at] = base;
        base += n;
    }
}

// Each wave takes a quarter of the workgroup's slots, 64 at a time in order;
// a slot's row is its expert's next row plus the equal experts in lower lanes.
__global__ __launch_bounds__(kBlock) void k_plan_place(PlanArgs a) {
    __shared__ uint32_t next[kBlock / 64][DT_MAX_EXPERTS];
    const uint64_t slots = uint64_t(a.rows.start[a.nranks]) * a.topk;
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    constexpr uint32_t kPer = kPlanSlots / (kBlock / 64);
    for (uint32_t e = threadIdx.x; e < a.nexperts; e += kBlock)
        for (int w = 0; w < kBlock / 64; w++) next[w][e] = 0;
    __syncthreads();
    const uint64_t first = uint64_t(blockIdx.x) * kPlanSlots + wave * kPer;
    for (uint32_t i = lane; i < kPer; i += 64) {
        const int32_t e = slot_expert(a, first + i, slots);
        if (e >= 0) atomicAdd(&next[wave][e], 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.nexperts; e += kBlock) {
        uint32_t at = a.counts[uint64_t(blockIdx.x) * a.nexperts + e];
        for (int w = 0; w < kBlock / 64; w++) {
            const uint32_t n = next[w][e];
            next[w][e] = at;
            at += n;
        }
    }
    __syncthreads();
    for (uint32_t i = lane; i < kPer; i += 64) {
        const uint64_t slot = first + i;
        const int32_t e = slot_expert(a, slot, slots);
        uint64_t same = __ballot(e >= 0);
        for (uint32_t b = 1; b < a.nexperts; b <<= 1) {
            const uint64_t set = __ballot(e >= 0 && (uint32_t(e) & b));
            same &= (uint32_t(e) & b) ? set : ~set;
        }
        const uint32_t before = uint32_t(__popcll(same & ((1ull << lane) - 1)));
        uint32_t pos = 0;
        if (e >= 0) pos = next[wave][e] + before;
        __builtin_amdgcn_wave_barrier();
        if (e >= 0 && before == 0) next[wave][e] += uint32_t(__popcll(same));
        __builtin_amdgcn_wave_barrier();
        if (slot < slots) {
            const int r = rank_of_row(a.rows, a.nranks, uint32_t(slot / a.topk));
            const bool kept = e >= 0 && pos < a.capacity[uint32_t(e) / a.per_rank];
            a.positions[r][slot - uint64_t(a.rows.start[r]) * a.topk] = kept ? int32_t(pos) : -1;
        }
    }
}

// Where slot j of a token lives: the owner rank and its row, or no row at all.
__device__ __forceinline__ bool slot_row(const ExchangeRowsArgs& a, int r, uint64_t slot, uint32_t& q, uint32_t& pos) {
    const int32_t e = a.experts[r][slot], p = a.positions[r][slot];
    if (e < 0 || uint32_t(e) >= a.nexperts || p < 0) return false;
    q = uint32_t(e) / a.per_rank;
    pos = uint32_t(p);
    return pos < a.capacity[q];
}

template <typename T>
__global__ __launch_bounds__(kBlock) void k_dispatch_rows(ExchangeRowsArgs a) {
    const uint32_t row = blockIdx.x;
    const int r = rank_of_row(a.rows, a.nranks, row);
    const uint64_t local = row - a.rows.start[r];
    const T* src = static_cast<const T*>(a.tokens_in[r]) + local * a.cols;
    for (uint32_t j = 0; j < a.topk; j++) {
        uint32_t q, pos;
        if (!slot_row(a, r, local * a.topk + j, q, pos)) continue;
        T* dst = static_cast<T*>(a.rows_out[q]) + uint64_t(pos) * a.cols;
        for (uint32_t c = threadIdx.x; c < a.cols; c += kBlock) dst[c] = src[c];
    }
}

// out[t] = sum_j w_tj y[owner][pos_tj], in slot order, fp32, one rounding.
template <int DT>
__global__ __launch_bounds__(kBlock) void k_combine(ExchangeRowsArgs a) {
    typedef typename Elem<DT>::type T;
    const uint32_t row = blockIdx.x;
    const int r = rank_of_row(a.rows, a.nranks, row);
    const uint64_t local = row - a.rows.start[r];
    T* out = static_cast<T*>(a.tokens_out[r]) + local * a.cols;
    for (uint32_t c = threadIdx.x; c < a.cols; c += kBlock) {
        float s = 0.f;
        for (uint32_t j = 0; j < a.topk; j++) {
            uint32_t q, pos;
            if (!slot_row(a, r, local * a.topk + j, q, pos)) continue;
            const float w = a.weights[r] != nullptr ? a.weights[r][local * a.topk + j] : 1.f;
            s += w * Elem<DT>::get(static_cast<const T*>(a.rows_in[q])[uint64_t(pos) * a.cols + c]);
        }
        out[c] = Elem<DT>::put(s);
    }
}

// dy[owner][pos] = w dout[t];  dw = <dout[t], y[owner][pos]>.
template <int DT>
__global__ __launch_bounds__(kBlock) void k_combine_backward(ExchangeRowsArgs a) {
    typedef typename Elem<DT>::type T;
    __shared__ float tmp[kBlock / 64];
    const uint32_t row = blockIdx.x;
    const int r = rank_of_row(a.rows, a.nranks, row);
    const uint64_t local = row - a.rows.start[r];
    const T* g = static_cast<const T*>(a.tokens_in[r]) + local * a.cols;
    for (uint32_t j = 0; j < a.topk; j++) {
        uint32_t q, pos;
        const uint64_t slot = local * a.topk + j;
        if (!slot_row(a, r, slot, q, pos)) {
            if (threadIdx.x == 0) a.dweights[r][slot] = 0.f;
            continue;
        }
        const float w = a.weights[r][slot];
        const T* y = static_cast<const T*>(a.rows_in[q]) + uint64_t(pos) * a.cols;
        T* dy = static_cast<T*>(a.rows_out[q]) + uint64_t(pos) * a.cols;
        float s = 0.f;
        for (uint32_t c = threadIdx.x; c < a.cols; c += kBlock) {
            const float gc = Elem<DT>::get(g[c]);
            s += gc * Elem<DT>::get(y[c]);
            dy[c] = Elem<DT>::put(w * gc);
        }
        s = block_sum<kBlock / 64>(s, tmp);
        if (threadIdx.x == 0) a.dweights[r][slot] = s;
        __syncthreads();
    }
}

template <int DT>
hipError_t route(const RouteArgs& a, int nranks, hipStream_t s) {
    const dim3 grid((a.rows.start[nranks] + kBlock / 64 - 1) / (kBlock / 64)), block(kBlock);
    const uint32_t nv = (a.nexperts + 63) / 64;
    if (nv <= 1) hipLaunchKernelGGL((k_route<DT, 1>), grid, block, 0, s, a, nranks);
    else if (nv <= 2) hipLaunchKernelGGL((k_route<DT, 2>), grid, block, 0, s, a, nranks);
    else if (nv <= 4) hipLaunchKernelGGL((k_route<DT, 4>), grid, block, 0, s, a, nranks);
    else if (nv <= 8) hipLaunchKernelGGL((k_route<DT, 8>), grid, block, 0, s, a, nranks);
    else hipLaunchKernelGGL((k_route<DT, 16>), grid, block, 0, s, a, nranks);
    return hipGetLastError();
}
template <int DT>
hipError_t route_backward(const RouteBackArgs& a, int nranks, hipStream_t s) {
    const dim3 grid((a.rows.start[nranks] + kBlock / 64 - 1) / (kBlock / 64)), block(kBlock);
    const uint32_t nv = (a.nexperts + 63) / 64;
    if (nv <= 1) hipLaunchKernelGGL((k_route_backward<DT, 1>), grid, block, 0, s, a, nranks);
    else if (nv <= 2) hipLaunchKernelGGL((k_route_backward<DT, 2>), grid, block, 0, s, a, nranks);
    else if (nv <= 4) hipLaunchKernelGGL((k_route_backward<DT, 4>), grid, block, 0, s, a, nranks);
    else if (nv <= 8) hipLaunchKernelGGL((k_route_backward<DT, 8>), grid, block, 0, s, a, nranks);
    else hipLaunchKernelGGL((k_route_backward<DT, 16>), grid, block, 0, s, a, nranks);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int nranks, int dtype, hipStream_t s) {
    return dtype == kBF16 ? route<kBF16>(a, nranks, s) : route<kF32>(a, nranks, s);
}
hipError_t launch_route_backward(const RouteBackArgs& a, int nranks, int dtype, hipStream_t s) {
    return dtype == kBF16 ? route_backward<kBF16>(a, nranks, s) : route_backward<kF32>(a, nranks, s);
}

hipError_t launch_plan(const PlanArgs& a, hipStream_t s) {
    const uint32_t blocks = plan_blocks(uint64_t(a.rows.start[a.nranks]) * a.topk);
    if (blocks > 0) hipLaunchKernelGGL(k_plan_count, dim3(blocks), dim3(kBlock), 0, s, a);
    hipLaunchKernelGGL(k_plan_scan, dim3(1), dim3(1024), 0, s, a, blocks);
    if (blocks > 0) hipLaunchKernelGGL(k_plan_place, dim3(blocks), dim3(kBlock), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_dispatch_rows(const ExchangeRowsArgs& a, int esize, hipStream_t s) {
    const dim3 grid(a.rows.start[a.nranks]), block(kBlock);
    if (esize == 2) hipLaunchKernelGGL(k_dispatch_rows<uint16_t>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_dispatch_rows<uint32_t>, grid, block, 0, s, a);
    return hipGetLastError();
}
hipError_t launch_combine(const ExchangeRowsArgs& a, int dtype, hipStream_t s) {
    const dim3 grid(a.rows.start[a.nranks]), block(kBlock);
    if (dtype == kBF16) hipLaunchKernelGGL(k_combine<kBF16>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_combine<kF32>, grid, block, 0, s, a);
    return hipGetLastError();
}
hipError_t launch_combine_backward(const ExchangeRowsArgs& a, int dtype, hipStream_t s) {
    const dim3 grid(a.rows.start[a.nranks]), block(kBlock);
    if (dtype == kBF16) hipLaunchKernelGGL(k_combine_backward<kBF16>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_combine_backward<kF32>, grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace dt
