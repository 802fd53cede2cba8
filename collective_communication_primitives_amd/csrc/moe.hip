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
// monotone), and by 64-bit scores where there is one and 32 bits do not tell.
#include <type_traits>

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

constexpr float kBiggest = 3.402823466e38f;
// A logit or bias as it counts: NaN is -inf, +inf the largest finite value.
__device__ __forceinline__ float in_range(float f) { return fminf(fmaxf(f, -INFINITY), kBiggest); }

// What a choice of logit x is in the sum over the chosen, whose largest logit is
// `top`: its score but for a factor that is the same for all of them, exp(-top) for
// softmax and exp(-min(top, 0)) for the sigmoid, so that the largest is not below a
// half and a share keeps its digits where the score itself underflows.
__device__ __forceinline__ float share_of(float x, float top, bool sigmoid) {
    if (!sigmoid) return expf(x - top);
    return x > 0.f ? 1.f / (1.f + expf(-x)) : expf(x - fminf(top, 0.f)) / (1.f + expf(x));
}

// One token per wave, scores in 64 bits: lane l holds experts l, l + 64, ...
// For the shapes that four tokens to a wave do not take: more than 512
// experts, more than 16 choices, and groups unless there are 64, 128, 256 or 512
// experts in groups of a power of two of whole lanes.  An exponential in 64 bits for
// each expert and a 64-bit reduction over the wave for each choice, and two for each
// group: 32768 fp32 tokens with a bias, 6 of 160 experts in 8 groups 243 us, 8 of 96
// in 4 137, 6 of 72 in 8 181, 8 of 1024 310, 17 of 128 136.
template <int DT, int NV>
__global__ __launch_bounds__(kBlock) void k_route_any(RouteArgs a, int nranks) {
    typedef typename Elem<DT>::type T;
    const uint32_t row = blockIdx.x * (kBlock / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
        v[i] = in_range(v[i]);
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
            if (a.bias != nullptr) c[i] += double(in_range(a.bias[e]));
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
        const float ctop = wave_max(has ? mylogit : -INFINITY);
        s = has ? share_of(mylogit, ctop, a.sigmoid) : 0.f;
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

// Floats as integers of the same order (no NaN, no -0), and back: integer
// maxima are one instruction with the lane exchange in it.
__device__ __forceinline__ int32_t ordered(float f) {
    const int32_t i = int32_t(__float_as_uint(f));
    return i ^ int32_t(uint32_t(i >> 31) >> 1);
}
__device__ __forceinline__ float unordered(int32_t i) { return __uint_as_float(uint32_t(i ^ int32_t(uint32_t(i >> 31) >> 1))); }
constexpr int32_t kNone = int32_t(0x807FFFFF);  // ordered(-inf)

// The NL logits of a lane's experts [lane * NL, lane * NL + NL), -inf for
// those that are not there or are NaN.
template <int DT, int NL>
__device__ __forceinline__ void load_logits(const void* base, uint64_t row, uint32_t nexperts, uint32_t first, bool vec, float (&x)[NL]) {
    typedef typename Elem<DT>::type T;
    const T* p = static_cast<const T*>(base) + row * nexperts + first;
    constexpr int E = 16 / int(sizeof(T));
    if (NL >= E && vec && first + NL <= nexperts) {
#pragma unroll
        for (int i = 0; i < NL / E; i++) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(p + i * E);
            T t[E];
            __builtin_memcpy(t, &v, 16);
#pragma unroll
            for (int e = 0; e < E; e++) x[i * E + e] = Elem<DT>::get(t[e]);
        }
    } else {
        // the last expert again instead of a branch around each load
        const T* all = static_cast<const T*>(base) + row * nexperts;
#pragma unroll
        for (int i = 0; i < NL; i++) {
            const uint32_t e = first + i < nexperts ? first + i : nexperts - 1;
            x[i] = Elem<DT>::get(all[e]);
        }
#pragma unroll
        for (int i = 0; i < NL; i++) x[i] = first + i < nexperts ? x[i] : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < NL; i++) x[i] = in_range(x[i]) + 0.f;  // + 0: no -0
}

// The lane's experts' biases.
template <int NL>
__device__ __forceinline__ void load_bias(const float* bias, uint32_t nexperts, uint32_t first, float (&b)[NL]) {
#pragma unroll
    for (int i = 0; i < NL; i++) b[i] = in_range(bias[first + i < nexperts ? first + i : nexperts - 1]);
}

__device__ __forceinline__ int64_t ordered(double f) {
    const int64_t i = __double_as_longlong(f);
    return i ^ int64_t(uint64_t(i >> 63) >> 1);
}
__device__ __forceinline__ double unordered(int64_t i) { return __longlong_as_double(i ^ int64_t(uint64_t(i >> 63) >> 1)); }

// The groups that stay: true in the lanes of one of them.  m1, m2: the lane's
// two largest candidates as ordered integers, `none` where there is none; a
// group is `width` neighbouring lanes, a power of two.  Scores are halved, so
// that the sum of two stays in range.  `margin`: how far the last half score
// that stays, of size `size`, is above the first that goes.
__device__ __forceinline__ bool stays_in(uint32_t topk_groups, uint32_t width, int32_t m1, int32_t m2, int32_t none, float& margin,
                                         float& size) {
    const uint32_t lane = threadIdx.x & 15, group = lane / width;
    uint32_t w = 1;
    over16([&](auto c) {
        const int32_t o1 = int32_t(dpp<decltype(c)::value>(uint32_t(m1))), o2 = int32_t(dpp<decltype(c)::value>(uint32_t(m2)));
        if (w < width) {
            const int32_t low = m1 < o1 ? m1 : o1, second = m2 > o2 ? m2 : o2;
            m2 = low > second ? low : second;
            m1 = o1 > m1 ? o1 : m1;
        }
        w *= 2;
    });
    // one expert left in a group: it alone; none: the group goes
    const float score = m1 == none ? -INFINITY : .5f * unordered(m1) + (m2 == none ? 0.f : .5f * unordered(m2));
    const int32_t key = score > -INFINITY ? ordered(score + 0.f) : none;
    uint32_t better = 0;
    rotations([&](auto c) {
        const int32_t o = int32_t(dpp<decltype(c)::value>(uint32_t(key)));
        const uint32_t og = dpp<decltype(c)::value>(group);
        better += og != group && (o > key || (o == key && og < group)) ? 1 : 0;
    });
    const bool stays = better < topk_groups * width && key != none;
    const float last = -max16(stays ? -score : -INFINITY), next = max16(stays ? -INFINITY : score);
    margin = last - next;
    size = fabsf(last);
    return stays;
}

// The choice for one token by the whole wave, in 64 bits: lane l has experts [l *
// NK, l * NK + NK), lane j gets choice j's expert, UINT32_MAX where none is left.
// The kernel's last waves wait for it, so it is short in time and in code: the 16
// lanes of the token alone, 4 NK experts each, took 10 us.
template <int DT, int NK>
__device__ __forceinline__ uint32_t choose_exactly(const RouteArgs& a, const typename Elem<DT>::type* logits) {
    const uint32_t lane = threadIdx.x & 63, first = lane * NK;
    constexpr int64_t kLowest = INT64_MIN;
    float x[NK], b[NK];
#pragma unroll
    for (int i = 0; i < NK; i++) {
        const uint32_t e = first + i < a.nexperts ? first + i : a.nexperts - 1;
        x[i] = Elem<DT>::get(logits[e]);
        b[i] = a.bias != nullptr ? in_range(a.bias[e]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NK; i++) x[i] = first + i < a.nexperts && x[i] > -INFINITY ? fminf(x[i], kBiggest) + 0.f : -INFINITY;
    const bool scored = a.bias != nullptr || a.groups > 1;
    double sum = 0., top = 0.;
    if (scored && !a.sigmoid) {
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < NK; i++) most = fmaxf(most, x[i]);
        top = double(wave_max(most));
#pragma unroll
        for (int i = 0; i < NK; i++) sum += x[i] > -INFINITY ? exp(double(x[i]) - top) : 0.;
#pragma unroll 1
        for (int m = 1; m < 64; m <<= 1) sum += shfl_xor_d(sum, m);
    }
    int64_t key[NK];
#pragma unroll
    for (int i = 0; i < NK; i++) {
        double v = double(x[i]);
        if (scored) v = a.sigmoid ? 1. / (1. + exp(-v)) : exp(v - top) / sum;
        if (a.bias != nullptr) v += double(b[i]);
        key[i] = x[i] > -INFINITY && b[i] > -INFINITY ? ordered(v + 0.) : kLowest;
    }
    if (a.groups > 1) {
        const uint32_t width = a.nexperts / a.groups / NK, group = lane / width;  // lanes of a group, a power of two
        int64_t m1 = kLowest, m2 = kLowest;
#pragma unroll
        for (int i = 0; i < NK; i++) {
            const int64_t low = m1 < key[i] ? m1 : key[i];
            m2 = low > m2 ? low : m2;
            m1 = key[i] > m1 ? key[i] : m1;
        }
#pragma unroll 1
        for (uint32_t w = 1; w < width; w <<= 1) {
            const int64_t o1 = __shfl_xor(m1, int(w)), o2 = __shfl_xor(m2, int(w));
            const int64_t low = m1 < o1 ? m1 : o1, second = m2 > o2 ? m2 : o2;
            m2 = low > second ? low : second;
            m1 = o1 > m1 ? o1 : m1;
        }
        const double score = m1 == kLowest ? -INFINITY : m2 == kLowest ? unordered(m1) : unordered(m1) + unordered(m2);
        const int64_t mine = m1 != kLowest ? ordered(score + 0.) : kLowest;
        uint32_t better = 0;
#pragma unroll 1
        for (uint32_t g = 0; g < a.groups; g++) {
            const int64_t o = __shfl(mine, int(g * width));
            better += g != group && (o > mine || (o == mine && g < group)) ? 1 : 0;
        }
        const bool stays = better < a.topk_groups && mine != kLowest;
#pragma unroll
        for (int i = 0; i < NK; i++) {
            if (!stays) key[i] = kLowest;
            else if (a.bias == nullptr && key[i] != kLowest) key[i] = ordered(double(x[i]));
        }
    }
    uint32_t mine = UINT32_MAX;
#pragma unroll 1
    for (uint32_t k = 0; k < a.topk; k++) {
        int64_t own = key[0];
        uint32_t at = first;
#pragma unroll
        for (int i = 1; i < NK; i++) {
            at = key[i] > own ? first + i : at;
            own = key[i] > own ? key[i] : own;
        }
        int64_t best = own;
        over16([&](auto c) {
            const uint64_t u = uint64_t(best);
            const int64_t o = int64_t(uint64_t(dpp<decltype(c)::value>(uint32_t(u >> 32))) << 32 | dpp<decltype(c)::value>(uint32_t(u)));
            best = o > best ? o : best;
        });
#pragma unroll
        for (int m = 16; m < 64; m <<= 1) {
            const int64_t o = __shfl_xor(best, m);
            best = o > best ? o : best;
        }
        if (best == kLowest) break;
        const uint32_t from = uint32_t(__builtin_ctzll(__ballot(own == best)));  // experts rise with the lanes
        at = uint32_t(__builtin_amdgcn_readlane(int(at), int(from)));
#pragma unroll
        for (int i = 0; i < NK; i++) key[i] = at == first + i ? kLowest : key[i];
        if (lane == k) mine = at;
    }
    return mine;
}

// Descending by odd-even merging: one maximum and one minimum per comparison.
template <int NL>
__device__ __forceinline__ void sort_down(int32_t (&key)[NL]) {
#pragma unroll
    for (int p = 1; p < NL; p <<= 1)
#pragma unroll
        for (int k = p; k >= 1; k >>= 1)
#pragma unroll
            for (int j = k % p; j + k < NL; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; i++)
                    if (j + i + k < NL && (j + i) / (2 * p) == (j + i + k) / (2 * p)) {
                        const int32_t u = key[j + i], v = key[j + i + k];
                        key[j + i] = u > v ? u : v;
                        key[j + i + k] = u > v ? v : u;
                    }
}

// Four tokens per wave, 16 lanes each; lane l of the 16 holds experts [l * NL, l
// * NL + NL), sorted once; then topk times the largest of the 16 lanes' heads
// is taken off its list.
//
// The keys are 32-bit: the logit, or the score where there is a bias, as an
// ordered integer whose last bits give way to the place in the lane.  The
// chosen ones' uncut values are compared afterwards.  They tell two candidates
// apart unless they are closer than twice `off`, the bound on a 32-bit score's
// error:
//   sigmoid  s (1 - s) (|x| + 2) U <= 0.8 U of the exponential and its argument, U of the
//            sum, 2 U of the reciprocal: under 5 U;
//   softmax, s <= 1:  (2 |d| + 2) s U <= 3 U of the exponential and its argument d = x - max,
//            (NL + 4) U <= 36 U of the sum and 4 U of the quotient: under 48 U;
//   the bias' addition  U |c|, for each of the two that are compared.
// Where two neighbours in the order, the last choice and the one behind it, or
// the last group that stays and the first that goes are that close, the wave
// chooses for that token again in 64 bits: about one token in a thousand of normally
// distributed logits with a bias.
//
// 32768 tokens, 8 of 256 experts, fp32, sigmoid, bias, 8 groups: 30 us (the logits'
// bytes alone are 7), 3 us of it the waves that choose again.  The vector units are
// busy for 67% of it, with 1230 instructions a wave; the rest is latency that too
// few waves hide: 96 registers, most of them choose_exactly's, let 5 of the 8 waves
// that each SIMD gets run at a time.  A wave per token with 64-bit scores
// throughout took 229 us; 16 lanes that scan for each choice 61 us.  Equal logits
// are close calls as well: 8 of 256 experts without groups and bias take 13 us, 49
// where all logits are the same.
template <int DT, int NL>
__global__ __launch_bounds__(kBlock) void k_route(RouteArgs a, int nranks, int vec) {
    typedef typename Elem<DT>::type T;
    const uint32_t total = a.rows.start[nranks], lane = threadIdx.x & 15;
    const uint32_t row0 = blockIdx.x * (kBlock / 16) + (threadIdx.x >> 4);
    const bool there = row0 < total;
    const uint32_t row = there ? row0 : total - 1;  // the last lanes repeat the last token and store nothing
    int r = 0;
    while (r + 1 < nranks && row >= a.rows.start[r + 1]) r++;
    const uint64_t local = row - a.rows.start[r];
    const uint32_t first = lane * NL;
    constexpr float U = 5.9604645e-8f;
    constexpr int32_t kPlace = NL - 1;
    float x[NL];
    int32_t key[NL];
    load_logits<DT, NL>(a.logits[r], local, a.nexperts, first, vec, x);
    const bool scored = a.bias != nullptr || a.groups > 1;
    float top = 0.f, sum = 0.f, off = 0.f;
    bool close = false, stays = true;
    if (scored || (!a.sigmoid && !a.renormalize)) {
        float c[NL];
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < NL; i++) c[i] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x[i] * -kLog2e));
            off = 5.f * U;
        } else {
            float most = x[0];
#pragma unroll
            for (int i = 1; i < NL; i++) most = fmaxf(most, x[i]);
            most = max16(most);
            top = most > -INFINITY ? most : 0.f;
#pragma unroll
            for (int i = 0; i < NL; i++) {
                c[i] = __builtin_amdgcn_exp2f((x[i] - top) * kLog2e);
                sum += c[i];
            }
            sum = sum16(sum);
            const float inv = 1.f / sum;
#pragma unroll
            for (int i = 0; i < NL; i++) c[i] *= inv;
            off = 48.f * U;
        }
        if (scored) {
            // a candidate that is out is -inf, also where the bias is NaN
            float big = 0.f;
            if (a.bias != nullptr) {
                float b[NL];
                load_bias<NL>(a.bias, a.nexperts, first, b);
#pragma unroll
                for (int i = 0; i < NL; i++) c[i] = fmaxf(x[i] > -INFINITY ? c[i] + b[i] : -INFINITY, -INFINITY);
                if (a.groups > 1) {
#pragma unroll
                    for (int i = 0; i < NL; i++) big = fmaxf(big, c[i] > -INFINITY ? fabsf(b[i]) : 0.f);
                }
            } else {
#pragma unroll
                for (int i = 0; i < NL; i++) c[i] = x[i] > -INFINITY ? c[i] : -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < NL; i++) key[i] = ordered(c[i]);
            if (a.groups > 1) {
                int32_t m1 = kNone, m2 = kNone;
#pragma unroll
                for (int i = 0; i < NL; i++) {
                    const int32_t low = m1 < key[i] ? m1 : key[i];
                    m2 = low > m2 ? low : m2;
                    m1 = key[i] > m1 ? key[i] : m1;
                }
                float margin = 0.f, size = 0.f;
                stays = stays_in(a.topk_groups, a.nexperts / a.groups / NL, m1, m2, kNone, margin, size);
                close = margin <= 2.f * (off + U * (1.f + max16(big))) + 2.f * U * size;
            }
        }
    }
    if (a.bias == nullptr) {  // the logits' own order
#pragma unroll
        for (int i = 0; i < NL; i++) key[i] = ordered(x[i]);
    }
    // kNone, also without its last bits, is below every finite value's key
#pragma unroll
    for (int i = 0; i < NL; i++) key[i] = stays ? (key[i] & ~kPlace) | (kPlace - i) : kNone;
    sort_down(key);
    uint32_t mine = UINT32_MAX;
    for (uint32_t k = 0; k < a.topk; k++) {
        const int32_t best = max16(key[0]);
        // the lowest of the lanes with that key, whatever the place in the lane
        const uint32_t equal = uint32_t(__ballot(((key[0] ^ best) & ~kPlace) == 0) >> (threadIdx.x & 48)) & 0xFFFFu;
        const uint32_t from = uint32_t(__builtin_ctz(equal | 0x10000u));
        const uint32_t at = uint32_t(__shfl(int(first + kPlace - (key[0] & kPlace)), int((threadIdx.x & 48) + from)));
        if (lane == k && best > kNone) mine = at;
        // bit selects: written as conditionals the compiler makes them indexed reads of the list
        const int32_t taken = lane == from ? -1 : 0;
#pragma unroll
        for (int i = 0; i + 1 < NL; i++) key[i] = (key[i + 1] & taken) | (key[i] & ~taken);
        key[NL - 1] = (kNone & taken) | (key[NL - 1] & ~taken);
    }
    const T* logits = static_cast<const T*>(a.logits[r]) + local * a.nexperts;
    float logit = mine != UINT32_MAX ? fminf(Elem<DT>::get(logits[mine]), kBiggest) : -INFINITY;
    if (a.bias != nullptr || DT == kF32) {
        // The choices' uncut values side by side, and the most that the best one left may be.  (bf16 logits keep all
        // their bits: equal keys are equal logits.)
        float v = logit;
        if (a.bias != nullptr && mine != UINT32_MAX) {
            v = a.sigmoid ? __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(logit * -kLog2e))
                          : __builtin_amdgcn_exp2f((logit - top) * kLog2e) * (1.f / sum);
            v += in_range(a.bias[mine]);
        }
        const int32_t left = max16(key[0]);
        const float after = dpp<0x101>(v), tail = left > kNone ? unordered(left | kPlace) : -INFINITY;
        const float next = lane + 1 < a.topk ? after : tail;
        close = close || (lane < a.topk && next > -INFINITY && v - next <= 2.f * off + 2.5f * U * fabsf(v));
    }
    for (uint64_t todo = __ballot(close); todo != 0;) {  // one of the wave's tokens at a time
        const uint32_t at = uint32_t(__builtin_ctzll(todo)) & 48;
        todo &= ~(0xFFFFull << at);
        const uint64_t p = reinterpret_cast<uint64_t>(logits);
        const uint64_t lo = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(p)), int(at)));
        const uint64_t hi = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(p >> 32)), int(at)));
        const uint32_t exact = choose_exactly<DT, NL / 4>(a, reinterpret_cast<const T*>(hi << 32 | lo));
        const uint32_t choice = uint32_t(__shfl(int(exact), int(lane)));
        if ((threadIdx.x & 48) == at) mine = choice;
    }
    if (__any(close)) {
        logit = mine != UINT32_MAX ? fminf(Elem<DT>::get(logits[mine]), kBiggest) : -INFINITY;
    }
    const bool has = mine != UINT32_MAX;
    float s;
    if (a.renormalize) {
        const float ctop = max16(logit);
        s = has ? share_of(logit, ctop, a.sigmoid) : 0.f;
        const float all = sum16(s);
        s = has ? s / all : 0.f;
    } else {
        s = !has ? 0.f : a.sigmoid ? 1.f / (1.f + expf(-logit)) : expf(logit - top) / sum;
    }
    if (there && lane < a.topk) {
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
// L lanes per token (16 where topk and the experts fit, else the wave), NL
// neighbouring experts each.  87000 tokens, 6 of 128 experts, bf16, dense: 18 us,
// 2.7 TB/s, bound by the vector unit: 450 instructions per wave, half of
// them the comparisons that bring a choice's gradient to its expert.
template <int L>
__device__ __forceinline__ float sum_lanes(float v) {
    if constexpr (L == 16) return sum16(v);
    else return wave_sum(v);
}
template <int L>
__device__ __forceinline__ float max_lanes(float v) {
    if constexpr (L == 16) return max16(v);
    else return wave_max(v);
}
template <int DT, int NL, int L>
__global__ __launch_bounds__(kBlock) void k_route_backward(RouteBackArgs a, int nranks, int vec) {
    typedef typename Elem<DT>::type T;
    const uint32_t total_rows = a.rows.start[nranks], lane = threadIdx.x % L;
    const uint32_t row0 = blockIdx.x * (kBlock / L) + threadIdx.x / L;
    const bool there = row0 < total_rows;
    const uint32_t row = there ? row0 : total_rows - 1;
    int r = 0;
    while (r + 1 < nranks && row >= a.rows.start[r + 1]) r++;
    const uint64_t local = row - a.rows.start[r];
    const uint32_t first = lane * NL;
    const bool dense = !a.sigmoid && !a.renormalize;
    float s[NL];
    float top = -INFINITY, total = 0.f;
    if (dense) {
        load_logits<DT, NL>(a.logits[r], local, a.nexperts, first, vec, s);
#pragma unroll
        for (int i = 0; i < NL; i++) top = fmaxf(top, s[i]);
        top = max_lanes<L>(top);
#pragma unroll
        for (int i = 0; i < NL; i++) {
            s[i] = s[i] > -INFINITY ? __builtin_amdgcn_exp2f((s[i] - top) * kLog2e) : 0.f;
            total += s[i];
        }
        total = sum_lanes<L>(total);
    }
    // lane j: choice j's logit and gradient
    int32_t e = lane < a.topk ? a.experts[r][local * a.topk + lane] : -1;
    float g = 0.f, logit = -INFINITY;
    if (lane < a.topk) g = a.dweights[r][local * a.topk + lane] * a.scale;
    // dense: the choice's score is in the registers of the lane that holds its expert
    if (!dense && e >= 0 && uint32_t(e) < a.nexperts) {
        const float l = Elem<DT>::get(static_cast<const T*>(a.logits[r])[local * a.nexperts + e]);
        logit = l > -INFINITY ? fminf(l, kBiggest) : -INFINITY;
    }
    const bool has = logit > -INFINITY;
    if (!dense && !has) {
        g = 0.f;
        e = -1;
    }
    float t;  // what choice j adds to its expert
    if (a.renormalize) {
        const float ctop = max_lanes<L>(logit);
        float w = has ? share_of(logit, ctop, a.sigmoid) : 0.f;
        const float sum = sum_lanes<L>(w);
        w = has ? w / sum : 0.f;
        t = w * (g - sum_lanes<L>(g * w));
        if (a.sigmoid && has) t *= 1.f / (1.f + expf(logit));
    } else if (a.sigmoid) {
        t = has ? g / (1.f + expf(-logit)) / (1.f + expf(logit)) : 0.f;
    } else {
        t = g;
    }
    float d[NL];
#pragma unroll
    for (int i = 0; i < NL; i++) d[i] = 0.f;
    auto add = [&](uint32_t ek, float tk) {
        const uint32_t at = ek - first;  // huge when it is not this lane's
#pragma unroll
        for (int i = 0; i < NL; i++) d[i] += at == uint32_t(i) ? tk : 0.f;
    };
    if constexpr (L == 16) {
        broadcasts16([&](auto k, auto c) {
            if (uint32_t(decltype(k)::value) < a.topk) add(dpp<decltype(c)::value>(uint32_t(e)), dpp<decltype(c)::value>(t));
        });
    } else {
        for (uint32_t k = 0; k < a.topk; k++) add(uint32_t(__shfl(e, int(k))), __shfl(t, int(k)));
    }
    if (dense) {
        const float inv = total > 0.f ? 1.f / total : 0.f;
        float all = 0.f;
#pragma unroll
        for (int i = 0; i < NL; i++) {
            s[i] *= inv;
            d[i] = s[i] > 0.f ? d[i] : 0.f;  // an expert that was out has no gradient
            all += s[i] * d[i];
        }
        all = sum_lanes<L>(all);
#pragma unroll
        for (int i = 0; i < NL; i++) d[i] = s[i] * (d[i] - all);
    }
    if (!there || first >= a.nexperts) return;
    T* dx = static_cast<T*>(a.dlogits[r]) + local * a.nexperts + first;
    constexpr int E = 16 / int(sizeof(T));
    if (NL >= E && vec && first + NL <= a.nexperts) {
#pragma unroll
        for (int i = 0; i < NL / E; i++) {
            T o[E];
#pragma unroll
            for (int k = 0; k < E; k++) o[k] = Elem<DT>::put(d[i * E + k]);
            u32x4 v;
            __builtin_memcpy(&v, o, 16);
            *reinterpret_cast<u32x4*>(dx + i * E) = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NL; i++)
            if (first + i < a.nexperts) dx[i] = Elem<DT>::put(d[i]);
    }
}

// --------------------------------------------------------------- exchange --
// The plan is a stable counting sort of the slots by expert, over all ranks.
// Slot order (rank, token, choice) is kept within an expert, so the rows' order
// does not depend on timing.  Two launches, latency-bound: 131072 slots of 64
// experts 7 us of counting and 14 us of placing, of 270 us with the rows.
__device__ __forceinline__ int32_t slot_expert(const PlanArgs& a, uint32_t slot, uint32_t slots) {
    if (slot >= slots) return -1;
    const uint32_t row = slot / a.topk;
    int r = 0;
    while (r + 1 < a.nranks && row >= a.rows.start[r + 1]) r++;
    const int32_t e = a.experts[r][slot - a.rows.start[r] * a.topk];
    return e >= 0 && uint32_t(e) < a.nexperts ? e : -1;
}
__device__ __forceinline__ void store_position(const PlanArgs& a, uint32_t slot, int32_t e, uint32_t pos) {
    const uint32_t row = slot / a.topk;
    int r = 0;
    while (r + 1 < a.nranks && row >= a.rows.start[r + 1]) r++;
    const bool kept = e >= 0 && pos < a.capacity[uint32_t(e) / a.per_rank];
    a.positions[r][slot - a.rows.start[r] * a.topk] = kept ? int32_t(pos) : -1;
}
// total[e]: slots of expert e over all ranks.  Each expert's first row, and the
// end, to its rank's offsets.
__device__ __forceinline__ void store_offsets(const PlanArgs& a, const uint32_t* total) {
    for (uint32_t e = threadIdx.x; e < a.nexperts; e += kBlock) {
        const uint32_t q = e / a.per_rank, cap = a.capacity[q];
        uint32_t base = 0;
        for (uint32_t f = q * a.per_rank; f < e; f++) base += total[f];
        a.offsets[q][e - q * a.per_rank] = int32_t(base < cap ? base : cap);
        base += total[e];
        if (e + 1 == (q + 1) * a.per_rank) a.offsets[q][a.per_rank] = int32_t(base < cap ? base : cap);
    }
}

// counts[b][e]: slots of expert e in workgroup b's share.
__global__ __launch_bounds__(kBlock) void k_plan_count(PlanArgs a) {
    __shared__ uint32_t hist[DT_MAX_EXPERTS];
    const uint32_t slots = a.rows.start[a.nranks] * a.topk;
    for (uint32_t e = threadIdx.x; e < a.nexperts; e += kBlock) hist[e] = 0;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < kPlanSlots; i += kBlock) {
        const int32_t e = slot_expert(a, blockIdx.x * kPlanSlots + i, slots);
        if (e >= 0) atomicAdd(&hist[e], 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.nexperts; e += kBlock) a.counts[uint64_t(blockIdx.x) * a.nexperts + e] = hist[e];
}

// Many workgroups: counts[b][e] becomes the number of expert e's slots in the
// workgroups before b, and row `blocks` of counts their number in all.
__global__ __launch_bounds__(64) void k_plan_scan(PlanArgs a, uint32_t blocks) {
    const uint32_t e = blockIdx.x * 64 + threadIdx.x;
    if (e >= a.nexperts) return;
    uint32_t sum = 0;
    for (uint32_t b0 = 0; b0 < blocks; b0 += 16) {
        uint32_t n[16];
#pragma unroll
        for (int i = 0; i < 16; i++) n[i] = b0 + i < blocks ? a.counts[uint64_t(b0 + i) * a.nexperts + e] : 0;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            if (b0 + i < blocks) a.counts[uint64_t(b0 + i) * a.nexperts + e] = sum;
            sum += n[i];
        }
    }
    a.counts[uint64_t(blocks) * a.nexperts + e] = sum;
}

// Each wave takes a quarter of the workgroup's slots, 64 at a time in order; a
// slot's row is its expert's next row plus the equal experts in lower lanes.
// Without a scan each workgroup adds up the counts before its own by itself.
__global__ __launch_bounds__(kBlock) void k_plan_place(PlanArgs a, uint32_t blocks, int scanned) {
    __shared__ uint32_t next[kBlock / 64][DT_MAX_EXPERTS];
    __shared__ uint32_t total[DT_MAX_EXPERTS];
    const uint32_t slots = a.rows.start[a.nranks] * a.topk;
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    constexpr uint32_t kPer = kPlanSlots / (kBlock / 64);
    for (uint32_t e = threadIdx.x; e < a.nexperts; e += kBlock)
        for (int w = 0; w < kBlock / 64; w++) next[w][e] = 0;
    __syncthreads();
    const uint32_t first = blockIdx.x * kPlanSlots + wave * kPer;
    int32_t ex[kPer / 64];
#pragma unroll
    for (uint32_t i = 0; i < kPer / 64; i++) ex[i] = slot_expert(a, first + i * 64 + lane, slots);
#pragma unroll
    for (uint32_t i = 0; i < kPer / 64; i++)
        if (ex[i] >= 0) atomicAdd(&next[wave][ex[i]], 1u);
    // slots of the experts in the workgroups before this one, and in all
    uint32_t before[DT_MAX_EXPERTS / kBlock];
#pragma unroll
    for (uint32_t i = 0; i < DT_MAX_EXPERTS / kBlock; i++) {
        const uint32_t e = threadIdx.x + i * kBlock;
        before[i] = 0;
        if (e >= a.nexperts) continue;
        uint32_t all = 0;
        if (scanned) {
            before[i] = a.counts[uint64_t(blockIdx.x) * a.nexperts + e];
            all = a.counts[uint64_t(blocks) * a.nexperts + e];
        } else {
            for (uint32_t b0 = 0; b0 < blocks; b0 += 16) {
                uint32_t n[16];
#pragma unroll
                for (int k = 0; k < 16; k++) n[k] = b0 + k < blocks ? a.counts[uint64_t(b0 + k) * a.nexperts + e] : 0;
#pragma unroll
                for (int k = 0; k < 16; k++) {
                    all += n[k];
                    if (b0 + k < blockIdx.x) before[i] += n[k];
                }
            }
        }
        total[e] = all;
    }
    __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < DT_MAX_EXPERTS / kBlock; i++) {
        const uint32_t e = threadIdx.x + i * kBlock;
        if (e >= a.nexperts) continue;
        uint32_t at = before[i];
        for (uint32_t f = e / a.per_rank * a.per_rank; f < e; f++) at += total[f];
        for (int w = 0; w < kBlock / 64; w++) {
            const uint32_t n = next[w][e];
            next[w][e] = at;
            at += n;
        }
    }
    if (blockIdx.x == 0) store_offsets(a, total);
    __syncthreads();
    volatile uint32_t* mine = next[wave];
#pragma unroll
    for (uint32_t i = 0; i < kPer / 64; i++) {
        const int32_t e = ex[i];
        uint64_t same = __ballot(e >= 0);
        for (uint32_t b = 1; b < a.nexperts; b <<= 1) {
            const uint64_t set = __ballot(e >= 0 && (uint32_t(e) & b));
            same &= (uint32_t(e) & b) ? set : ~set;
        }
        const uint32_t before_me = uint32_t(__popcll(same & ((1ull << lane) - 1)));
        uint32_t pos = 0;
        if (e >= 0) pos = mine[e] + before_me;
        __builtin_amdgcn_wave_barrier();
        if (e >= 0 && before_me == 0) mine[e] = pos + uint32_t(__popcll(same));
        __builtin_amdgcn_wave_barrier();
        const uint32_t slot = first + i * 64 + lane;
        if (slot < slots) store_position(a, slot, e, pos);
    }
}

// Where slot j of a token lives: the owner rank and its row, or no row at all.
__device__ __forceinline__ bool slot_row(const ExchangeRowsArgs& a, int32_t e, int32_t p, uint32_t& q, uint32_t& pos) {
    if (e < 0 || uint32_t(e) >= a.nexperts || p < 0) return false;
    q = uint32_t(e) / a.per_rank;
    pos = uint32_t(p);
    return pos < a.capacity[q];
}

// The choices of one token: lane j of the wave knows choice j's row.
struct Choices {
    uint64_t at;     // lane j: the row's address in the expert rank's buffer
    uint64_t kept;   // bit j: choice j has a row (the same in all lanes)
};
__device__ __forceinline__ const char* choice_row(const Choices& c, int j) {
    const uint32_t lo = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(c.at)), j));
    const uint32_t hi = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(c.at >> 32)), j));
    return reinterpret_cast<const char*>(uint64_t(hi) << 32 | lo);
}
template <typename P>
__device__ __forceinline__ Choices choices(const ExchangeRowsArgs& a, P* const (&buffers)[kMaxRanksHost], int r, uint64_t local,
                                           uint32_t pitch) {
    const uint32_t lane = threadIdx.x & 63;
    Choices c = {0, 0};
    bool kept = false;
    if (lane < a.topk) {
        const uint64_t slot = local * a.topk + lane;
        uint32_t q, pos;
        kept = slot_row(a, a.experts[r][slot], a.positions[r][slot], q, pos);
        if (kept) c.at = reinterpret_cast<uint64_t>(buffers[q]) + uint64_t(pos) * pitch;
    }
    c.kept = __ballot(kept);
    return c;
}

// The rows' traffic is bound by memory: 32768 rows of 8 KiB to 4 experts each
// (1.34 GB) take 247 us, 5.4 TB/s.  Each row is read
// once and stored to all its places from registers.
//
// A token's row is worked on by WPT waves (1 for rows of up to 4 KiB, where four
// waves would have less than one load each, else 4), NV units of 16 bytes per
// lane at a time.  VEC: rows start and end on 16-byte
// boundaries; the others are read at their elements' alignment, with a last
// unit that may be partly behind the row's end.
template <int ES, bool VEC>
__device__ __forceinline__ u32x4 load_at(const char* row, uint32_t u, uint32_t bytes) {
    if constexpr (VEC) return load16(row + u * 16);
    else return load_loose<ES>(row, u, bytes);
}
// Written through towards memory, like the fan-out copies.
template <int ES, bool VEC>
__device__ __forceinline__ void store_at(const char* row, uint32_t u, uint32_t bytes, u32x4 v) {
    if constexpr (VEC) bstore16<kPolNT | kPolDevice>(make_rsrc(row, bytes), u * 16, v);
    else store_loose<ES>(const_cast<char*>(row), u, bytes, v);
}

template <int ES, bool VEC, int WPT>
__device__ __forceinline__ void dispatch_row(const char* src, uint32_t bytes, const Choices& c, uint32_t lane) {
    constexpr int NV = 4, L = 64 * WPT;
    const uint32_t units = (bytes + 15) / 16;
    for (uint32_t u0 = lane; u0 < units; u0 += NV * L) {
        u32x4 x[NV];
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (u0 + i * L < units) {
                // with writes dominating, plain loads (247 us against 280 with the non-temporal hint, 8 choices of 4 KiB rows)
                if constexpr (VEC) x[i] = load16_h<false>(src + (u0 + i * L) * 16);
                else x[i] = load_loose<ES>(src, u0 + i * L, bytes);
            }
        for (uint64_t m = c.kept; m != 0; m &= m - 1) {
            const char* to = choice_row(c, __builtin_ctzll(m));
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (u0 + i * L < units) store_at<ES, VEC>(to, u0 + i * L, bytes, x[i]);
        }
    }
}

// The token of this wave (WPT 1) or workgroup, or none.
template <int WPT>
__device__ __forceinline__ uint32_t token_of() {
    return WPT == 1 ? blockIdx.x * (kBlock / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : blockIdx.x;
}

template <int ES, bool VEC, int WPT>
__global__ __launch_bounds__(kBlock) void k_dispatch_rows(ExchangeRowsArgs a) {
    const uint32_t row = token_of<WPT>();
    if (row >= a.rows.start[a.nranks]) return;
    const int r = rank_of_row(a.rows, a.nranks, row);
    const uint64_t local = row - a.rows.start[r];
    const uint32_t pitch = a.cols * ES;
    const Choices c = choices(a, a.rows_out, r, local, pitch);
    dispatch_row<ES, VEC, WPT>(static_cast<const char*>(a.tokens_in[r]) + local * pitch, pitch, c,
                               threadIdx.x % (64 * WPT));
}

// Few slots: plan and copy in one launch.  Every workgroup finds the rows of
// its own tokens' slots by itself, from all slots: slot s of expert e comes
// behind the slots of its rank's lower experts and behind the earlier slots of
// e.  The workgroup behind the last one writes the offsets.  128 tokens of 8 KiB to
// 4 of 64 experts: 7.4 us where plan and copy apart take three launches.
template <int ES, bool VEC, int WPT>
__global__ __launch_bounds__(kBlock) void k_dispatch_few(ExchangeRowsArgs a, PlanArgs p) {
    __shared__ uint32_t shared[DT_MAX_EXPERTS];
    const uint32_t tokens = a.rows.start[a.nranks], slots = tokens * a.topk;
    if (blockIdx.x + 1 == gridDim.x) {
        for (uint32_t e = threadIdx.x; e < p.nexperts; e += kBlock) shared[e] = 0;
        __syncthreads();
        for (uint32_t s = threadIdx.x; s < slots; s += kBlock) {
            const int32_t e = slot_expert(p, s, slots);
            if (e >= 0) atomicAdd(&shared[e], 1u);
        }
        __syncthreads();
        store_offsets(p, shared);
        return;
    }
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t row = token_of<WPT>();
    const bool there = row < tokens;
    const uint32_t own = there ? row * a.topk : 0;  // the token's first slot
    const int32_t mine = there && lane < a.topk ? slot_expert(p, own + lane, slots) : -1;
    uint32_t pos = 0;  // lane j: the row of choice j
    // a wave takes all slots (WPT 1), or the workgroup's waves share them
    for (uint32_t s0 = WPT == 1 ? 0 : wave * 64; there && s0 < slots; s0 += 64 * WPT) {
        const uint32_t s = s0 + lane;
        const int32_t e = slot_expert(p, s, slots);
        for (uint32_t j = 0; j < a.topk; j++) {
            const int32_t ej = __builtin_amdgcn_readlane(mine, int(j));
            if (ej < 0) continue;
            const int32_t lowest = ej - int32_t(uint32_t(ej) % a.per_rank);
            const uint64_t m = __ballot((e >= lowest && e < ej) || (e == ej && s < own + j));
            if (lane == j) pos += uint32_t(__popcll(m));
        }
    }
    if constexpr (WPT > 1) {
        shared[threadIdx.x] = pos;
        __syncthreads();
        pos = 0;
#pragma unroll
        for (int w = 0; w < WPT; w++) pos += shared[w * 64 + lane];
    }
    if (!there) return;
    const int r = rank_of_row(a.rows, a.nranks, row);
    const uint64_t local = row - a.rows.start[r];
    const uint32_t pitch = a.cols * ES;
    Choices c = {0, 0};
    bool kept = false;
    if (lane < a.topk) {
        const uint32_t q = mine >= 0 ? uint32_t(mine) / a.per_rank : 0;
        kept = mine >= 0 && pos < a.capacity[q];
        if (kept) c.at = reinterpret_cast<uint64_t>(a.rows_out[q]) + uint64_t(pos) * pitch;
        if (WPT == 1 || wave == 0) p.positions[r][local * a.topk + lane] = kept ? int32_t(pos) : -1;
    }
    c.kept = __ballot(kept);
    dispatch_row<ES, VEC, WPT>(static_cast<const char*>(a.tokens_in[r]) + local * pitch, pitch, c,
                               threadIdx.x % (64 * WPT));
}

// The elements of a unit as fp32.
template <int DT>
struct Values {
    static constexpr int ES = DT == kBF16 ? 2 : 4, n = 16 / ES;
    typedef typename Elem<DT>::type T;
    static __device__ __forceinline__ void get(u32x4 x, float (&f)[n]) {
        T t[n];
        __builtin_memcpy(t, &x, 16);
#pragma unroll
        for (int i = 0; i < n; i++) f[i] = Elem<DT>::get(t[i]);
    }
    static __device__ __forceinline__ u32x4 put(const float (&f)[n]) {
        T t[n];
#pragma unroll
        for (int i = 0; i < n; i++) t[i] = Elem<DT>::put(f[i]);
        u32x4 x;
        __builtin_memcpy(&x, t, 16);
        return x;
    }
};

// out[t] = sum_j w_tj y[owner][pos_tj], in slot order, fp32, one rounding.  The
// rows of up to four choices are on their way at a time.  12519 rows of 1001
// fp32, 3 choices: 41 us, 4.9 TB/s on rows that start at any 4-byte boundary.
template <int DT, bool VEC, int WPT>
__global__ __launch_bounds__(kBlock) void k_combine(ExchangeRowsArgs a) {
    typedef Values<DT> V;
    constexpr int NV = 2, L = 64 * WPT, AHEAD = 4;
    const uint32_t row = token_of<WPT>();
    if (row >= a.rows.start[a.nranks]) return;
    const int r = rank_of_row(a.rows, a.nranks, row);
    const uint64_t local = row - a.rows.start[r];
    const uint32_t pitch = a.cols * V::ES, units = (pitch + 15) / 16, lane = threadIdx.x & 63;
    const Choices c = choices(a, a.rows_in, r, local, pitch);
    float w = 1.f;
    if (a.weights[r] != nullptr && lane < a.topk) w = a.weights[r][local * a.topk + lane];
    const char* out = static_cast<const char*>(a.tokens_out[r]) + local * pitch;
    for (uint32_t u0 = threadIdx.x % L; u0 < units; u0 += NV * L) {
        float s[NV][V::n];
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int e = 0; e < V::n; e++) s[i][e] = 0.f;
        for (uint64_t m = c.kept; m != 0;) {
            u32x4 x[AHEAD][NV];
            float wj[AHEAD];
            bool got[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; k++) {
                got[k] = m != 0;
                if (!got[k]) continue;
                const int j = __builtin_ctzll(m);
                m &= m - 1;
                wj[k] = __uint_as_float(uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(w)), j)));
                const char* y = choice_row(c, j);
#pragma unroll
                for (int i = 0; i < NV; i++)
                    if (u0 + i * L < units) x[k][i] = load_at<V::ES, VEC>(y, u0 + i * L, pitch);
            }
#pragma unroll
            for (int k = 0; k < AHEAD; k++) {
                if (!got[k]) continue;
#pragma unroll
                for (int i = 0; i < NV; i++) {
                    float f[V::n];
                    V::get(x[k][i], f);
#pragma unroll
                    for (int e = 0; e < V::n; e++) s[i][e] += wj[k] * f[e];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (u0 + i * L < units) store_at<V::ES, VEC>(out, u0 + i * L, pitch, V::put(s[i]));
    }
}

// dy[owner][pos] = w dout[t];  dw = <dout[t], y[owner][pos]>.  One pass over dout
// and y; the same rows as above: 79 us, 4.4 TB/s.
template <int DT, bool VEC, int WPT>
__global__ __launch_bounds__(kBlock) void k_combine_backward(ExchangeRowsArgs a) {
    typedef Values<DT> V;
    constexpr int NV = 2, L = 64 * WPT;
    __shared__ float dots[kBlock / 64][64];
    const uint32_t row = token_of<WPT>(), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (row >= a.rows.start[a.nranks]) return;
    const int r = rank_of_row(a.rows, a.nranks, row);
    const uint64_t local = row - a.rows.start[r];
    const uint32_t pitch = a.cols * V::ES, units = (pitch + 15) / 16;
    const Choices from = choices(a, a.rows_in, r, local, pitch), to = choices(a, a.rows_out, r, local, pitch);
    float w = 0.f;
    if (lane < a.topk) w = a.weights[r][local * a.topk + lane];
    const char* g = static_cast<const char*>(a.tokens_in[r]) + local * pitch;
    float dot = 0.f;  // lane j: this wave's part of choice j's
    for (uint32_t u0 = threadIdx.x % L; u0 - threadIdx.x % L < units; u0 += NV * L) {
        float gf[NV][V::n];
#pragma unroll
        for (int i = 0; i < NV; i++) {
#pragma unroll
            for (int e = 0; e < V::n; e++) gf[i][e] = 0.f;
            if (u0 + i * L < units) V::get(load_at<V::ES, VEC>(g, u0 + i * L, pitch), gf[i]);
        }
        for (uint64_t m = from.kept; m != 0; m &= m - 1) {
            const int j = __builtin_ctzll(m);
            const float wj = __uint_as_float(uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(w)), j)));
            const char* y = choice_row(from, j);
            const char* dy = choice_row(to, j);
            u32x4 x[NV];
#pragma unroll
            for (int i = 0; i < NV; i++)
                if (u0 + i * L < units) x[i] = load_at<V::ES, VEC>(y, u0 + i * L, pitch);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                if (u0 + i * L >= units) continue;
                float f[V::n], o[V::n];
                V::get(x[i], f);
#pragma unroll
                for (int e = 0; e < V::n; e++) {
                    s += gf[i][e] * f[e];
                    o[e] = wj * gf[i][e];
                }
                store_at<V::ES, VEC>(dy, u0 + i * L, pitch, V::put(o));
            }
            s = wave_sum(s);
            if (lane == uint32_t(j)) dot += s;
        }
    }
    if constexpr (WPT > 1) {
        dots[wave][lane] = dot;
        __syncthreads();
        if (wave > 0) return;
        dot = 0.f;
#pragma unroll
        for (int k = 0; k < WPT; k++) dot += dots[k][lane];
    }
    if (lane < a.topk) a.dweights[r][local * a.topk + lane] = dot;
}

// Lanes per token and experts per lane: 16 lanes for up to 512 experts and 16
// choices; with groups a group has to be whole lanes, a power of two of them.
int lane_experts(uint32_t nexperts, uint32_t topk, uint32_t groups) {
    if (topk > 16 || nexperts > 512) return 0;
    const int nl = nexperts <= 64 ? 4 : nexperts <= 128 ? 8 : nexperts <= 256 ? 16 : 32;
    if (groups > 1) {
        const uint32_t per = nexperts / groups, width = per / nl;
        if (per % nl != 0 || (width & (width - 1)) != 0 || nexperts != uint32_t(16 * nl) || width > 8) return 0;
    }
    return nl;
}
bool vector_rows(const void* const* list, int n, uint32_t elems, int dtype) {
    if (elems * (dtype == kBF16 ? 2 : 4) % 16 != 0) return false;
    for (int r = 0; r < n; r++)
        if (reinterpret_cast<uintptr_t>(list[r]) % 16 != 0) return false;
    return true;
}

template <int DT>
hipError_t route(const RouteArgs& a, int nranks, hipStream_t s) {
    const uint32_t rows = a.rows.start[nranks];
    const dim3 block(kBlock), few((rows + kBlock / 16 - 1) / (kBlock / 16)), any((rows + kBlock / 64 - 1) / (kBlock / 64));
    const int vec = vector_rows(a.logits, nranks, a.nexperts, DT);
    switch (lane_experts(a.nexperts, a.topk, a.groups)) {
        case 4: hipLaunchKernelGGL((k_route<DT, 4>), few, block, 0, s, a, nranks, vec); break;
        case 8: hipLaunchKernelGGL((k_route<DT, 8>), few, block, 0, s, a, nranks, vec); break;
        case 16: hipLaunchKernelGGL((k_route<DT, 16>), few, block, 0, s, a, nranks, vec); break;
        case 32: hipLaunchKernelGGL((k_route<DT, 32>), few, block, 0, s, a, nranks, vec); break;
        default:
            if (a.nexperts <= 128) hipLaunchKernelGGL((k_route_any<DT, 2>), any, block, 0, s, a, nranks);
            else if (a.nexperts <= 512) hipLaunchKernelGGL((k_route_any<DT, 8>), any, block, 0, s, a, nranks);
            else hipLaunchKernelGGL((k_route_any<DT, 16>), any, block, 0, s, a, nranks);
    }
    return hipGetLastError();
}
template <int DT>
hipError_t route_backward(const RouteBackArgs& a, int nranks, hipStream_t s) {
    const uint32_t rows = a.rows.start[nranks];
    const dim3 block(kBlock), few((rows + kBlock / 16 - 1) / (kBlock / 16)), any((rows + kBlock / 64 - 1) / (kBlock / 64));
    const int vec = vector_rows(a.logits, nranks, a.nexperts, DT) && vector_rows(a.dlogits, nranks, a.nexperts, DT);
    switch (lane_experts(a.nexperts, a.topk, 1)) {
        case 4: hipLaunchKernelGGL((k_route_backward<DT, 4, 16>), few, block, 0, s, a, nranks, vec); break;
        case 8: hipLaunchKernelGGL((k_route_backward<DT, 8, 16>), few, block, 0, s, a, nranks, vec); break;
        case 16: hipLaunchKernelGGL((k_route_backward<DT, 16, 16>), few, block, 0, s, a, nranks, vec); break;
        case 32: hipLaunchKernelGGL((k_route_backward<DT, 32, 16>), few, block, 0, s, a, nranks, vec); break;
        default: hipLaunchKernelGGL((k_route_backward<DT, 16, 64>), any, block, 0, s, a, nranks, vec);
    }
    return hipGetLastError();
}

// Short rows take a wave, long ones (over 4 KiB) the workgroup.
uint32_t token_blocks(uint32_t tokens, bool shorter) { return shorter ? (tokens + kBlock / 64 - 1) / (kBlock / 64) : tokens; }
template <typename F>
void with_rows(bool vec, bool shorter, F&& run) {
    if (vec && shorter) run(std::true_type(), std::integral_constant<int, 1>());
    else if (vec) run(std::true_type(), std::integral_constant<int, 4>());
    else if (shorter) run(std::false_type(), std::integral_constant<int, 1>());
    else run(std::false_type(), std::integral_constant<int, 4>());
}
}  // namespace

hipError_t launch_route(const RouteArgs& a, int nranks, int dtype, hipStream_t s) {
    return dtype == kBF16 ? route<kBF16>(a, nranks, s) : route<kF32>(a, nranks, s);
}
hipError_t launch_route_backward(const RouteBackArgs& a, int nranks, int dtype, hipStream_t s) {
    return dtype == kBF16 ? route_backward<kBF16>(a, nranks, s) : route_backward<kF32>(a, nranks, s);
}

hipError_t launch_dispatch(const PlanArgs& p, const ExchangeRowsArgs& a, int esize, hipStream_t s) {
    const uint32_t tokens = a.rows.start[a.nranks], slots = tokens * a.topk, blocks = plan_blocks(slots);
    const bool vec = vector_rows(a.tokens_in, a.nranks, a.cols, esize == 2 ? kBF16 : kF32) &&
                     vector_rows(a.rows_out, a.nranks, a.cols, esize == 2 ? kBF16 : kF32);
    const bool shorter = uint64_t(a.cols) * esize <= 4096;
    const uint32_t grid = token_blocks(tokens, shorter);
    if (slots <= kFewSlots) {
        with_rows(vec, shorter, [&](auto v, auto w) {
            if (esize == 2) hipLaunchKernelGGL((k_dispatch_few<2, decltype(v)::value, decltype(w)::value>), dim3(grid + 1), dim3(kBlock), 0, s, a, p);
            else hipLaunchKernelGGL((k_dispatch_few<4, decltype(v)::value, decltype(w)::value>), dim3(grid + 1), dim3(kBlock), 0, s, a, p);
        });
        return hipGetLastError();
    }
    // up to 128 workgroups of the plan each add up the counts before their own
    const int scanned = blocks > 128;
    hipLaunchKernelGGL(k_plan_count, dim3(blocks), dim3(kBlock), 0, s, p);
    if (scanned) hipLaunchKernelGGL(k_plan_scan, dim3((p.nexperts + 63) / 64), dim3(64), 0, s, p, blocks);
    hipLaunchKernelGGL(k_plan_place, dim3(blocks), dim3(kBlock), 0, s, p, blocks, scanned);
    with_rows(vec, shorter, [&](auto v, auto w) {
        if (esize == 2) hipLaunchKernelGGL((k_dispatch_rows<2, decltype(v)::value, decltype(w)::value>), dim3(grid), dim3(kBlock), 0, s, a);
        else hipLaunchKernelGGL((k_dispatch_rows<4, decltype(v)::value, decltype(w)::value>), dim3(grid), dim3(kBlock), 0, s, a);
    });
    return hipGetLastError();
}
hipError_t launch_combine(const ExchangeRowsArgs& a, int dtype, hipStream_t s) {
    const bool vec = vector_rows(a.tokens_out, a.nranks, a.cols, dtype) && vector_rows(a.rows_in, a.nranks, a.cols, dtype);
    const bool shorter = uint64_t(a.cols) * (dtype == kBF16 ? 2 : 4) <= 4096;
    const dim3 grid(token_blocks(a.rows.start[a.nranks], shorter)), block(kBlock);
    with_rows(vec, shorter, [&](auto v, auto w) {
        if (dtype == kBF16) hipLaunchKernelGGL((k_combine<kBF16, decltype(v)::value, decltype(w)::value>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_combine<kF32, decltype(v)::value, decltype(w)::value>), grid, block, 0, s, a);
    });
    return hipGetLastError();
}
hipError_t launch_combine_backward(const ExchangeRowsArgs& a, int dtype, hipStream_t s) {
    const bool vec = vector_rows(a.tokens_in, a.nranks, a.cols, dtype) && vector_rows(a.rows_in, a.nranks, a.cols, dtype) &&
                     vector_rows(a.rows_out, a.nranks, a.cols, dtype);
    const bool shorter = uint64_t(a.cols) * (dtype == kBF16 ? 2 : 4) <= 4096;
    const dim3 grid(token_blocks(a.rows.start[a.nranks], shorter)), block(kBlock);
    with_rows(vec, shorter, [&](auto v, auto w) {
        if (dtype == kBF16) hipLaunchKernelGGL((k_combine_backward<kBF16, decltype(v)::value, decltype(w)::value>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_combine_backward<kF32, decltype(v)::value, decltype(w)::value>), grid, block, 0, s, a);
    });
    return hipGetLastError();
}

}  // namespace dt
