// layer.hip -- the experts' layer for few tokens, in two launches.
//
//   h_s = w_s act(W1_e x_t + b1_e)          slot s = (t, j), e its expert, w_s its weight
//   out_t = residual_t + sum over t's slots of (W2_e h_s + w_s b2_e)
//   gated: act(g) u with [g; u] the first product
//
// Few tokens meet many weights: the layer is bound by the bytes of the chosen
// experts' weights, which are read once.  The first kernel gives 16 features of one
// expert to a workgroup, whose waves share the summed index; the second gives 16
// columns of `out` to a workgroup, whose waves share the summed index of all
// experts in use.  Weights go from memory straight into the registers of the matrix
// instructions, 16 rows by 64 bytes at a time, with the tokens as the other operand.
//
// All sums are fp32, in a fixed order.  Between the products h is kept in fp32, for
// bf16 in two parts, its rounding and the rest's: the second matrix instruction is
// free beside the weight's bytes.  A slot's weight is multiplied into h, so that the
// second product runs on over the experts without a sum for each of them.
#include "dt_act.h"
#include "dt_matrix.h"

namespace dt {
namespace {

constexpr uint32_t kInWaves = 4, kOutWaves = 16;
constexpr int kUnroll = 4;       // steps of 64 bytes whose loads go out together
constexpr uint32_t kTokens = DT_MAX_LAYER_TOKENS;

// A lane's 16 bytes of a weight row, which no other workgroup reads: past the cache.
template <int DT, bool VEC>
__device__ __forceinline__ u32x4 weight_at(const char* row, uint32_t at) {
    if constexpr (VEC) return load16(row + at);
    else return __builtin_nontemporal_load(reinterpret_cast<const typename Loose<DT == kBF16 ? 2 : 4>::type*>(row + at));
}
template <int DT, bool VEC>
__device__ __forceinline__ u32x4 token_at(const char* row, uint32_t at) {
    if constexpr (VEC) return *reinterpret_cast<const u32x4*>(row + at);
    else return *reinterpret_cast<const typename Loose<DT == kBF16 ? 2 : 4>::type*>(row + at);
}
// The same where the row may end inside the 16 bytes or before them.
template <int DT, bool VEC>
__device__ __forceinline__ u32x4 end_at(const char* row, uint32_t at, uint32_t bytes) {
    if constexpr (VEC) return at < bytes ? *reinterpret_cast<const u32x4*>(row + at) : u32x4{0, 0, 0, 0};
    else return read_loose<DT == kBF16 ? 2 : 4>(row, at, bytes);
}

// The tokens of the i-th expert in use, in ascending order.
struct Plan {
    uint32_t map[DT_MAX_EXPERTS / 32];   // experts in use
    uint32_t expert, used, count;
    uint32_t starts[kInWaves];
    uint16_t token[kTokens], slot[kTokens];
    float weight[kTokens];
};
__device__ __forceinline__ int32_t expert_of(const LayerArgs& a, int r, uint32_t local, uint32_t j) {
    const int32_t e = a.experts[r][uint64_t(local) * a.topk + j];
    return e >= 0 && uint32_t(e) < a.nexperts ? e : -1;
}
// False: fewer than i + 1 experts are in use.  A thread per token.
__device__ __forceinline__ bool make_plan(const LayerArgs& a, uint32_t i, Plan& p) {
    const uint32_t t = threadIdx.x, lane = t & 63;
    for (uint32_t w = t; w < DT_MAX_EXPERTS / 32; w += kInWaves * 64) p.map[w] = 0;
    __syncthreads();
    int r = 0;
    uint32_t local = 0;
    if (t < a.tokens) {
        while (r + 1 < a.nranks && t >= a.rows.start[r + 1]) r++;
        local = t - a.rows.start[r];
        for (uint32_t j = 0; j < a.topk; j++) {
            const int32_t e = expert_of(a, r, local, j);
            if (e >= 0) atomicOr(&p.map[e / 32], 1u << (e % 32));
        }
    }
    __syncthreads();
    // every wave finds the i-th bit set for itself
    const uint32_t bits = lane < DT_MAX_EXPERTS / 32 ? p.map[lane] : 0, n = __builtin_popcount(bits);
    uint32_t upto = n;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint32_t o = uint32_t(__shfl_up(int(upto), m));
        if (int(lane) >= m) upto += o;
    }
    const uint32_t used = uint32_t(__builtin_amdgcn_readlane(int(upto), 63));
    if (t == 0) p.used = used;
    if (i >= used) return false;   // the same in every wave
    if (upto > i && upto - n <= i) {
        uint32_t left = bits;
        for (uint32_t k = upto - n; k < i; k++) left &= left - 1;
        p.expert = lane * 32 + uint32_t(__builtin_ctz(left));
    }
    __syncthreads();
    const int32_t e = int32_t(p.expert);
    uint32_t slot = UINT32_MAX;
    float w = 0.f;
    if (t < a.tokens)
        for (uint32_t j = 0; j < a.topk; j++)
            if (expert_of(a, r, local, j) == e) {
                if (slot == UINT32_MAX) slot = j;
                w += a.weights[r][uint64_t(local) * a.topk + j];   // the same expert twice counts twice
            }
    const uint64_t has = __ballot(slot != UINT32_MAX);
    if (lane == 0) p.starts[t >> 6] = uint32_t(__builtin_popcountll(has));
    __syncthreads();
    uint32_t at = uint32_t(__builtin_popcountll(has & ((1ull << lane) - 1))), all = 0;
    for (uint32_t k = 0; k < kInWaves; k++) {
        if (k < (t >> 6)) at += p.starts[k];
        all += p.starts[k];
    }
    if (slot != UINT32_MAX) {
        p.token[at] = uint16_t(t);
        p.slot[at] = uint16_t(slot);
        p.weight[at] = w;
    }
    if (t == 0) p.count = all;
    if (blockIdx.x == 0 && t < a.tpad) {   // what the second kernel needs to know
        a.table[kLayerHeader + a.used + i * a.tpad + t] = slot != UINT32_MAX ? int32_t(t * a.topk + slot) : -1;
        if (t == 0) a.table[kLayerHeader + i] = e;
    }
    __syncthreads();
    return true;
}

// ---------------------------------------------------------- first product --
// Tokens [base, base + 16 G) of the plan.
template <int DT, bool VEC, bool GATED, int G>
__device__ __forceinline__ void in_tile(const LayerArgs& a, const Plan& p, uint32_t base, f32x4 (*sums)[64]) {
    typedef typename Elem<DT>::type T;
    constexpr int W = GATED ? 2 : 1;
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t e = __builtin_amdgcn_readfirstlane(p.expert), q = e / a.per_rank, local = e % a.per_rank;
    const uint32_t pitch = a.cols * uint32_t(sizeof(T)), m0 = blockIdx.x * 16;
    // lane: row (or token) lane % 16, 16 bytes lane / 16 of a step; rows behind the last one repeat it
    const uint32_t m = m0 + (lane & 15) < a.inner ? m0 + (lane & 15) : a.inner - 1;
    const char* w[W];
#pragma unroll
    for (int k = 0; k < W; k++)
        w[k] = static_cast<const char*>(a.w_in[q]) + (uint64_t(local) * W * a.inner + uint64_t(k) * a.inner + m) * pitch + (lane >> 4) * 16;
    const char* x[G];
#pragma unroll
    for (int g = 0; g < G; g++) {
        const uint32_t c = base + g * 16 + (lane & 15), t = p.token[c < p.count ? c : p.count - 1];
        int r = 0;
        while (r + 1 < a.nranks && t >= a.rows.start[r + 1]) r++;
        x[g] = static_cast<const char*>(a.x[r]) + uint64_t(t - a.rows.start[r]) * pitch + (lane >> 4) * 16;
    }
    f32x4 acc[W][G];
#pragma unroll
    for (int k = 0; k < W; k++)
#pragma unroll
        for (int g = 0; g < G; g++) acc[k][g] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint32_t whole = pitch / kStepBytes, each = (whole + kInWaves - 1) / kInWaves;
    const uint32_t lo = wave * each, hi = lo + each < whole ? lo + each : whole;
    auto steps = [&](uint32_t s, auto count) {
        constexpr int N = decltype(count)::value;
        u32x4 fa[N][W], fb[N][G];
#pragma unroll
        for (int i = 0; i < N; i++) {
#pragma unroll
            for (int k = 0; k < W; k++) fa[i][k] = weight_at<DT, VEC>(w[k], (s + i) * kStepBytes);
#pragma unroll
            for (int g = 0; g < G; g++) fb[i][g] = token_at<DT, VEC>(x[g], (s + i) * kStepBytes);
        }
#pragma unroll
        for (int i = 0; i < N; i++)
#pragma unroll
            for (int k = 0; k < W; k++)
#pragma unroll
                for (int g = 0; g < G; g++) acc[k][g] = multiply<DT>(fa[i][k], fb[i][g], acc[k][g]);
    };
    uint32_t s = lo;
    for (; s + kUnroll <= hi; s += kUnroll) steps(s, std::integral_constant<int, kUnroll>());
    for (; s < hi; s++) steps(s, std::integral_constant<int, 1>());
    if (wave == kInWaves - 1 && pitch % kStepBytes != 0) {   // the row's end
        const uint32_t at = whole * kStepBytes, from = (lane >> 4) * 16;
        u32x4 fb[G];
#pragma unroll
        for (int g = 0; g < G; g++) fb[g] = end_at<DT, VEC>(x[g] - from, at + from, pitch);
#pragma unroll
        for (int k = 0; k < W; k++) {
            const u32x4 fa = end_at<DT, VEC>(w[k] - from, at + from, pitch);
#pragma unroll
            for (int g = 0; g < G; g++) acc[k][g] = multiply<DT>(fa, fb[g], acc[k][g]);
        }
    }
#pragma unroll
    for (int k = 0; k < W; k++)
#pragma unroll
        for (int g = 0; g < G; g++) sums[(wave * G + g) * W + k][lane] = acc[k][g];
    __syncthreads();
    // thread: token group threadIdx.x / 64, the lane's four features of its token
    const uint32_t g = threadIdx.x >> 6, c = base + g * 16 + (lane & 15), f = m0 + (lane >> 4) * 4;
    if (g < uint32_t(G) && c < p.count && f < a.inner) {
        f32x4 z = {0.f, 0.f, 0.f, 0.f}, u = z;
#pragma unroll
        for (uint32_t k = 0; k < kInWaves; k++) {
            z += sums[(k * G + g) * W][lane];
            if (GATED) u += sums[(k * G + g) * W + W - 1][lane];
        }
        T* to = reinterpret_cast<T*>(a.hidden + (uint64_t(p.token[c]) * a.topk + p.slot[c]) * a.hpitch) + f;
        const T* b = a.b_in[q] != nullptr ? static_cast<const T*>(a.b_in[q]) + uint64_t(local) * W * a.inner + f : nullptr;
        f32x4 h, rest;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const bool in = f + i < a.inner;
            if (b != nullptr && in) {
                z[i] += Elem<DT>::get(b[i]);
                if (GATED) u[i] += Elem<DT>::get(b[a.inner + i]);
            }
            const float v = act(z[i], a.act) * (GATED ? u[i] : 1.f) * p.weight[c];
            h[i] = in ? v : 0.f;   // zeros up to the row's pitch
            const float near = Elem<DT>::get(Elem<DT>::put(h[i]));
            rest[i] = fabsf(near) < INFINITY ? h[i] - near : 0.f;
        }
        store_quad<DT>(to, h, true);   // a row's pitch is whole fours
        if (DT == kBF16) store_quad<DT>(reinterpret_cast<T*>(reinterpret_cast<char*>(to) + a.hpart), rest, true);
        if (f + 4 >= a.inner)  // and what is left of its last 16 bytes
            for (uint32_t i = f + 4; i < a.hpitch / sizeof(T); i++) {
                to[i - f] = T(0);
                if (DT == kBF16) reinterpret_cast<T*>(reinterpret_cast<char*>(to) + a.hpart)[i - f] = T(0);
            }
    }
    __syncthreads();  // the next tokens' sums
}

template <int DT, bool VEC, bool GATED>
__global__ __launch_bounds__(kInWaves * 64) void k_layer_in(LayerArgs a) {
    __shared__ Plan p;
    __shared__ f32x4 sums[kInWaves * 4 * (GATED ? 2 : 1)][64];
    const bool there = make_plan(a, blockIdx.y, p);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.table[0] = int32_t(p.used);
    if (!there) return;
    const uint32_t count = __builtin_amdgcn_readfirstlane(p.count);
    uint32_t base = 0;
    for (; count - base > 32 && base < count; base += 64) in_tile<DT, VEC, GATED, 4>(a, p, base, sums);
    if (base < count) {
        if (count - base > 16) in_tile<DT, VEC, GATED, 2>(a, p, base, sums);
        else in_tile<DT, VEC, GATED, 1>(a, p, base, sums);
    }
}

// --------------------------------------------------------- second product --
// NG: groups of 16 tokens.
template <int DT, bool VEC, int NG>
__global__ __launch_bounds__(kOutWaves * 64) void k_layer_out(LayerArgs a) {
    typedef typename Elem<DT>::type T;
    constexpr int PARTS = DT == kBF16 ? 2 : 1;
    __shared__ f32x4 sums[kOutWaves][64];
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), m0 = blockIdx.x * 16;
    const uint32_t pitch = a.inner * uint32_t(sizeof(T)), whole = pitch / kStepBytes;
    const uint32_t steps = (pitch + kStepBytes - 1) / kStepBytes, each = (steps + kUnroll - 1) / kUnroll;
    const uint32_t used = __builtin_amdgcn_readfirstlane(a.table[0]);
    const uint32_t m = m0 + (lane & 15) < a.cols ? m0 + (lane & 15) : a.cols - 1, from = (lane >> 4) * 16;
    f32x4 acc[NG];
#pragma unroll
    for (int g = 0; g < NG; g++) acc[g] = f32x4{0.f, 0.f, 0.f, 0.f};
    // a unit: kUnroll steps of one expert
    for (uint32_t unit = wave; unit < used * each; unit += kOutWaves) {
        const uint32_t i = unit / each, s = unit % each * kUnroll;
        const uint32_t e = __builtin_amdgcn_readfirstlane(a.table[kLayerHeader + i]), q = e / a.per_rank, local = e % a.per_rank;
        const char* w = static_cast<const char*>(a.w_out[q]) + (uint64_t(local) * a.cols + m) * pitch;
        const int32_t* slots = a.table + kLayerHeader + a.used + i * a.tpad + (lane & 15);
        int32_t slot[NG];
#pragma unroll
        for (int g = 0; g < NG; g++) slot[g] = uint32_t(g) * 16 < a.tpad ? slots[g * 16] : -1;
        u32x4 fa[kUnroll];
        const bool full = s + kUnroll <= whole;
#pragma unroll
        for (int k = 0; k < kUnroll; k++) {
            const uint32_t at = (s + k) * kStepBytes + from;
            fa[k] = full ? weight_at<DT, VEC>(w, at) : end_at<DT, VEC>(w, at, pitch);
        }
#pragma unroll
        for (int g = 0; g < NG; g++) {
            if (!__any(slot[g] >= 0)) continue;
            const char* h = a.hidden + uint64_t(slot[g] < 0 ? 0 : slot[g]) * a.hpitch;
            u32x4 fb[PARTS][kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; k++)
#pragma unroll
                for (int part = 0; part < PARTS; part++) {
                    const uint32_t at = (s + k) * kStepBytes + from;
                    fb[part][k] = u32x4{0, 0, 0, 0};
                    if (slot[g] >= 0 && at < a.hpitch)
                        fb[part][k] = *reinterpret_cast<const u32x4*>(h + part * a.hpart + at);
                }
            f32x4 sum = acc[g];
#pragma unroll
            for (int k = 0; k < kUnroll; k++)
#pragma unroll
                for (int part = 0; part < PARTS; part++) sum = multiply<DT>(fa[k], fb[part][k], sum);
            // zeros times an infinite weight are NaN: a token keeps its sum where the expert is not its own
            if (slot[g] >= 0) acc[g] = sum;
        }
    }
#pragma unroll
    for (int g = 0; g < NG; g++) {
        __syncthreads();
        sums[wave][lane] = acc[g];
        __syncthreads();
        // thread: element threadIdx.x % 4 of lane threadIdx.x / 4's four
        if (threadIdx.x >= 256) continue;
        const uint32_t l = threadIdx.x >> 2, t = g * 16 + (l & 15), c = m0 + (l >> 4) * 4 + (threadIdx.x & 3);
        if (t >= a.tokens || c >= a.cols) continue;
        float v = 0.f;
#pragma unroll
        for (uint32_t k = 0; k < kOutWaves; k++) v += sums[k][l][threadIdx.x & 3];
        int r = 0;
        while (r + 1 < a.nranks && t >= a.rows.start[r + 1]) r++;
        const uint32_t row = t - a.rows.start[r];
        if (a.b_out[0] != nullptr)
            for (uint32_t j = 0; j < a.topk; j++) {
                const int32_t e = expert_of(a, r, row, j);
                if (e >= 0)
                    v += a.weights[r][uint64_t(row) * a.topk + j] *
                         Elem<DT>::get(static_cast<const T*>(a.b_out[uint32_t(e) / a.per_rank])[uint64_t(uint32_t(e) % a.per_rank) * a.cols + c]);
            }
        const uint64_t at = uint64_t(row) * a.cols + c;
        if (a.residual[r] != nullptr) v += Elem<DT>::get(static_cast<const T*>(a.residual[r])[at]);
        static_cast<T*>(a.out[r])[at] = Elem<DT>::put(v);
    }
}

// -------------------------------------------------------------------- host --
uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

struct LayerParts {
    uint64_t hpitch, hpart, table, bytes;
    uint32_t used, tpad;
};
LayerParts layer_parts(uint64_t tokens, uint64_t inner, uint32_t nexperts, uint32_t topk, int dtype) {
    LayerParts b;
    const uint64_t slots = tokens * topk;
    b.hpitch = up(inner * (dtype == kBF16 ? 2 : 4), 16);
    b.hpart = slots * b.hpitch;
    b.used = uint32_t(slots < nexperts ? slots : nexperts);
    b.tpad = uint32_t(up(tokens, 16));
    b.table = up(b.hpart * (dtype == kBF16 ? 2 : 1), 256);
    b.bytes = b.table + up((kLayerHeader + b.used + uint64_t(b.used) * b.tpad) * 4, 256);
    return b;
}
bool on16(const void* const* list, int n) {
    for (int r = 0; r < n; r++)
        if (reinterpret_cast<uintptr_t>(list[r]) % 16 != 0) return false;
    return true;
}

template <int DT, bool VEC>
void first(const LayerArgs& a, hipStream_t s) {
    const dim3 grid((a.inner + 15) / 16, a.used);
    if (a.gated) hipLaunchKernelGGL((k_layer_in<DT, VEC, true>), grid, dim3(kInWaves * 64), 0, s, a);
    else hipLaunchKernelGGL((k_layer_in<DT, VEC, false>), grid, dim3(kInWaves * 64), 0, s, a);
}
template <int DT, bool VEC>
void second(const LayerArgs& a, hipStream_t s) {
    const dim3 grid((a.cols + 15) / 16), block(kOutWaves * 64);
    const uint32_t groups = a.tpad / 16;
    if (groups <= 1) hipLaunchKernelGGL((k_layer_out<DT, VEC, 1>), grid, block, 0, s, a);
    else if (groups <= 2) hipLaunchKernelGGL((k_layer_out<DT, VEC, 2>), grid, block, 0, s, a);
    else if (groups <= 4) hipLaunchKernelGGL((k_layer_out<DT, VEC, 4>), grid, block, 0, s, a);
    else if (groups <= 8) hipLaunchKernelGGL((k_layer_out<DT, VEC, 8>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_layer_out<DT, VEC, 16>), grid, block, 0, s, a);
}
template <int DT>
hipError_t layer(const LayerArgs& a, hipStream_t s) {
    const uint64_t es = sizeof(typename Elem<DT>::type);
    if (a.cols * es % 16 == 0 && on16(a.x, a.nranks) && on16(a.w_in, a.nranks)) first<DT, true>(a, s);
    else first<DT, false>(a, s);
    if (a.inner * es % 16 == 0 && on16(a.w_out, a.nranks)) second<DT, true>(a, s);
    else second<DT, false>(a, s);
    return hipGetLastError();
}

}  // namespace

uint64_t layer_workspace(uint64_t tokens, uint64_t, uint64_t inner, uint32_t nexperts, uint32_t topk, int dtype) {
    return tokens == 0 ? 0 : layer_parts(tokens, inner, nexperts, topk, dtype).bytes;
}

hipError_t launch_layer(LayerArgs a, void* workspace, int dtype, hipStream_t s) {
    const LayerParts b = layer_parts(a.tokens, a.inner, a.nexperts, a.topk, dtype);
    a.hidden = static_cast<char*>(workspace);
    a.hpitch = uint32_t(b.hpitch);
    a.hpart = b.hpart;
    a.table = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + b.table);
    a.used = b.used;
    a.tpad = b.tpad;
    return dtype == kBF16 ? layer<kBF16>(a, s) : layer<kF32>(a, s);
}

}  // namespace dt
