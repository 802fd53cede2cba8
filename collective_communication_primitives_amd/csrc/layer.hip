// layer.hip -- the experts' layer for few tokens, in two launches.
//
//   h_s = w_s act(W1_e x_t + b1_e)          slot s = (t, j), e its expert, w_s its weight
//   out_t = residual_t + sum over t's slots of (W2_e h_s + w_s b2_e)
//   gated: act(g) u with [g; u] the first product
//
// Few tokens meet many weights: the layer is bound by the bytes of the chosen
// experts' weights, which are read once.  The first kernel gives 16 features of one
// expert to a workgroup, whose waves share the summed index; the second gives 16
// columns of `out` to a workgroup, whose waves share the experts in use and their
// summed index.  An expert's tokens stand side by side as the columns of the matrix
// instructions, so that each weight meets no more of them than it has.
//
// 128 bf16 tokens of 4096 to 4 of 64 experts of 2 x 2048: 389 us for the first
// product's 2.1 GB (5.5 TB/s), 238 for the second's 1.1 GB (4.5 TB/s: fewer columns,
// each workgroup with all experts).  One token of 2048 to 2 of 64 of 2 x 1024: 11.5 +
// 7.5 us, latency, where the bytes take 4 in all: two launches of 128 workgroups, on
// half of the CUs, and the first one's make their plan, five barriers and two
// dependent reads of the choice, before they ask for the first weight.
//
// All sums are fp32, in a fixed order.  Between the products h is kept in fp32, for
// bf16 in two parts, its rounding and the rest's: the second matrix instruction, and
// the sums of its own that it has, are free beside the weight's bytes.  A slot's
// weight is multiplied into h, so that the second product runs on over the experts
// without a sum for each of them.
#include "dt_act.h"
#include "dt_stream.h"

namespace dt {
namespace {

constexpr int kPairs = 2;   // pairs of steps on their way in a wave
constexpr uint32_t kTokens = DT_MAX_LAYER_TOKENS;

// The tokens of the i-th expert in use, in ascending order.
struct Plan {
    uint32_t map[DT_MAX_EXPERTS / 32];   // experts in use
    uint32_t expert, used, count;
    uint32_t starts[kTokens / 64];
    uint16_t token[kTokens], slot[kTokens];
    float weight[kTokens];
};
__device__ __forceinline__ int32_t expert_of(const LayerArgs& a, int r, uint32_t local, uint32_t j) {
    const int32_t e = a.experts[r][uint64_t(local) * a.topk + j];
    return e >= 0 && uint32_t(e) < a.nexperts ? e : -1;
}
// False: fewer than i + 1 experts are in use.  A thread per token: 256 threads at least.
__device__ __forceinline__ bool make_plan(const LayerArgs& a, uint32_t i, Plan& p) {
    const uint32_t t = threadIdx.x, lane = t & 63;
    if (t < DT_MAX_EXPERTS / 32) p.map[t] = 0;
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
    if (lane == 0 && t < kTokens) p.starts[t >> 6] = uint32_t(__builtin_popcountll(has));
    __syncthreads();
    uint32_t at = uint32_t(__builtin_popcountll(has & ((1ull << lane) - 1))), all = 0;
    for (uint32_t k = 0; k < kTokens / 64; k++) {
        if (k < (t >> 6)) at += p.starts[k];
        all += p.starts[k];
    }
    const bool tell = blockIdx.x == 0;   // the second kernel
    if (slot != UINT32_MAX) {
        p.token[at] = uint16_t(t);
        p.slot[at] = uint16_t(slot);
        p.weight[at] = w;
        if (tell) a.table[kLayerHeader + 2 * a.used + i * a.tpad + at] = int32_t(t * a.topk + slot);
    }
    if (t == 0) {
        p.count = all;
        if (tell) {
            a.table[kLayerHeader + 2 * i] = e;
            a.table[kLayerHeader + 2 * i + 1] = int32_t(all);
        }
    }
    __syncthreads();
    return true;
}

// ---------------------------------------------------------- first product --
// Features [m0, m0 + 16) of tokens [base, base + 16 G) of the plan.
template <int DT, bool VEC, bool GATED, int NW, int G>
__device__ __forceinline__ void in_tile(const LayerArgs& a, const Plan& p, uint32_t m0, uint32_t base, f32x4 (*sums)[64]) {
    typedef typename Elem<DT>::type T;
    constexpr int W = GATED ? 2 : 1, P = G > 1 ? 1 : kPairs;
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t e = __builtin_amdgcn_readfirstlane(p.expert), q = e / a.per_rank, local = e % a.per_rank;
    const uint32_t pitch = a.cols * uint32_t(sizeof(T));
    // the rows that the lane loads; behind the last one it is repeated
    const uint32_t m = m0 + (lane >> 2) < a.inner ? m0 + (lane >> 2) : a.inner - 1;
    const char *w[W], *x[1][G];
#pragma unroll
    for (int k = 0; k < W; k++) w[k] = static_cast<const char*>(a.w_in[q]) + ((uint64_t(local) * W + k) * a.inner + m) * pitch;
#pragma unroll
    for (int g = 0; g < G; g++) {
        const uint32_t c = base + g * 16 + (lane >> 2), t = p.token[c < p.count ? c : p.count - 1];
        int r = 0;
        while (r + 1 < a.nranks && t >= a.rows.start[r + 1]) r++;
        x[0][g] = static_cast<const char*>(a.x[r]) + uint64_t(t - a.rows.start[r]) * pitch;
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
    // thread: token group threadIdx.x / 64, the lane's four features of its token
    const uint32_t g = threadIdx.x >> 6, c = base + g * 16 + (lane & 15), f = m0 + (lane >> 4) * 4;
    if (g < uint32_t(G) && c < p.count && f < a.inner) {
        f32x4 z = {0.f, 0.f, 0.f, 0.f}, u = z;
#pragma unroll
        for (uint32_t k = 0; k < NW; k++) {
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

// GM: most groups of 16 tokens that meet the weights at a time.  fp32 keeps two sets
// of sums, whose registers are held to three waves to a SIMD (144 tokens of 2048 to 4
// of 6 experts of 2 x 1792: both products 236 us, 249 with two waves).
template <int DT, bool VEC, bool GATED, int NW, int GM>
__global__ __launch_bounds__(NW * 64, DT == kF32 && GM > 1 ? 3 : 1) void k_layer_in(LayerArgs a) {
    __shared__ Plan p;
    __shared__ f32x4 sums[NW * GM * (GATED ? 2 : 1)][64];
    const bool there = make_plan(a, blockIdx.y, p);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.table[0] = int32_t(p.used);
    if (!there) return;
    const uint32_t count = __builtin_amdgcn_readfirstlane(p.count);
    for (uint32_t m0 = blockIdx.x * 16; m0 < a.inner; m0 += gridDim.x * 16) {
        uint32_t base = 0;
        if constexpr (GM > 1)
            for (; base < count && count - base > 16; base += 16 * GM) in_tile<DT, VEC, GATED, NW, GM>(a, p, m0, base, sums);
        for (; base < count; base += 16) in_tile<DT, VEC, GATED, NW, 1>(a, p, m0, base, sums);
    }
}

// --------------------------------------------------------- second product --
// Value c of token t's row of `out`: biases and residual.
template <int DT>
__device__ __forceinline__ void finish(const LayerArgs& a, uint32_t t, uint32_t c, float v) {
    typedef typename Elem<DT>::type T;
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

// Columns [base, base + 16 G) of an expert's list: their share of `out`, 16 values
// for each token, is added to the wave's own sums in LDS.
template <int DT, bool VEC, int G>
__device__ __forceinline__ void out_part(const LayerArgs& a, const char* weight, const int32_t* list, uint32_t base, uint32_t count, uint32_t lo,
                                         uint32_t hi, uint32_t pitch, f32x4* mine) {
    constexpr int PARTS = DT == kBF16 ? 2 : 1, P = G > 1 ? 1 : kPairs;
    const uint32_t lane = threadIdx.x & 63;
    const char* const w[1] = {weight};
    const char* x[PARTS][G];
#pragma unroll
    for (int g = 0; g < G; g++) {
        const uint32_t c = base + g * 16 + (lane >> 2), slot = uint32_t(list[c < count ? c : count - 1]);
#pragma unroll
        for (int p = 0; p < PARTS; p++) x[p][g] = a.hidden + uint64_t(slot) * a.hpitch + p * a.hpart;
    }
    f32x4 acc[1][G];
#pragma unroll
    for (int g = 0; g < G; g++) acc[0][g] = f32x4{0.f, 0.f, 0.f, 0.f};
    stream_rows<DT, VEC, 1, G, PARTS, P>(w, x, lo, hi, pitch, a.hpitch, acc);
#pragma unroll
    for (int g = 0; g < G; g++) {
        const uint32_t c = base + g * 16 + (lane & 15);
        if (c < count) mine[uint32_t(list[c]) / a.topk * 4 + (lane >> 4)] += acc[0][g];
    }
}

template <int DT, bool VEC, int NW, int GM>
__global__ __launch_bounds__(NW * 64) void k_layer_out(LayerArgs a) {
    typedef typename Elem<DT>::type T;
    extern __shared__ f32x4 sums[];   // [NW][tokens][4]
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), m0 = blockIdx.x * 16;
    const uint32_t pitch = a.inner * uint32_t(sizeof(T)), steps = (pitch + kStepBytes - 1) / kStepBytes;
    for (uint32_t i = threadIdx.x; i < NW * a.tokens * 4; i += NW * 64) sums[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint32_t used = __builtin_amdgcn_readfirstlane(a.table[0]);
    __syncthreads();
    // A unit: one of an expert's `parts` shares of the summed index.  Fewer experts than waves are shared by them, as
    // far as a share has four pairs of steps.
    const uint32_t waves = NW * gridDim.y, most = steps / 8 > 0 ? steps / 8 : 1;
    uint32_t parts = used >= waves ? 1 : used > 0 ? (waves + used - 1) / used : 1;
    if (parts > most) parts = most;
    const uint32_t m = m0 + (lane >> 2) < a.cols ? m0 + (lane >> 2) : a.cols - 1;
    f32x4* mine = sums + wave * a.tokens * 4;
    for (uint32_t unit = blockIdx.y * NW + wave; unit < used * parts; unit += waves) {
        const uint32_t i = unit / parts;
        const uint32_t e = __builtin_amdgcn_readfirstlane(a.table[kLayerHeader + 2 * i]), count = __builtin_amdgcn_readfirstlane(a.table[kLayerHeader + 2 * i + 1]);
        const uint32_t q = e / a.per_rank, local = e % a.per_rank;
        const char* w = static_cast<const char*>(a.w_out[q]) + (uint64_t(local) * a.cols + m) * pitch;
        const int32_t* list = a.table + kLayerHeader + 2 * a.used + i * a.tpad;
        uint32_t lo, hi, base = 0;
        share_steps(steps, unit % parts, parts, lo, hi);
        if constexpr (GM > 1)
            for (; base < count && count - base > 16; base += 16 * GM) out_part<DT, VEC, GM>(a, w, list, base, count, lo, hi, pitch, mine);
        for (; base < count; base += 16) out_part<DT, VEC, 1>(a, w, list, base, count, lo, hi, pitch, mine);
    }
    __syncthreads();
    // a thread for each value: the waves' sums in order
    const float* all = reinterpret_cast<const float*>(sums);
    for (uint32_t i = threadIdx.x; i < a.tokens * 16; i += NW * 64) {
        const uint32_t t = i / 16, c = m0 + i % 16;
        if (c >= a.cols) continue;
        float v = 0.f;
#pragma unroll
        for (uint32_t k = 0; k < NW; k++) v += all[k * a.tokens * 16 + i];
        if (a.splits > 1) a.partial[(uint64_t(blockIdx.y) * a.tokens + t) * a.cols + c] = v;
        else finish<DT>(a, t, c, v);
    }
}

// The workgroups' shares of `out` added up in order, where the experts are split among several.
template <int DT>
__global__ __launch_bounds__(kBlock) void k_layer_join(LayerArgs a) {
    const uint32_t c = blockIdx.x * kBlock + threadIdx.x, t = blockIdx.y;
    if (c >= a.cols) return;
    float v = 0.f;
    for (uint32_t k = 0; k < a.splits; k++) v += a.partial[(uint64_t(k) * a.tokens + t) * a.cols + c];
    finish<DT>(a, t, c, v);
}

// -------------------------------------------------------------------- host --
uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

// Waves of the second product's workgroups; their sums take 64 bytes of LDS each for
// a token: 16 for up to 128 of them.  Many tokens to an expert take the registers of
// 8 (128 tokens to 4 of 64 experts of 2048 x 4096 bf16: 239 us with 16).
bool many_tokens(uint64_t slots, uint64_t used) { return slots > 24 * used; }
uint32_t out_waves(uint64_t tokens, uint64_t slots, uint64_t used) { return tokens > 128 || many_tokens(slots, used) ? 8 : 16; }

struct LayerParts {
    uint64_t hpitch, hpart, table, partial, bytes;
    uint32_t used, tpad, splits;
};
LayerParts layer_parts(uint64_t tokens, uint64_t cols, uint64_t inner, uint32_t nexperts, uint32_t topk, int dtype) {
    LayerParts b;
    const uint64_t slots = tokens * topk;
    b.hpitch = up(inner * (dtype == kBF16 ? 2 : 4), 16);
    b.hpart = slots * b.hpitch;
    b.used = uint32_t(slots < nexperts ? slots : nexperts);
    b.tpad = uint32_t(up(tokens, 16));
    // Few columns are too few workgroups for the experts' bytes: the experts are split among several then, each wave
    // with four pairs of steps at least, and a third launch adds up (108 tokens of 192 to 3 of 72 experts of 3840 bf16:
    // 299 us in 12 workgroups).
    const uint64_t tiles = (cols + 15) / 16, steps = (b.hpitch + kStepBytes - 1) / kStepBytes;
    uint64_t splits = 256 / tiles;
    const uint64_t most = b.used * steps / (out_waves(tokens, slots, b.used) * 8);
    if (splits > most) splits = most;
    b.splits = uint32_t(splits < 1 ? 1 : splits > 32 ? 32 : splits);
    b.table = up(b.hpart * (dtype == kBF16 ? 2 : 1), 256);
    b.partial = b.table + up((kLayerHeader + 2 * uint64_t(b.used) + uint64_t(b.used) * b.tpad) * 4, 256);
    b.bytes = b.partial + (b.splits > 1 ? up(b.splits * tokens * cols * 4, 256) : 0);
    return b;
}
bool on16(const void* const* list, int n) {
    for (int r = 0; r < n; r++)
        if (reinterpret_cast<uintptr_t>(list[r]) % 16 != 0) return false;
    return true;
}

// Few workgroups: 16 waves to each, so that a wave has a shorter way through the
// summed index.  Many tokens to an expert: 64 of them at a time.
template <int DT, bool VEC, bool GATED>
void first(const LayerArgs& a, hipStream_t s) {
    // Where the weights' rows are short a workgroup takes several tiles of them: each makes the plan for itself, which
    // takes as long as 64 KiB of weights (108 tokens of 192 to 3 of 72 experts of 2 x 3840 bf16: 128 us with one tile).
    const uint64_t tiles = (a.inner + 15) / 16, bytes = uint64_t(GATED ? 32 : 16) * a.cols * sizeof(typename Elem<DT>::type);
    uint64_t each = bytes < 65536 ? 65536 / bytes : 1;
    while (each > 1 && tiles / each * a.used < 1024) each /= 2;
    const dim3 grid(uint32_t((tiles + each - 1) / each), a.used);
    if (many_tokens(uint64_t(a.tokens) * a.topk, a.used)) hipLaunchKernelGGL((k_layer_in<DT, VEC, GATED, 4, 4>), grid, dim3(4 * 64), 0, s, a);
    else if (uint64_t(grid.x) * grid.y <= 1024) hipLaunchKernelGGL((k_layer_in<DT, VEC, GATED, 16, 1>), grid, dim3(16 * 64), 0, s, a);
    else hipLaunchKernelGGL((k_layer_in<DT, VEC, GATED, 4, 1>), grid, dim3(4 * 64), 0, s, a);
}
template <int DT, bool VEC>
void second(const LayerArgs& a, hipStream_t s) {
    const dim3 grid((a.cols + 15) / 16, a.splits);
    const uint64_t slots = uint64_t(a.tokens) * a.topk;
    if (many_tokens(slots, a.used)) hipLaunchKernelGGL((k_layer_out<DT, VEC, 8, 4>), grid, dim3(8 * 64), 8 * a.tokens * 64, s, a);
    else if (out_waves(a.tokens, slots, a.used) == 8) hipLaunchKernelGGL((k_layer_out<DT, VEC, 8, 1>), grid, dim3(8 * 64), 8 * a.tokens * 64, s, a);
    else hipLaunchKernelGGL((k_layer_out<DT, VEC, 16, 1>), grid, dim3(16 * 64), 16 * a.tokens * 64, s, a);
    if (a.splits > 1) hipLaunchKernelGGL(k_layer_join<DT>, dim3((a.cols + kBlock - 1) / kBlock, a.tokens), dim3(kBlock), 0, s, a);
}
template <int DT>
hipError_t layer(const LayerArgs& a, hipStream_t s) {
    const uint64_t es = sizeof(typename Elem<DT>::type);
    const bool vec = a.cols * es % 16 == 0 && on16(a.x, a.nranks) && on16(a.w_in, a.nranks);
    if (a.gated) vec ? first<DT, true, true>(a, s) : first<DT, false, true>(a, s);
    else vec ? first<DT, true, false>(a, s) : first<DT, false, false>(a, s);
    if (a.inner * es % 16 == 0 && on16(a.w_out, a.nranks)) second<DT, true>(a, s);
    else second<DT, false>(a, s);
    return hipGetLastError();
}

}  // namespace

uint64_t layer_workspace(uint64_t tokens, uint64_t cols, uint64_t inner, uint32_t nexperts, uint32_t topk, int dtype) {
    return tokens == 0 ? 0 : layer_parts(tokens, cols, inner, nexperts, topk, dtype).bytes;
}

hipError_t launch_layer(LayerArgs a, void* workspace, int dtype, hipStream_t s) {
    const LayerParts b = layer_parts(a.tokens, a.cols, a.inner, a.nexperts, a.topk, dtype);
    a.hidden = static_cast<char*>(workspace);
    a.hpitch = uint32_t(b.hpitch);
    a.hpart = b.hpart;
    a.table = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + b.table);
    a.used = b.used;
    a.tpad = b.tpad;
    a.splits = b.splits;
    a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + b.partial);
    return dtype == kBF16 ? layer<kBF16>(a, s) : layer<kF32>(a, s);
}

}  // namespace dt
