// loss.hip -- softmax cross entropy over a vocabulary sharded over the ranks,
// forward and backward, without keeping the logits.
//
//   z_tv = <hidden_t, weight_v>;   lse_t = log sum_v exp(z_tv)
//   loss_t = lse_t - z_t,target
//   d_tv = (exp(z_tv - lse_t) - [v = target_t]) dloss_t
//   dhidden_t = sum_v d_tv weight_v  (over all ranks' rows: an AllReduce)
//   dweight_v = sum_t d_tv hidden_t
//
// The forward pass forms the logits tile by tile in registers and keeps each
// tile's maximum and sum of exponentials per token; a second kernel joins
// them over the tiles of all ranks (the AllReduces of the maximum and the sum
// that a sharded vocabulary needs).  The backward pass forms the logits
// again, one piece of a rank's vocabulary at a time, and multiplies the
// piece's d into both gradients.
//
// All products have both operands contiguous along the summed index, so one
// matrix routine serves: out[n][m] = sum_k A[m][k] B[n][k].
#include "dt_step_device.h"

namespace dt {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kTile = 128;        // rows of A and of B per workgroup
constexpr int kChunks = 8;        // 16-byte chunks of the summed index per step
constexpr int kThreads = 256;

template <int DT>
struct Chunk {
    static constexpr int elems = 16 / int(sizeof(typename Elem<DT>::type));
};

// 16 bytes of row `row` at element k, zero past either end.
template <int DT, bool VEC>
__device__ __forceinline__ u32x4 load_chunk(const typename Elem<DT>::type* p, uint32_t row, uint32_t rows, uint64_t ld,
                                            uint32_t k, uint32_t K) {
    typedef typename Elem<DT>::type T;
    u32x4 v = {0, 0, 0, 0};
    if (row >= rows || k >= K) return v;
    const T* s = p + row * ld + k;
    if constexpr (VEC) {
        v = *reinterpret_cast<const u32x4*>(s);
    } else {
        T e[Chunk<DT>::elems];
#pragma unroll
        for (int i = 0; i < Chunk<DT>::elems; i++) e[i] = k + i < K ? s[i] : T(0);
        __builtin_memcpy(&v, e, 16);
    }
    return v;
}

// acc[i][j]: rows (of A) m = 64 (wave & 1) + 16 i + 4 (lane / 16) + r, columns
// (rows of B) n = 64 (wave >> 1) + 16 j + lane % 16.
template <int DT, bool VEC>
__device__ __forceinline__ void matrix_tile(const typename Elem<DT>::type* A, uint32_t rows_a, uint64_t lda,
                                            const typename Elem<DT>::type* B, uint32_t rows_b, uint64_t ldb, uint32_t K,
                                            f32x4 (&acc)[4][4]) {
    __shared__ u32x4 sa[kTile * kChunks], sb[kTile * kChunks];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    constexpr int CE = Chunk<DT>::elems;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (uint32_t k0 = 0; k0 < K; k0 += kChunks * CE) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTile * kChunks / kThreads; i++) {
            const uint32_t at = tid + i * kThreads, row = at / kChunks, c = at % kChunks;
            // the chunk's place is turned by the row, so that 16 rows' reads spread over the banks
            const uint32_t to = row * kChunks + (c ^ (row & 7));
            sa[to] = load_chunk<DT, VEC>(A, row, rows_a, lda, k0 + c * CE, K);
            sb[to] = load_chunk<DT, VEC>(B, row, rows_b, ldb, k0 + c * CE, K);
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kChunks / 4; kk++) {
            u32x4 fa[4], fb[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint32_t c = kk * 4 + (lane >> 4);
                const uint32_t ra = (wave & 1) * 64 + i * 16 + (lane & 15), rb = (wave >> 1) * 64 + i * 16 + (lane & 15);
                fa[i] = sa[ra * kChunks + (c ^ (ra & 7))];
                fb[i] = sb[rb * kChunks + (c ^ (rb & 7))];
            }
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    if constexpr (DT == kBF16) {
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fa[i]),
                                                                            __builtin_bit_cast(bf16x8, fb[j]), acc[i][j],
                                                                            0, 0, 0);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(fa[i][e]),
                                                                             __uint_as_float(fb[j][e]), acc[i][j], 0, 0, 0);
                    }
                }
        }
    }
}

// ---------------------------------------------------------------- forward --
struct StatsArgs {
    RowTable tiles;   // vocabulary tiles of the ranks
    float2* part;     // [tiles][tokens]: maximum, sum of exponentials
    float* target;    // [tokens]: the target's logit
};

template <int DT, bool VEC>
__global__ __launch_bounds__(kThreads) void k_loss_stats(LossArgs a, StatsArgs p) {
    typedef typename Elem<DT>::type T;
    __shared__ float2 half[2][kTile];
    const uint32_t tile = blockIdx.x, n0 = blockIdx.y * kTile;
    const int r = rank_of_row(p.tiles, a.nranks, tile);
    const uint32_t m0 = (tile - p.tiles.start[r]) * kTile;
    const uint32_t V = a.vocab.start[r + 1] - a.vocab.start[r];
    f32x4 acc[4][4];
    matrix_tile<DT, VEC>(static_cast<const T*>(a.weight[r]) + uint64_t(m0) * a.cols, V - m0, a.cols,
                         static_cast<const T*>(a.hidden[r]) + uint64_t(n0) * a.cols, a.tokens - n0, a.cols, a.cols, acc);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const uint32_t nl = (wave >> 1) * 64 + j * 16 + (lane & 15), n = n0 + nl;
        const int64_t t = n < a.tokens ? a.targets[r][n] : -1;
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const uint32_t m = m0 + (wave & 1) * 64 + i * 16 + (lane >> 4) * 4 + e;
                if (m >= V) acc[i][j][e] = -INFINITY;
                else if (t == int64_t(a.vocab.start[r]) + m) p.target[n] = acc[i][j][e];
                top = fmaxf(top, acc[i][j][e]);
            }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        float s = 0.f;
        const float base = top > -INFINITY ? top : 0.f;
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) s += expf(acc[i][j][e] - base);
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (lane < 16) half[wave & 1][nl] = make_float2(top, s);
    }
    __syncthreads();
    if (threadIdx.x < kTile && n0 + threadIdx.x < a.tokens) {
        const float2 u = half[0][threadIdx.x], v = half[1][threadIdx.x];
        const float top = fmaxf(u.x, v.x), base = top > -INFINITY ? top : 0.f;
        p.part[uint64_t(tile) * a.tokens + n0 + threadIdx.x] =
            make_float2(top, u.y * expf(u.x - base) + v.y * expf(v.x - base));
    }
}

__device__ __forceinline__ bool counted(const LossArgs& a, int64_t t) {
    return t != a.ignore_index && t >= 0 && t < int64_t(a.vocab.start[a.nranks]);
}

__global__ __launch_bounds__(kThreads) void k_loss_join(LossArgs a, StatsArgs p) {
    const uint32_t n = blockIdx.x * kThreads + threadIdx.x;
    if (n >= a.tokens) return;
    const uint32_t tiles = p.tiles.start[a.nranks];
    float top = -INFINITY, s = 0.f;
    for (uint32_t i = 0; i < tiles; i++) {
        const float2 v = p.part[uint64_t(i) * a.tokens + n];
        const float t = fmaxf(top, v.x), base = t > -INFINITY ? t : 0.f;
        s = s * expf(top - base) + v.y * expf(v.x - base);
        top = t;
    }
    const float lse = top + logf(s);
    for (int r = 0; r < a.nranks; r++) {
        a.lse[r][n] = lse;
        a.loss[r][n] = counted(a, a.targets[r][n]) ? lse - p.target[n] : 0.f;
    }
}

// --------------------------------------------------------------- backward --
// One piece: vocabulary rows [first, first + count) of rank `rank`.
struct PieceOfVocab {
    char* d;          // [tokens][ldv]
    char* dt;         // [count][ldt]
    char* wt;         // [cols][ldv]
    char* xt;         // [cols][ldt]
    float* acc;       // [tokens][ldx]
    uint64_t ldv, ldt, ldx;
    uint32_t first, count;
    int rank, add;    // add: acc holds the earlier pieces' sum
};

template <int DT, bool VEC>
__global__ __launch_bounds__(kThreads) void k_loss_d(LossArgs a, PieceOfVocab p) {
    typedef typename Elem<DT>::type T;
    const uint32_t m0 = blockIdx.x * kTile, n0 = blockIdx.y * kTile;
    const int r = p.rank;
    f32x4 acc[4][4];
    matrix_tile<DT, VEC>(static_cast<const T*>(a.weight[r]) + uint64_t(p.first + m0) * a.cols, p.count - m0, a.cols,
                         static_cast<const T*>(a.hidden[r]) + uint64_t(n0) * a.cols, a.tokens - n0, a.cols, a.cols, acc);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    T* d = reinterpret_cast<T*>(p.d);
    T* dt = reinterpret_cast<T*>(p.dt);
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const uint32_t n = n0 + (wave >> 1) * 64 + j * 16 + (lane & 15);
        const bool in = n < a.tokens;
        const int64_t t = in ? a.targets[r][n] : -1;
        const float lse = in ? a.lse[r][n] : 0.f;
        const bool use = in && counted(a, t);
        const float g = use ? a.dloss[r][n] : 0.f;
        const int64_t at = t - int64_t(a.vocab.start[r]) - int64_t(p.first);  // the target's row in the piece
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const uint32_t m = m0 + (wave & 1) * 64 + i * 16 + (lane >> 4) * 4 + e;
                float v = 0.f;
                if (use && m < p.count) v = (expf(acc[i][j][e] - lse) - (at == int64_t(m) ? 1.f : 0.f)) * g;
                const T o = Elem<DT>::put(v);
                if (in && m < p.ldv) d[uint64_t(n) * p.ldv + m] = o;
                if (m < p.count && n < p.ldt) dt[uint64_t(m) * p.ldt + n] = o;
            }
    }
}

// dst[c][r] = src[r][c], zeros for r in [rows, ld).
template <typename T>
__global__ __launch_bounds__(kThreads) void k_transpose(const T* src, T* dst, uint32_t rows, uint32_t cols, uint64_t ld) {
    __shared__ T tile[64][65];
    const uint32_t r0 = blockIdx.x * 64, c0 = blockIdx.y * 64;
    const uint32_t tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
    for (uint32_t i = ty; i < 64; i += 4) {
        const uint32_t r = r0 + i, c = c0 + tx;
        tile[i][tx] = r < rows && c < cols ? src[uint64_t(r) * cols + c] : T(0);
    }
    __syncthreads();
    for (uint32_t i = ty; i < 64; i += 4) {
        const uint32_t c = c0 + i, r = r0 + tx;
        if (c < cols && r < ld) dst[uint64_t(c) * ld + r] = tile[tx][i];
    }
}

// acc[t][h] (+)= sum over the piece of d[t][v] weight[v][h].
template <int DT>
__global__ __launch_bounds__(kThreads) void k_loss_dhidden(LossArgs a, PieceOfVocab p) {
    typedef typename Elem<DT>::type T;
    const uint32_t m0 = blockIdx.x * kTile, n0 = blockIdx.y * kTile;
    f32x4 acc[4][4];
    matrix_tile<DT, true>(reinterpret_cast<const T*>(p.wt) + uint64_t(m0) * p.ldv, a.cols - m0, p.ldv,
                          reinterpret_cast<const T*>(p.d) + uint64_t(n0) * p.ldv, a.tokens - n0, p.ldv, uint32_t(p.ldv),
                          acc);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t n = n0 + (wave >> 1) * 64 + j * 16 + (lane & 15);
            const uint32_t m = m0 + (wave & 1) * 64 + i * 16 + (lane >> 4) * 4;
            if (n >= a.tokens || m >= p.ldx) continue;
            f32x4* o = reinterpret_cast<f32x4*>(p.acc + uint64_t(n) * p.ldx + m);
            *o = p.add ? *o + acc[i][j] : acc[i][j];
        }
}

// dweight[v][h] = sum_t d[t][v] hidden[t][h].
template <int DT>
__global__ __launch_bounds__(kThreads) void k_loss_dweight(LossArgs a, PieceOfVocab p) {
    typedef typename Elem<DT>::type T;
    const uint32_t m0 = blockIdx.x * kTile, n0 = blockIdx.y * kTile;
    f32x4 acc[4][4];
    matrix_tile<DT, true>(reinterpret_cast<const T*>(p.xt) + uint64_t(m0) * p.ldt, a.cols - m0, p.ldt,
                          reinterpret_cast<const T*>(p.dt) + uint64_t(n0) * p.ldt, p.count - n0, p.ldt, uint32_t(p.ldt),
                          acc);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    T* out = static_cast<T*>(a.dweight[p.rank]) + uint64_t(p.first) * a.cols;
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const uint32_t n = n0 + (wave >> 1) * 64 + j * 16 + (lane & 15);
                const uint32_t m = m0 + (wave & 1) * 64 + i * 16 + (lane >> 4) * 4 + e;
                if (n < p.count && m < a.cols) out[uint64_t(n) * a.cols + m] = Elem<DT>::put(acc[i][j][e]);
            }
}

// Every rank's dhidden from the sum over all pieces, rounded once.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_loss_out(LossArgs a, const float* acc, uint64_t ldx) {
    typedef typename Elem<DT>::type T;
    const uint32_t n = blockIdx.x;
    for (uint32_t c = threadIdx.x; c < a.cols; c += kThreads) {
        const T v = Elem<DT>::put(acc[uint64_t(n) * ldx + c]);
        for (int r = 0; r < a.nranks; r++) static_cast<T*>(a.dhidden[r])[uint64_t(n) * a.cols + c] = v;
    }
}

uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }
uint32_t tiles_of(uint64_t n) { return uint32_t((n + kTile - 1) / kTile); }
uint64_t esize(int dtype) { return dtype == kBF16 ? 2 : 4; }
uint64_t pad_of(int dtype) { return kChunks * 16 / esize(dtype); }  // elements per step of the summed index

RowTable vocab_tiles(const RowTable& vocab, int nranks) {
    RowTable t = {};
    for (int r = 0; r < kMaxRanksHost; r++)
        t.start[r + 1] = t.start[r] + (r < nranks ? tiles_of(vocab.start[r + 1] - vocab.start[r]) : 0);
    return t;
}

// The workspace's parts, each on a 256-byte boundary.
struct BackwardParts {
    uint64_t ldv, ldt, ldx, d, dt, wt, xt, acc, bytes;
};
BackwardParts backward_parts(uint64_t tokens, uint64_t cols, uint64_t piece, int dtype) {
    BackwardParts b;
    const uint64_t es = esize(dtype);
    b.ldv = up(piece, pad_of(dtype));
    b.ldt = up(tokens, pad_of(dtype));
    b.ldx = up(cols, 4);
    uint64_t at = 0;
    auto take = [&](uint64_t n) {
        const uint64_t here = at;
        at += up(n, 256);
        return here;
    };
    b.d = take(tokens * b.ldv * es);
    b.dt = take(piece * b.ldt * es);
    b.wt = take(cols * b.ldv * es);
    b.xt = take(cols * b.ldt * es);
    b.acc = take(tokens * b.ldx * 4);
    b.bytes = at;
    return b;
}

bool rows_aligned(const LossArgs& a, int dtype) {
    if (a.cols * esize(dtype) % 16 != 0) return false;
    for (int r = 0; r < a.nranks; r++)
        if (reinterpret_cast<uintptr_t>(a.hidden[r]) % 16 || reinterpret_cast<uintptr_t>(a.weight[r]) % 16) return false;
    return true;
}

template <int DT>
hipError_t forward(const LossArgs& a, hipStream_t s) {
    StatsArgs p;
    p.tiles = vocab_tiles(a.vocab, a.nranks);
    p.part = reinterpret_cast<float2*>(a.workspace);
    const uint32_t tiles = p.tiles.start[a.nranks];
    p.target = reinterpret_cast<float*>(a.workspace + up(uint64_t(tiles) * a.tokens * sizeof(float2), 256));
    const dim3 grid(tiles, tiles_of(a.tokens));
    if (rows_aligned(a, DT)) hipLaunchKernelGGL((k_loss_stats<DT, true>), grid, dim3(kThreads), 0, s, a, p);
    else hipLaunchKernelGGL((k_loss_stats<DT, false>), grid, dim3(kThreads), 0, s, a, p);
    hipLaunchKernelGGL(k_loss_join, dim3((a.tokens + kThreads - 1) / kThreads), dim3(kThreads), 0, s, a, p);
    return hipGetLastError();
}

template <int DT>
hipError_t backward(const LossArgs& a, hipStream_t s) {
    typedef typename Elem<DT>::type T;
    const BackwardParts b = backward_parts(a.tokens, a.cols, a.piece, DT);
    const bool vec = rows_aligned(a, DT);
    const uint32_t ht = tiles_of(a.cols), tt = tiles_of(a.tokens);
    PieceOfVocab p = {};
    p.d = a.workspace + b.d;
    p.dt = a.workspace + b.dt;
    p.wt = a.workspace + b.wt;
    p.xt = a.workspace + b.xt;
    p.acc = reinterpret_cast<float*>(a.workspace + b.acc);
    p.ldt = b.ldt;
    p.ldx = b.ldx;
    const dim3 block(kThreads);
    for (int r = 0; r < a.nranks; r++) {
        const uint32_t V = a.vocab.start[r + 1] - a.vocab.start[r];
        if (V == 0) continue;
        p.rank = r;
        if (a.tokens > 0)
            hipLaunchKernelGGL(k_transpose<T>, dim3(uint32_t((b.ldt + 63) / 64), (a.cols + 63) / 64), block, 0, s,
                               static_cast<const T*>(a.hidden[r]), reinterpret_cast<T*>(p.xt), a.tokens, a.cols, b.ldt);
        for (uint32_t first = 0; first < V; first += a.piece) {
            p.first = first;
            p.count = V - first < a.piece ? V - first : a.piece;
            p.ldv = up(p.count, pad_of(DT));
            if (a.tokens > 0) {
                const dim3 gd(tiles_of(p.ldv), tiles_of(p.ldt));
                if (vec) hipLaunchKernelGGL((k_loss_d<DT, true>), gd, block, 0, s, a, p);
                else hipLaunchKernelGGL((k_loss_d<DT, false>), gd, block, 0, s, a, p);
                hipLaunchKernelGGL(k_transpose<T>, dim3(uint32_t((p.ldv + 63) / 64), (a.cols + 63) / 64), block, 0, s,
                                   static_cast<const T*>(a.weight[r]) + uint64_t(first) * a.cols,
                                   reinterpret_cast<T*>(p.wt), p.count, a.cols, p.ldv);
                hipLaunchKernelGGL(k_loss_dhidden<DT>, dim3(ht, tt), block, 0, s, a, p);
                p.add = 1;
            }
            hipLaunchKernelGGL(k_loss_dweight<DT>, dim3(ht, tiles_of(p.count)), block, 0, s, a, p);
        }
    }
    if (a.tokens > 0)
        hipLaunchKernelGGL(k_loss_out<DT>, dim3(a.tokens), block, 0, s, a, static_cast<const float*>(p.acc), p.ldx);
    return hipGetLastError();
}

}  // namespace

uint64_t loss_workspace(const RowTable& vocab, int nranks, uint64_t tokens, uint64_t, int) {
    const uint64_t tiles = vocab_tiles(vocab, nranks).start[nranks];
    return up(tiles * tokens * sizeof(float2), 256) + up(tokens * 4, 256);
}

// Vocabulary rows per piece: the largest shard, at most what was asked for
// (16384 by default).
uint32_t loss_piece(const RowTable& vocab, int nranks, uint64_t, uint64_t, int, uint64_t asked) {
    uint64_t most = 1;
    for (int r = 0; r < nranks; r++)
        if (vocab.start[r + 1] - vocab.start[r] > most) most = vocab.start[r + 1] - vocab.start[r];
    const uint64_t want = asked > 0 ? asked : 16384;
    return uint32_t(want < most ? want : most);
}

uint64_t loss_backward_workspace(const RowTable&, int, uint64_t tokens, uint64_t cols, uint32_t piece, int dtype) {
    return backward_parts(tokens, cols, piece, dtype).bytes;
}

hipError_t launch_loss(const LossArgs& a, int dtype, hipStream_t s) {
    return dtype == kBF16 ? forward<kBF16>(a, s) : forward<kF32>(a, s);
}
hipError_t launch_loss_backward(const LossArgs& a, int dtype, hipStream_t s) {
    return dtype == kBF16 ? backward<kBF16>(a, s) : backward<kF32>(a, s);
}

}  // namespace dt
