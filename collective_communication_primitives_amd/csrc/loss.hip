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

constexpr int kChunks = 8;        // 16-byte chunks of the summed index per step: 128 bytes of a row
constexpr int kThreads = 256;     // workgroups of the kernels without a matrix tile

// A workgroup's tile of `out`: BM rows of A by BN rows of B, cut among GM x GN
// waves.  Both operands are staged through LDS, two steps of 128 bytes of the
// summed index at a time (one is multiplied while the next one loads).
template <int BM_, int BN_, int GM_, int GN_>
struct Shape {
    static constexpr int BM = BM_, BN = BN_, GM = GM_, GN = GN_;
    static constexpr int waves = GM * GN, threads = waves * 64;
    static constexpr int WM = BM / GM, WN = BN / GN;  // a wave's part
    static constexpr int MI = WM / 16, NI = WN / 16;  // in matrix instructions of 16 x 16
    static constexpr int lds = 2 * (BM + BN) * kChunks;  // u32x4
    static constexpr int loads = (BM + BN) / 8 / waves;  // load instructions of 8 rows per wave and step
};

template <int DT>
struct Chunk {
    static constexpr int elems = 16 / int(sizeof(typename Elem<DT>::type));
};

// One operand: rows of `ld` elements, 16-byte aligned; the buffer resource
// ends behind the last row, so rows past it load zeros.
struct Operand {
    rsrc_t r;
    uint32_t pitch;   // bytes per row
};
__device__ __forceinline__ Operand operand(const void* p, uint32_t rows, int most, uint64_t pitch) {
    const uint32_t n = rows < uint32_t(most) ? rows : uint32_t(most);
    return Operand{make_rsrc(p, uint32_t(n * pitch)), uint32_t(pitch)};
}

// acc[i][j][e]: row m = WM (wave % GM) + 16 i + 4 (lane / 16) + e of A's tile,
// row n = WN (wave / GM) + 16 j + lane % 16 of B's.  `steps` is the number of
// 128-byte steps, `bytes` the valid bytes of a row (a multiple of 16).
template <int DT, typename S>
__device__ __forceinline__ void matrix_tile(const Operand& A, const Operand& B, uint32_t first, uint32_t bytes,
                                            u32x4* lds, f32x4 (&acc)[S::MI][S::NI]) {
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int i = 0; i < S::MI; i++)
#pragma unroll
        for (int j = 0; j < S::NI; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (first >= bytes) return;
    // A load instruction fills 8 rows of 128 bytes: lane l brings row l / 8.
    // The chunk that lands in place l % 8 is turned by the row, so that the 16
    // rows that a read of one chunk touches spread over all banks.
    const uint32_t row = lane >> 3, turn = ((lane & 7) ^ row) * 16;
    auto stage = [&](uint32_t at, int buf) {
        u32x4* to = lds + buf * (S::BM + S::BN) * kChunks;
        const bool in = at + turn < bytes;  // zeros behind the row's end
#pragma unroll
        for (int i = 0; i < S::loads; i++) {
            const uint32_t g = wave * S::loads + i;  // group of 8 rows: A's, then B's
            const bool a = g < S::BM / 8;
            const uint32_t r0 = (a ? g : g - S::BM / 8) * 8;
            const uint32_t off = (r0 + row) * (a ? A.pitch : B.pitch) + at + turn;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(a ? A.r : B.r, (__attribute__((address_space(3))) void*)(to + g * 64), 16,
                                                     int(in ? off : 0x80000000u), 0, 0, 0);
        }
    };
    stage(first, 0);
    const uint32_t wm = (wave % S::GM) * S::WM, wn = (wave / S::GM) * S::WN;
    int buf = 0;
    for (uint32_t at = first; at < bytes; at += kChunks * 16, buf ^= 1) {
        __syncthreads();  // this step's loads have landed, and the other half is no longer read
        if (at + kChunks * 16 < bytes) stage(at + kChunks * 16, buf ^ 1);
        const u32x4* sa = lds + buf * (S::BM + S::BN) * kChunks;
        const u32x4* sb = sa + S::BM * kChunks;
#pragma unroll
        for (int kk = 0; kk < kChunks / 4; kk++) {
            u32x4 fa[S::MI], fb[S::NI];
            const uint32_t c = kk * 4 + (lane >> 4);
#pragma unroll
            for (int i = 0; i < S::MI; i++) {
                const uint32_t r = wm + i * 16 + (lane & 15);
                fa[i] = sa[r * kChunks + (c ^ (r & 7))];
            }
#pragma unroll
            for (int j = 0; j < S::NI; j++) {
                const uint32_t r = wn + j * 16 + (lane & 15);
                fb[j] = sb[r * kChunks + (c ^ (r & 7))];
            }
#pragma unroll
            for (int i = 0; i < S::MI; i++)
#pragma unroll
                for (int j = 0; j < S::NI; j++) {
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

// Tile `id` of mt x nt in an order that keeps an XCD's workgroups on
// neighbouring tiles: ids go round the 8 XCDs, so each XCD gets a run of the
// tiles, walked in bands of 8 rows of tiles.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t mt, uint32_t nt, uint32_t& m, uint32_t& n) {
    const uint32_t total = mt * nt, q = total / 8, rem = total % 8, x = id % 8;
    const uint32_t t = x * q + (x < rem ? x : rem) + id / 8;
    const uint32_t band = t / (8 * nt), first = band * 8, in = t - band * 8 * nt;
    const uint32_t high = mt - first < 8 ? mt - first : 8;
    m = first + in % high;
    n = in / high;
}

__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f); }

// ---------------------------------------------------------------- forward --
// Vocabulary rows [first, first + count) of rank `rank`, and the operands as
// the matrix routine reads them: rows of `pitch` bytes (a multiple of 16) with
// `bytes` valid ones.
struct LossRows {
    const char* weight;
    const char* hidden;
    uint64_t pitch;
    uint32_t bytes;
    uint32_t first, count;
    int rank;
};
struct StatsArgs {
    uint32_t tiles, token_tiles;  // of this launch
    uint32_t first_tile, all;     // the launch's first tile among all, and how many all are
    float2* part;                 // [all][tokens]: maximum, sum of exponentials
    float* target;                // [tokens]: the target's logit
};

// (top, s) joined with another maximum and sum.
__device__ __forceinline__ void join(float& top, float& s, float2 v) {
    const float t = fmaxf(top, v.x), base = t > -INFINITY ? t : 0.f;
    s = s * exp_of(top - base) + v.y * exp_of(v.x - base);
    top = t;
}

template <int DT, typename S>
__global__ __launch_bounds__(S::threads) void k_loss_stats(LossArgs a, LossRows p, StatsArgs q) {
    __shared__ u32x4 lds[S::lds];
    __shared__ float2 part[S::GM][S::BN];
    uint32_t mt, nt;
    tile_of(blockIdx.x, q.tiles, q.token_tiles, mt, nt);
    const uint32_t m0 = mt * S::BM, n0 = nt * S::BN;
    const int r = p.rank;
    f32x4 acc[S::MI][S::NI];
    matrix_tile<DT, S>(operand(p.weight + uint64_t(m0) * p.pitch, p.count - m0, S::BM, p.pitch),
                       operand(p.hidden + uint64_t(n0) * p.pitch, a.tokens - n0, S::BN, p.pitch), 0, p.bytes, lds, acc);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t wm = wave % S::GM, wn = wave / S::GM;
    const uint32_t mlane = m0 + wm * S::WM + (lane >> 4) * 4;
#pragma unroll
    for (int j = 0; j < S::NI; j++) {
        const uint32_t nl = wn * S::WN + j * 16 + (lane & 15), n = n0 + nl;
        const int64_t t = n < a.tokens ? a.targets[r][n] - int64_t(a.vocab.start[r]) - int64_t(p.first) : -1;
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < S::MI; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const uint32_t m = mlane + i * 16 + e;
                if (m >= p.count) acc[i][j][e] = -INFINITY;
                else if (t == int64_t(m)) q.target[n] = acc[i][j][e];
                top = fmaxf(top, acc[i][j][e]);
            }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        float s = 0.f;
        const float base = top > -INFINITY ? top : 0.f;
#pragma unroll
        for (int i = 0; i < S::MI; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) s += exp_of(acc[i][j][e] - base);
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (lane < 16) part[wm][nl] = make_float2(top, s);
    }
    __syncthreads();
    for (uint32_t nl = threadIdx.x; nl < S::BN && n0 + nl < a.tokens; nl += S::threads) {
        float top = part[0][nl].x, s = part[0][nl].y;
#pragma unroll
        for (int w = 1; w < S::GM; w++) join(top, s, part[w][nl]);
        q.part[uint64_t(q.first_tile + mt) * a.tokens + n0 + nl] = make_float2(top, s);
    }
}

__device__ __forceinline__ bool counted(const LossArgs& a, int64_t t) {
    return t != a.ignore_index && t >= 0 && t < int64_t(a.vocab.start[a.nranks]);
}

__global__ __launch_bounds__(kThreads) void k_loss_join(LossArgs a, StatsArgs p) {
    const uint32_t n = blockIdx.x * kThreads + threadIdx.x;
    if (n >= a.tokens) return;
    float top = -INFINITY, s = 0.f;
    for (uint32_t i = 0; i < p.all; i++) join(top, s, p.part[uint64_t(i) * a.tokens + n]);
    const float lse = top + logf(s);
    for (int r = 0; r < a.nranks; r++) {
        a.lse[r][n] = lse;
        a.loss[r][n] = counted(a, a.targets[r][n]) ? lse - p.target[n] : 0.f;
    }
}

// --------------------------------------------------------------- backward --
// The piece's buffers in the workspace.
struct PieceOfVocab {
    char* d;          // [tokens][ldv]
    char* dt;         // [count][ldt]
    char* wt;         // [cols][ldv]
    char* xt;         // [cols][ldt]
    float* acc;       // [splits][tokens][ldx]
    uint64_t ldv, ldt, ldx;
    uint32_t mt, nt;  // tiles of the launch
    uint32_t splits;  // workgroups that share one tile's sum over the piece
    int add;          // acc holds the earlier pieces' sum
};

// d of the piece, in both layouts; the rows' padding is zero.
template <int DT, typename S>
__global__ __launch_bounds__(S::threads) void k_loss_d(LossArgs a, LossRows w, PieceOfVocab p) {
    typedef typename Elem<DT>::type T;
    __shared__ u32x4 lds[S::lds];
    uint32_t mt, nt;
    tile_of(blockIdx.x, p.mt, p.nt, mt, nt);
    const uint32_t m0 = mt * S::BM, n0 = nt * S::BN;
    const int r = w.rank;
    f32x4 acc[S::MI][S::NI];
    // the last tiles may lie in the padding alone
    const uint32_t rows_a = w.count > m0 ? w.count - m0 : 0, rows_b = a.tokens > n0 ? a.tokens - n0 : 0;
    matrix_tile<DT, S>(operand(w.weight + uint64_t(m0) * w.pitch, rows_a, S::BM, w.pitch),
                       operand(w.hidden + uint64_t(n0) * w.pitch, rows_b, S::BN, w.pitch), 0, w.bytes, lds, acc);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    T* d = reinterpret_cast<T*>(p.d);
    T* dt = reinterpret_cast<T*>(p.dt);
#pragma unroll
    for (int j = 0; j < S::NI; j++) {
        const uint32_t n = n0 + (wave / S::GM) * S::WN + j * 16 + (lane & 15);
        const bool in = n < a.tokens;
        const int64_t t = in ? a.targets[r][n] : -1;
        const float lse = in ? a.lse[r][n] : 0.f;
        const bool use = in && counted(a, t);
        const float g = use ? a.dloss[r][n] : 0.f;
        const int64_t at = t - int64_t(a.vocab.start[r]) - int64_t(w.first);  // the target's row in the piece
#pragma unroll
        for (int i = 0; i < S::MI; i++) {
            const uint32_t m = m0 + (wave % S::GM) * S::WM + i * 16 + (lane >> 4) * 4;
            T o[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                float v = 0.f;
                if (use && m + e < w.count) v = (exp_of(acc[i][j][e] - lse) - (at == int64_t(m + e) ? 1.f : 0.f)) * g;
                o[e] = Elem<DT>::put(v);
            }
            // ldv is a multiple of 4: the four are all inside a row or all behind it
            if (in && m < p.ldv) __builtin_memcpy(__builtin_assume_aligned(d + uint64_t(n) * p.ldv + m, 4 * sizeof(T)), o, sizeof o);
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (m + e < w.count && n < p.ldt) dt[uint64_t(m + e) * p.ldt + n] = o[e];
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

// acc[split][t][h] (+)= sum over the split's part of the piece of d[t][v] weight[v][h].
template <int DT, typename S>
__global__ __launch_bounds__(S::threads) void k_loss_dhidden(LossArgs a, PieceOfVocab p) {
    typedef typename Elem<DT>::type T;
    __shared__ u32x4 lds[S::lds];
    uint32_t mt, nt;
    tile_of(blockIdx.x, p.mt, p.nt, mt, nt);
    const uint32_t m0 = mt * S::BM, n0 = nt * S::BN;
    f32x4 acc[S::MI][S::NI];
    const uint64_t pitch = p.ldv * sizeof(T);
    const uint32_t steps = uint32_t(pitch / (kChunks * 16));
    const uint32_t lo = uint32_t(uint64_t(steps) * blockIdx.y / p.splits), hi = uint32_t(uint64_t(steps) * (blockIdx.y + 1) / p.splits);
    matrix_tile<DT, S>(operand(p.wt + uint64_t(m0) * pitch, a.cols - m0, S::BM, pitch),
                       operand(p.d + uint64_t(n0) * pitch, a.tokens - n0, S::BN, pitch), lo * kChunks * 16, hi * kChunks * 16,
                       lds, acc);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float* to = p.acc + uint64_t(blockIdx.y) * a.tokens * p.ldx;
#pragma unroll
    for (int j = 0; j < S::NI; j++)
#pragma unroll
        for (int i = 0; i < S::MI; i++) {
            const uint32_t n = n0 + (wave / S::GM) * S::WN + j * 16 + (lane & 15);
            const uint32_t m = m0 + (wave % S::GM) * S::WM + i * 16 + (lane >> 4) * 4;
            if (n >= a.tokens || m >= p.ldx) continue;
            f32x4* o = reinterpret_cast<f32x4*>(to + uint64_t(n) * p.ldx + m);
            *o = p.add ? *o + acc[i][j] : acc[i][j];
        }
}

// dweight[v][h] = sum_t d[t][v] hidden[t][h].
template <int DT, typename S>
__global__ __launch_bounds__(S::threads) void k_loss_dweight(LossArgs a, LossRows w, PieceOfVocab p) {
    typedef typename Elem<DT>::type T;
    __shared__ u32x4 lds[S::lds];
    uint32_t mt, nt;
    tile_of(blockIdx.x, p.mt, p.nt, mt, nt);
    const uint32_t m0 = mt * S::BM, n0 = nt * S::BN;
    f32x4 acc[S::MI][S::NI];
    const uint64_t pitch = p.ldt * sizeof(T);
    matrix_tile<DT, S>(operand(p.xt + uint64_t(m0) * pitch, a.cols - m0, S::BM, pitch),
                       operand(p.dt + uint64_t(n0) * pitch, w.count - n0, S::BN, pitch), 0, uint32_t(pitch), lds, acc);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    T* out = static_cast<T*>(a.dweight[w.rank]) + uint64_t(w.first) * a.cols;
    const bool quads = a.cols % 4 == 0 && reinterpret_cast<uintptr_t>(out) % (4 * sizeof(T)) == 0;
#pragma unroll
    for (int j = 0; j < S::NI; j++)
#pragma unroll
        for (int i = 0; i < S::MI; i++) {
            const uint32_t n = n0 + (wave / S::GM) * S::WN + j * 16 + (lane & 15);
            const uint32_t m = m0 + (wave % S::GM) * S::WM + i * 16 + (lane >> 4) * 4;
            if (n >= w.count || m >= a.cols) continue;
            T o[4];
#pragma unroll
            for (int e = 0; e < 4; e++) o[e] = Elem<DT>::put(acc[i][j][e]);
            T* to = out + uint64_t(n) * a.cols + m;
            if (quads) {
                __builtin_memcpy(__builtin_assume_aligned(to, 4 * sizeof(T)), o, sizeof o);
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (m + e < a.cols) to[e] = o[e];
            }
        }
}

// Every rank's dhidden from the sums of the splits, in order, rounded once.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_loss_out(LossArgs a, const float* acc, uint64_t ldx, uint32_t splits) {
    typedef typename Elem<DT>::type T;
    const uint32_t n = blockIdx.x;
    for (uint32_t c = threadIdx.x; c < a.cols; c += kThreads) {
        float s = 0.f;
        for (uint32_t k = 0; k < splits; k++) s += acc[(uint64_t(k) * a.tokens + n) * ldx + c];
        const T v = Elem<DT>::put(s);
        for (int r = 0; r < a.nranks; r++) static_cast<T*>(a.dhidden[r])[uint64_t(n) * a.cols + c] = v;
    }
}

// Rows of `cols` elements copied to rows of ld elements (a multiple of 16 bytes).
template <typename T>
__global__ __launch_bounds__(kThreads) void k_pad_rows(const T* src, T* dst, uint32_t cols, uint64_t ld) {
    const uint64_t row = blockIdx.x;
    for (uint32_t c = threadIdx.x; c < ld; c += kThreads) dst[row * ld + c] = c < cols ? src[row * cols + c] : T(0);
}

uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }
uint32_t ceil_div(uint64_t n, uint64_t by) { return uint32_t((n + by - 1) / by); }
uint64_t esize(int dtype) { return dtype == kBF16 ? 2 : 4; }
uint64_t pad_of(int dtype) { return kChunks * 16 / esize(dtype); }  // elements per step of the summed index

typedef Shape<256, 256, 2, 4> Wide;
typedef Shape<128, 128, 2, 2> Square;
typedef Shape<128, 64, 4, 1> Narrow;
constexpr uint32_t kStatsRows = 128;  // vocabulary rows that one entry of the partial statistics covers, at least

// The tile for an m x n product: the largest that still gives every one of
// the 256 CUs a workgroup.
enum Tile { kWide, kSquare, kNarrow };
Tile pick_tile(uint64_t m, uint64_t n, uint32_t splits = 1) {
    if (n <= 64) return kNarrow;
    if (uint64_t(ceil_div(m, 256)) * ceil_div(n, 256) * splits >= 224) return kWide;
    return kSquare;
}

// Rows that start and end on 16-byte boundaries are read where they are;
// others are copied to padded rows first, a piece at a time.
constexpr uint32_t kPiece = 16384;

// The workspace's parts, each on a 256-byte boundary.
struct Parts {
    uint64_t at = 0;
    uint64_t take(uint64_t n) {
        const uint64_t here = at;
        at += up(n, 256);
        return here;
    }
};
struct PadParts {
    uint64_t pitch, hidden, weight;
};
PadParts pad_parts(Parts& w, uint64_t tokens, uint64_t cols, uint64_t piece, int dtype) {
    PadParts b;
    b.pitch = up(cols * esize(dtype), 16);
    b.hidden = w.take(tokens * b.pitch);
    b.weight = w.take(piece * b.pitch);
    return b;
}
uint32_t splits_of(uint64_t tokens, uint64_t cols) {
    // few tiles of dhidden: the sum over the piece is cut among workgroups
    const uint64_t tiles = uint64_t(ceil_div(cols, 128)) * ceil_div(tokens, tokens <= 64 ? 64 : 128);
    if (tiles == 0 || tiles >= 256) return 1;
    const uint64_t want = ceil_div(512, tiles);
    return uint32_t(want < 16 ? want : 16);
}
struct BackwardParts {
    uint64_t ldv, ldt, ldx, d, dt, wt, xt, acc;
    uint32_t splits;
    PadParts pad;
    uint64_t bytes;
};
BackwardParts backward_parts(uint64_t tokens, uint64_t cols, uint64_t piece, int dtype) {
    BackwardParts b;
    const uint64_t es = esize(dtype);
    b.ldv = up(piece, pad_of(dtype));
    b.ldt = up(tokens, pad_of(dtype));
    b.ldx = up(cols, 4);
    b.splits = splits_of(tokens, cols);
    Parts w;
    b.d = w.take(tokens * b.ldv * es);
    b.dt = w.take(piece * b.ldt * es);
    b.wt = w.take(cols * b.ldv * es);
    b.xt = w.take(cols * b.ldt * es);
    b.acc = w.take(b.splits * tokens * b.ldx * 4);
    b.pad = pad_parts(w, tokens, cols, piece, dtype);
    b.bytes = w.at;
    return b;
}

bool rows_aligned(const void* p, uint64_t cols, int dtype) {
    return cols * esize(dtype) % 16 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// The operands of vocabulary rows [first, first + count) of rank r, copied to
// padded rows in the workspace where they are not aligned.  `fresh`: the
// rank's first piece.
template <int DT>
LossRows loss_rows(const LossArgs& a, const PadParts& pad, int r, uint32_t first, uint32_t count, bool fresh, hipStream_t s) {
    typedef typename Elem<DT>::type T;
    LossRows w = {};
    const T* weight = static_cast<const T*>(a.weight[r]) + uint64_t(first) * a.cols;
    w.rank = r;
    w.first = first;
    w.count = count;
    if (rows_aligned(a.weight[r], a.cols, DT) && rows_aligned(a.hidden[r], a.cols, DT)) {
        w.pitch = uint64_t(a.cols) * sizeof(T);
        w.weight = reinterpret_cast<const char*>(weight);
        w.hidden = static_cast<const char*>(a.hidden[r]);
    } else {
        w.pitch = pad.pitch;
        char* to = a.workspace + pad.weight;
        char* hidden = a.workspace + pad.hidden;
        const uint64_t ld = pad.pitch / sizeof(T);
        if (fresh)
            hipLaunchKernelGGL(k_pad_rows<T>, dim3(a.tokens), dim3(kThreads), 0, s, static_cast<const T*>(a.hidden[r]),
                               reinterpret_cast<T*>(hidden), a.cols, ld);
        hipLaunchKernelGGL(k_pad_rows<T>, dim3(count), dim3(kThreads), 0, s, weight, reinterpret_cast<T*>(to), a.cols, ld);
        w.weight = to;
        w.hidden = hidden;
    }
    w.bytes = uint32_t(w.pitch);
    return w;
}

template <int DT, typename S>
void stats(const LossArgs& a, const LossRows& w, StatsArgs q, hipStream_t s) {
    q.tiles = ceil_div(w.count, S::BM);
    q.token_tiles = ceil_div(a.tokens, S::BN);
    hipLaunchKernelGGL((k_loss_stats<DT, S>), dim3(q.tiles * q.token_tiles), dim3(S::threads), 0, s, a, w, q);
}

template <int DT>
hipError_t forward(const LossArgs& a, hipStream_t s) {
    Parts parts;
    uint64_t entries = 0;
    for (int r = 0; r < a.nranks; r++)
        for (uint32_t V = a.vocab.start[r + 1] - a.vocab.start[r], f = 0; f < V; f += kPiece)
            entries += ceil_div(V - f < kPiece ? V - f : kPiece, kStatsRows);
    StatsArgs q = {};
    q.part = reinterpret_cast<float2*>(a.workspace + parts.take(entries * a.tokens * sizeof(float2)));
    q.target = reinterpret_cast<float*>(a.workspace + parts.take(uint64_t(a.tokens) * 4));
    const PadParts pad = pad_parts(parts, a.tokens, a.cols, loss_piece(a.vocab, a.nranks, a.tokens, a.cols, DT, 0), DT);
    for (int r = 0; r < a.nranks; r++) {
        const uint32_t V = a.vocab.start[r + 1] - a.vocab.start[r];
        for (uint32_t f = 0; f < V; f += kPiece) {
            const LossRows w = loss_rows<DT>(a, pad, r, f, V - f < kPiece ? V - f : kPiece, f == 0, s);
            const Tile t = pick_tile(w.count, a.tokens);
            if (t == kWide) stats<DT, Wide>(a, w, q, s);
            else if (t == kSquare) stats<DT, Square>(a, w, q, s);
            else stats<DT, Narrow>(a, w, q, s);
            q.first_tile += ceil_div(w.count, t == kWide ? 256 : 128);
        }
    }
    q.all = q.first_tile;
    hipLaunchKernelGGL(k_loss_join, dim3((a.tokens + kThreads - 1) / kThreads), dim3(kThreads), 0, s, a, q);
    return hipGetLastError();
}

template <int DT, typename S>
void piece_d(const LossArgs& a, const LossRows& w, PieceOfVocab p, hipStream_t s) {
    p.mt = ceil_div(p.ldv, S::BM);
    p.nt = ceil_div(p.ldt, S::BN);
    hipLaunchKernelGGL((k_loss_d<DT, S>), dim3(p.mt * p.nt), dim3(S::threads), 0, s, a, w, p);
}
template <int DT, typename S>
void piece_dhidden(const LossArgs& a, PieceOfVocab p, hipStream_t s) {
    p.mt = ceil_div(a.cols, S::BM);
    p.nt = ceil_div(a.tokens, S::BN);
    hipLaunchKernelGGL((k_loss_dhidden<DT, S>), dim3(p.mt * p.nt, p.splits), dim3(S::threads), 0, s, a, p);
}
template <int DT, typename S>
void piece_dweight(const LossArgs& a, const LossRows& w, PieceOfVocab p, hipStream_t s) {
    p.mt = ceil_div(a.cols, S::BM);
    p.nt = ceil_div(w.count, S::BN);
    hipLaunchKernelGGL((k_loss_dweight<DT, S>), dim3(p.mt * p.nt), dim3(S::threads), 0, s, a, w, p);
}

template <int DT>
hipError_t backward(const LossArgs& a, hipStream_t s) {
    typedef typename Elem<DT>::type T;
    const BackwardParts b = backward_parts(a.tokens, a.cols, a.piece, DT);
    PieceOfVocab p = {};
    p.d = a.workspace + b.d;
    p.dt = a.workspace + b.dt;
    p.wt = a.workspace + b.wt;
    p.xt = a.workspace + b.xt;
    p.acc = reinterpret_cast<float*>(a.workspace + b.acc);
    p.ldt = b.ldt;
    p.ldx = b.ldx;
    p.splits = b.splits;
    const dim3 block(kThreads);
    for (int r = 0; r < a.nranks; r++) {
        const uint32_t V = a.vocab.start[r + 1] - a.vocab.start[r];
        if (V == 0) continue;
        if (a.tokens > 0)
            hipLaunchKernelGGL(k_transpose<T>, dim3(uint32_t((b.ldt + 63) / 64), (a.cols + 63) / 64), block, 0, s,
                               static_cast<const T*>(a.hidden[r]), reinterpret_cast<T*>(p.xt), a.tokens, a.cols, b.ldt);
        for (uint32_t first = 0; first < V; first += a.piece) {
            const uint32_t count = V - first < a.piece ? V - first : a.piece;
            LossRows w = {};
            w.rank = r;
            w.first = first;
            w.count = count;
            p.ldv = up(count, pad_of(DT));
            if (a.tokens > 0) {
                w = loss_rows<DT>(a, b.pad, r, first, count, first == 0, s);
                const Tile t = pick_tile(count, a.tokens);
                if (t == kWide) piece_d<DT, Wide>(a, w, p, s);
                else if (t == kSquare) piece_d<DT, Square>(a, w, p, s);
                else piece_d<DT, Narrow>(a, w, p, s);
                hipLaunchKernelGGL(k_transpose<T>, dim3(uint32_t((p.ldv + 63) / 64), (a.cols + 63) / 64), block, 0, s,
                                   static_cast<const T*>(a.weight[r]) + uint64_t(first) * a.cols,
                                   reinterpret_cast<T*>(p.wt), count, a.cols, p.ldv);
                const Tile h = pick_tile(a.cols, a.tokens, p.splits);
                if (h == kWide) piece_dhidden<DT, Wide>(a, p, s);
                else if (h == kSquare) piece_dhidden<DT, Square>(a, p, s);
                else piece_dhidden<DT, Narrow>(a, p, s);
                p.add = 1;
            }
            const Tile v = pick_tile(a.cols, count);
            if (v == kWide) piece_dweight<DT, Wide>(a, w, p, s);
            else if (v == kSquare) piece_dweight<DT, Square>(a, w, p, s);
            else piece_dweight<DT, Narrow>(a, w, p, s);
        }
    }
    if (a.tokens > 0)
        hipLaunchKernelGGL(k_loss_out<DT>, dim3(a.tokens), block, 0, s, a, static_cast<const float*>(p.acc), p.ldx, p.splits);
    return hipGetLastError();
}

}  // namespace

uint64_t loss_workspace(const RowTable& vocab, int nranks, uint64_t tokens, uint64_t cols, int dtype) {
    uint64_t entries = 0;
    for (int r = 0; r < nranks; r++)
        for (uint32_t V = vocab.start[r + 1] - vocab.start[r], f = 0; f < V; f += kPiece)
            entries += ceil_div(V - f < kPiece ? V - f : kPiece, kStatsRows);
    Parts w;
    w.take(entries * tokens * sizeof(float2));
    w.take(tokens * 4);
    pad_parts(w, tokens, cols, loss_piece(vocab, nranks, tokens, cols, dtype, 0), dtype);
    return w.at;
}

// Vocabulary rows per piece: the largest shard, at most what was asked for
// (16384 by default).
uint32_t loss_piece(const RowTable& vocab, int nranks, uint64_t, uint64_t, int, uint64_t asked) {
    uint64_t most = 1;
    for (int r = 0; r < nranks; r++)
        if (vocab.start[r + 1] - vocab.start[r] > most) most = vocab.start[r + 1] - vocab.start[r];
    const uint64_t want = asked > 0 ? asked : kPiece;
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
