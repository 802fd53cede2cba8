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
// again, one piece of the vocabulary at a time (a piece may span ranks), and
// multiplies the piece's d into both gradients.
//
// All three products are the same routine: out[n][m] = sum_k A(m, k) B(n, k),
// where an operand lies in memory either with k contiguous (kRows: hidden,
// weight in the logits; d in dhidden) or with m or n contiguous (kCols:
// weight in dhidden, hidden and d in dweight).  The second kind is turned on
// the way from LDS to the registers, so nothing is stored transposed.
//
// 4096 tokens x 4096, 131072 rows in bf16: the forward pass takes 3.4 ms, 1.29
// PFLOP/s, with gradients 14.2 ms: 1.24 PFLOP/s over its four products (the logits
// twice), where a plain matrix product of that size reaches 1.46.  The matrix
// units are busy for 68% of the time, at a clock of 1.8 GHz: bound by them and by
// power.  In fp32 (154 TFLOP/s in a large product) 509 tokens x 1000, 10007 rows
// take 365 us with gradients, 111 TFLOP/s, the matrix units of a running workgroup
// 83% busy.
#include "dt_step_device.h"

namespace dt {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
#define DT_LDS __attribute__((address_space(3)))

constexpr int kChunks = 4;             // 16-byte chunks of the summed index per step
constexpr int kStepBytes = kChunks * 16;
constexpr int kThreads = 256;          // workgroups of the kernels without a matrix tile
enum { kRows = 0, kCols = 1 };

// A workgroup's tile of `out`: BM rows of A by BN rows of B, cut among GM x GN
// waves.  Both operands go through LDS, four steps of the summed index at a
// time: one step is in registers and multiplied, the next one is read from
// LDS, and the others are on their way from memory.
template <int BM_, int BN_, int GM_, int GN_>
struct Shape {
    static constexpr int BM = BM_, BN = BN_, GM = GM_, GN = GN_;
    static constexpr int waves = GM * GN, threads = waves * 64;
    static constexpr int WM = BM / GM, WN = BN / GN;  // a wave's part
    static constexpr int MI = WM / 16, NI = WN / 16;  // in matrix instructions of 16 x 16
    static constexpr int stage = (BM + BN) * kChunks;     // u32x4 of a step in LDS
    static constexpr int loads_a = BM / 16 / waves, loads_b = BN / 16 / waves;  // load instructions of 1 KiB per wave and step
    static constexpr int loads = loads_a + loads_b;
};

// A buffer resource from values that are the same in every lane, kept in scalar registers.
__device__ __forceinline__ rsrc_t scalar_rsrc(const char* p, uint32_t bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    const uint64_t lo = uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(at))), hi = uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(at >> 32)));
    return make_rsrc(reinterpret_cast<const char*>(hi << 32 | lo), __builtin_amdgcn_readfirstlane(bytes));
}

// An operand gives the bytes of each step as a buffer resource that ends
// behind the last valid row (empty when not `any`), so what lies past it
// loads zeros without touching memory.
//
// kRows: rows of `pitch` bytes, read up to `bytes`, a multiple of 16.  TAIL: the
// row ends before that, after `valid` bytes (a multiple of 4), and what is read
// behind its end, the next row's first values, is masked in the registers: the
// other operand has zeros there, but an infinity times zero is NaN.
template <bool TAIL>
struct RowOperand {
    static constexpr bool tail = TAIL;
    const char* p;     // the tile's first row
    uint32_t rows, pitch, bytes, valid;
    __device__ __forceinline__ rsrc_t at(uint32_t step, bool any) const {
        return scalar_rsrc(p + step * kStepBytes, any && rows > 0 ? rows * pitch - step * kStepBytes : 0);
    }
    __device__ __forceinline__ uint32_t left(uint32_t step) const { return bytes - step * kStepBytes; }
    // the lane's chunk of a step, without what lies behind the row
    __device__ __forceinline__ u32x4 cut(u32x4 v, uint32_t step) const {
        if constexpr (TAIL) {
            const uint32_t at = step * kStepBytes + (threadIdx.x >> 4 & 3) * 16;
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = at + 4 * e < valid ? v[e] : 0;
        }
        return v;
    }
};
// The rows of d in two parts, the second one `part` bytes behind the first: its
// steps follow after the first one's `steps`.
struct PartsOperand : RowOperand<false> {
    uint32_t steps;
    uint64_t part;
    __device__ __forceinline__ rsrc_t at(uint32_t step, bool any) const {
        const bool second = step >= steps;
        const uint32_t s = second ? step - steps : step;
        return scalar_rsrc(p + (second ? part : 0) + s * kStepBytes, any && rows > 0 ? rows * pitch - s * kStepBytes : 0);
    }
    __device__ __forceinline__ uint32_t left(uint32_t step) const { return bytes - (step >= steps ? step - steps : step) * kStepBytes; }
};
// kCols: row k of `pitch` bytes holds the operand's m (or n) side by side.
// PARTS 2: after the steps of all rows come those of a second part, `part` bytes
// behind the first (0: the same rows again).
template <int KR, int PARTS>
struct ColOperand {
    const char* p;     // row 0 at the tile's first column
    uint32_t rows, pitch, skip;   // skip: bytes of a row before the tile
    uint64_t part;
    __device__ __forceinline__ rsrc_t at(uint32_t step, bool any) const {
        const uint32_t steps = (rows + KR - 1) / KR;
        const bool second = PARTS > 1 && step >= steps;
        const uint32_t k = (second ? step - steps : step) * KR, n = any && k < rows ? rows - k : 0;
        return scalar_rsrc(p + (second ? part : 0) + uint64_t(k) * pitch, n > 0 ? (n < KR ? n : KR) * pitch - skip : 0);
    }
    __device__ __forceinline__ uint32_t left(uint32_t) const { return UINT32_MAX; }
    __device__ __forceinline__ u32x4 cut(u32x4 v, uint32_t) const { return v; }
};

// Rows of k per step and the turned layout of a kCols operand in LDS: a row
// of k holds R elements in units of 16, unit u of row k in place u ^ f(k),
// where f differs between the rows that one read instruction touches.
template <int DT, int R>
struct ColTile {
    static constexpr int ES = DT == kBF16 ? 2 : 4;
    static constexpr int KR = kStepBytes / ES;
    static constexpr int row_bytes = R * ES, units = R / 16, unit_bytes = 16 * ES;
    static constexpr int per_load = 1024 / row_bytes;  // rows per load instruction
    static __device__ __forceinline__ uint32_t f(uint32_t k) {
        if constexpr (DT == kBF16) return units >= 8 ? (k & 3) | ((k >> 3) & 1) << 2 : k & 3;
        else return (k >> 2) & 3;
    }
};

// kRows: the chunk of row r that lies in place p of the row's 64 bytes is p ^
// row_turn(r).  A read takes one chunk of 16 rows in lanes 0-15, the next chunk
// in 16-31 and so on, and serves 16 lanes at a time: 0-3, 12-15, 20-23, 24-27,
// then 4-11, 16-19, 28-31, and the same of the upper half.  Rows four apart lie
// on the same banks; turned by 0, 2, 3, 1 in fours, each such 16 lanes take all
// 64 banks once (turned by 0, 1, 2, 3 half the reads' cycles were conflicts).
__device__ __forceinline__ uint32_t row_turn(uint32_t row) {
    const uint32_t q = row >> 2 & 3;
    return (q & 1) << 1 ^ (q >> 1) * 3;
}

// One load instruction of the wave brings 1 KiB of the operand's step into
// LDS, 16 bytes per lane in lane order: the lane's place in the step.
template <int DT, int MODE, int R>
__device__ __forceinline__ uint32_t load_place(uint32_t group, uint32_t pitch) {
    const uint32_t lane = threadIdx.x & 63;
    if constexpr (MODE == kRows) {
        // 16 rows of 64 bytes: lane l brings row l / 4
        const uint32_t row = lane >> 2;
        return (group * 16 + row) * pitch + ((lane & 3) ^ row_turn(row)) * 16;
    } else {
        typedef ColTile<DT, R> C;
        constexpr uint32_t slots = C::row_bytes / 16, per_unit = C::unit_bytes / 16;
        const uint32_t k = group * C::per_load + lane / slots, slot = lane % slots;
        return k * pitch + ((slot / per_unit) ^ C::f(k)) * C::unit_bytes + slot % per_unit * 16;
    }
}
// `groups` load instructions of the wave; kRows: zeros behind a row's last byte.
template <int MODE, int N, typename OP>
__device__ __forceinline__ void load_step(const OP& op, uint32_t step, bool any, const uint32_t (&place)[N], u32x4* to) {
    const rsrc_t r = op.at(step, any);
    const uint32_t lane = threadIdx.x & 63, c = ((lane & 3) ^ row_turn(lane >> 2)) * 16;
#pragma unroll
    for (int i = 0; i < N; i++) {
        const bool in = MODE == kCols || c < op.left(step);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (DT_LDS void*)(to + i * 64), 16, int(in ? place[i] : 0x80000000u), 0, 0, 0);
    }
}

// The wave's registers of 16 rows (of A or B): lane l gets row l % 16 and
// chunk l / 16 of the step.  `place` is the lane's byte in the operand's part
// of a stage for the wave's first 16 rows; the others are a constant away.
template <int DT, int MODE, int R>
__device__ __forceinline__ uint32_t fragment_place(uint32_t at) {
    const uint32_t lane = threadIdx.x & 63;
    if constexpr (MODE == kRows) {
        const uint32_t row = at + (lane & 15);
        return row * kStepBytes + ((lane >> 4) ^ row_turn(row)) * 16;
    } else {
        typedef ColTile<DT, R> C;
        // bf16: row k = 8 (lane / 16) + lane % 16 / 4 of the first transposing read; fp32: k = 4 (lane / 16)
        const uint32_t k = DT == kBF16 ? (lane >> 4) * 8 + ((lane & 15) >> 2) : (lane >> 4) * 4;
        return k * C::row_bytes + ((at / 16) ^ C::f(k)) * C::unit_bytes + (DT == kBF16 ? (lane & 3) * 8 : (lane & 15) * 4);
    }
}
template <int DT, int MODE, int R>
__device__ __forceinline__ u32x4 fragment(const u32x4* tile, uint32_t place, int i) {
    const char* base = reinterpret_cast<const char*>(tile);
    if constexpr (MODE == kRows) {
        return *reinterpret_cast<const u32x4*>(base + place + i * 16 * kStepBytes);
    } else {
        typedef ColTile<DT, R> C;
        const char* from = base + (place ^ (i * C::unit_bytes));  // unit + i: the wave's first unit is a multiple of the others' number
        u32x4 v;
        if constexpr (DT == kBF16) {
            // two transposing reads of 4 rows of k x 16 each
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DT_LDS s16x4*)(from + h * 4 * C::row_bytes));
                uint32_t w[2];
                __builtin_memcpy(w, &x, 8);
                v[2 * h] = w[0];
                v[2 * h + 1] = w[1];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = *reinterpret_cast<const uint32_t*>(from + e * C::row_bytes);
        }
        return v;
    }
}

// Waits until at most `loads` of this wave's loads and `reads` of its LDS reads
// (15: as many as the counter holds) are outstanding, then for the workgroup's
// other waves.
template <int loads, int reads>
__device__ __forceinline__ void arrive() {
    static_assert(loads < 64 && reads < 16, "the counters hold 6 and 4 bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((loads & 15) | (loads >> 4) << 14 | 7 << 4 | reads << 8);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// acc[i][j][e] over steps [lo, hi): row m = WM (wave % GM) + 16 i + 4 (lane /
// 16) + e of A's tile, row n = WN (wave / GM) + 16 j + lane % 16 of B's.
//
// The four LDS stages are arrays of their own, and the loop goes round them
// with constant indices: only so does the compiler see that a read of one
// stage need not wait for the loads into another.
template <int DT, typename S, int MA, int MB, typename OA, typename OB>
__device__ __forceinline__ void matrix_tile(const OA& A, const OB& B, uint32_t lo, uint32_t hi, f32x4 (&acc)[S::MI][S::NI]) {
    __shared__ u32x4 s0[S::stage], s1[S::stage], s2[S::stage], s3[S::stage];
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int i = 0; i < S::MI; i++)
#pragma unroll
        for (int j = 0; j < S::NI; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (lo >= hi) return;
    const uint32_t wm = (wave % S::GM) * S::WM, wn = (wave / S::GM) * S::WN;
    // the wave's shares of A's and B's groups of 1 KiB
    uint32_t pa[S::loads_a], pb[S::loads_b];
#pragma unroll
    for (int i = 0; i < S::loads_a; i++) pa[i] = load_place<DT, MA, S::BM>(wave * S::loads_a + i, A.pitch);
#pragma unroll
    for (int i = 0; i < S::loads_b; i++) pb[i] = load_place<DT, MB, S::BN>(wave * S::loads_b + i, B.pitch);
    // The loop runs in whole rounds of four steps: what is loaded for the steps
    // behind the last one is zeros (from an empty buffer, no memory is read), so
    // a wave's outstanding loads can be counted and the loop has one exit.
    auto load = [&](uint32_t step, u32x4* to) {
        load_step<MA>(A, step, step < hi, pa, to + wave * S::loads_a * 64);
        load_step<MB>(B, step, step < hi, pb, to + S::BM * kChunks + wave * S::loads_b * 64);
    };
    load(lo, s0);
    load(lo + 1, s1);
    load(lo + 2, s2);
    arrive<2 * S::loads, 15>();
    u32x4 fa[S::MI], fb[2][S::NI];
    uint32_t ra = fragment_place<DT, MA, S::BM>(wm), rb = fragment_place<DT, MB, S::BN>(wn);
#pragma unroll
    for (int i = 0; i < S::MI; i++) fa[i] = A.cut(fragment<DT, MA, S::BM>(s0, ra, i), lo);
#pragma unroll
    for (int j = 0; j < S::NI; j++) fb[0][j] = fragment<DT, MB, S::BN>(s0 + S::BM * kChunks, rb, j);
    // Step `step`: its registers are loaded, and the next step's bytes are in
    // LDS once all waves are here.  The stage that is loaded into, the one
    // before this step's, was read two turns ago, so the last turn's reads may
    // still be on their way at the barrier, but none before them: LDS answers in
    // order, and a turn reads each fragment with one instruction at least (kCols:
    // two, as none reads from more than two places).  Their use in the last turn
    // does not see to that, since the compiler may move a matrix instruction, and
    // its wait, behind the barrier.  A row of A's registers takes the next step's
    // as soon as it is multiplied; behind the last step these are bytes that
    // nothing uses.
    constexpr int turn_reads = S::MI * (MA == kRows ? 1 : 2) + S::NI * (MB == kRows ? 1 : 2);
    auto turn = [&](uint32_t step, u32x4* free, const u32x4* following, const u32x4 (&now)[S::NI], u32x4 (&next)[S::NI]) {
        arrive<S::loads, turn_reads < 15 ? turn_reads : 15>();
        load(step + 3, free);
        // keeps the compiler from holding every fragment's address of every stage in a register
        asm volatile("" : "+v"(ra), "+v"(rb));
#pragma unroll
        for (int j = 0; j < S::NI; j++) next[j] = fragment<DT, MB, S::BN>(following + S::BM * kChunks, rb, j);
#pragma unroll
        for (int i = 0; i < S::MI; i++) {
#pragma unroll
            for (int j = 0; j < S::NI; j++) {
                if constexpr (DT == kBF16) {
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fa[i]),
                                                                        __builtin_bit_cast(bf16x8, now[j]), acc[i][j], 0, 0, 0);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(fa[i][e]), __uint_as_float(now[j][e]),
                                                                         acc[i][j], 0, 0, 0);
                }
            }
            fa[i] = A.cut(fragment<DT, MA, S::BM>(following, ra, i), step + 1);
        }
    };
    for (uint32_t step = lo; step < hi; step += 4) {
        turn(step, s3, s1, fb[0], fb[1]);
        turn(step + 1, s0, s2, fb[1], fb[0]);
        turn(step + 2, s1, s3, fb[0], fb[1]);
        turn(step + 3, s2, s0, fb[1], fb[0]);
    }
    arrive<0, 0>();  // nothing is on its way into LDS when the workgroup ends
}

// Tile `id` of mt x nt in an order that keeps an XCD's workgroups on
// neighbouring tiles: ids go round the 8 XCDs, so each XCD gets a run of the
// tiles, walked in bands of 8 rows of tiles.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t mt, uint32_t nt, uint32_t& m, uint32_t& n) {
    const uint32_t total = mt * nt, q = total / 8, rem = total % 8, x = id % 8;
    const uint32_t t = x * q + (x < rem ? x : rem) + id / 8;
    const uint32_t band = t / (8 * nt), first = band * 8, in = t - band * 8 * nt;
    const uint32_t high = mt - first < 8 ? mt - first : 8;
    // divisions run on the vector unit: back into scalar registers, where the buffer resources are built
    m = __builtin_amdgcn_readfirstlane(first + in % high);
    n = __builtin_amdgcn_readfirstlane(in / high);
}

// exp(x): the argument's product with log2 e is off by half a step of |x| log2 e,
// which adds |x| half steps to the result's error.  So the difference is taken
// before the product: where a token's probability is near 1 its gradient is
// what is left of 1 - p, and a product of logit and lse apart would leave |lse|
// half steps in it.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// Four values rounded to the dtype and stored as one (`to` aligned for it); zeros unless `use`.
template <int DT>
__device__ __forceinline__ void store_quad(typename Elem<DT>::type* to, f32x4 v, bool use) {
    if constexpr (DT == kBF16) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        uint2 o;
        o.x = __builtin_bit_cast(uint32_t, bf16x2{__bf16(v[0]), __bf16(v[1])});
        o.y = __builtin_bit_cast(uint32_t, bf16x2{__bf16(v[2]), __bf16(v[3])});
        if (!use) o = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(to) = o;
    } else {
        *reinterpret_cast<f32x4*>(to) = use ? v : f32x4{0.f, 0.f, 0.f, 0.f};
    }
}

// A piece of the vocabulary: the parts of it that single ranks hold.
struct Segments {
    const char* weight[kMaxRanksHost];   // the part's first row, rows of `pitch` bytes
    char* dweight[kMaxRanksHost];        // its gradient, rows of the caller's width
    uint32_t count[kMaxRanksHost];       // rows
    uint32_t vocab[kMaxRanksHost];       // first row in the whole vocabulary
    uint32_t tile[kMaxRanksHost + 1];    // first tile of vocabulary rows
    uint32_t col[kMaxRanksHost + 1];     // first column in d; each part ends on a whole step
    int n;
};
__device__ __forceinline__ int segment_of(const uint32_t* first, int n, uint32_t at) {
    int s = 0;
    while (s + 1 < n && at >= first[s + 1]) s++;
    return s;
}

struct LossProblem {
    const char* hidden;      // [tokens] rows of `pitch` bytes
    const int64_t* targets;
    const float* lse;
    const float* dloss;
    uint32_t hpitch;         // bytes between hidden's rows, a multiple of 16; all of them valid
    uint32_t wpitch;         // bytes between weight's rows; not a multiple of 16: the kernels' TAIL form
    uint32_t tokens, cols, vocab;
    int64_t ignore_index;
};
__device__ __forceinline__ bool counted(const LossProblem& a, int64_t t) {
    return t != a.ignore_index && t >= 0 && t < int64_t(a.vocab);
}

// ---------------------------------------------------------------- forward --
struct StatsArgs {
    uint32_t token_tiles;
    uint32_t entry, entries;      // the launch's first tile among all, and how many all are
    float2* part;                 // [tokens][entries]: maximum, sum of exponentials
    float* target;                // [tokens]: the target's logit
};

// (top, s) joined with another maximum and sum.
__device__ __forceinline__ void join(float& top, float& s, float top2, float s2) {
    const float t = fmaxf(top, top2), base = t > -INFINITY ? t : 0.f;
    s = s * exp_of(top - base) + s2 * exp_of(top2 - base);
    top = t;
}

template <int DT, typename S, bool TAIL>
__global__ __launch_bounds__(S::threads) void k_loss_stats(LossProblem a, Segments g, StatsArgs q) {
    __shared__ float2 part[S::GM][S::BN];
    uint32_t mt, nt;
    tile_of(blockIdx.x, g.tile[g.n], q.token_tiles, mt, nt);
    const int sg = segment_of(g.tile, g.n, mt);
    const uint32_t m0 = (mt - g.tile[sg]) * S::BM, n0 = nt * S::BN, left = g.count[sg] - m0;
    f32x4 acc[S::MI][S::NI];
    const RowOperand<TAIL> A{g.weight[sg] + uint64_t(m0) * a.wpitch, left < S::BM ? left : S::BM, a.wpitch, a.hpitch,
                             a.cols * uint32_t(sizeof(typename Elem<DT>::type))};
    const RowOperand<false> B{a.hidden + uint64_t(n0) * a.hpitch, a.tokens - n0 < S::BN ? a.tokens - n0 : S::BN, a.hpitch, a.hpitch, a.hpitch};
    matrix_tile<DT, S, kRows, kRows>(A, B, 0, (a.hpitch + kStepBytes - 1) / kStepBytes, acc);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t wm = wave % S::GM, wn = wave / S::GM;
    const uint32_t mlane = wm * S::WM + (lane >> 4) * 4;  // acc[i][j][e] is row mlane + 16 i + e of the tile
    if (left < S::BM) {  // rows behind the shard's last one
#pragma unroll
        for (int i = 0; i < S::MI; i++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (mlane + i * 16 + e >= left) {
#pragma unroll
                    for (int j = 0; j < S::NI; j++) acc[i][j][e] = -INFINITY;
                }
    }
#pragma unroll
    for (int j = 0; j < S::NI; j++) {
        const uint32_t nl = wn * S::WN + j * 16 + (lane & 15), n = n0 + nl;
        const int64_t t = n < a.tokens ? a.targets[n] - int64_t(g.vocab[sg]) - int64_t(m0) : -1;
        const bool here = t >= 0 && t < int64_t(left < S::BM ? left : S::BM);
        if (__any(here)) {  // few tiles hold a target of their tokens
#pragma unroll
            for (int i = 0; i < S::MI; i++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (here && uint32_t(t) == mlane + i * 16 + e) q.target[n] = acc[i][j][e];
        }
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < S::MI; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) top = fmaxf(top, acc[i][j][e]);
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
        for (int w = 1; w < S::GM; w++) join(top, s, part[w][nl].x, part[w][nl].y);
        q.part[uint64_t(n0 + nl) * q.entries + q.entry + mt] = make_float2(top, s);
    }
}

// One wave per token: the tiles' maxima and sums joined, every rank's loss and lse written.
struct LossOut {
    float* loss[kMaxRanksHost];
    float* lse[kMaxRanksHost];
    int nranks;
};
__global__ __launch_bounds__(kThreads) void k_loss_join(LossProblem a, StatsArgs q, LossOut o) {
    const uint32_t n = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (n >= a.tokens) return;
    float top = -INFINITY, s = 0.f;
    for (uint32_t i = lane; i < q.entries; i += 64) {
        const float2 v = q.part[uint64_t(n) * q.entries + i];
        join(top, s, v.x, v.y);
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) join(top, s, __shfl_xor(top, m), __shfl_xor(s, m));
    // the first lane's for every rank: a join rounds differently with its sides swapped
    const float lse = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(top + logf(s))));
    const float loss = counted(a, a.targets[n]) ? lse - q.target[n] : 0.f;
    if (lane < uint32_t(o.nranks)) {
        o.lse[lane][n] = lse;
        o.loss[lane][n] = loss;
    }
}

// --------------------------------------------------------------- backward --
// d in bf16 is rounded once more than the gradients themselves.  Two things keep
// that small beside their own rounding:
//  - Where few tokens make a sum, one of them may carry a whole row of a gradient,
//    and half a step of d shows in all of it.  So up to kTwoPartTokens d is kept in
//    two parts, its rounding and the rest's, and both enter the products, which are
//    bound by the weight's bytes there (error of 12 tokens' gradients against 64
//    bits: 3.1e-3 with one part, 1.7e-3, that of the result's rounding, with two).
//  - Above it d is kept relative to the mantissa of the largest |dloss|, which the
//    products are multiplied with in fp32.  A mean's gradient is the same for every
//    token, and so was its rounding, all in one direction (3481 tokens: 2.8e-3);
//    relative to that mantissa it is a power of two.  The exponent stays in d:
//    divided by a dloss of 1e38, the other tokens' d would vanish.
// The cost of two parts for many tokens, where the matrix units are the bound: 4096
// tokens x 4096, 131072 rows take 21.4 ms instead of 14.2, and the gradients are
// off by 1.7e-3 (the rounding of the results alone, as with d in fp32) instead of
// 1.9e-3.
constexpr uint32_t kTwoPartTokens = 512;
int d_parts(uint64_t tokens, int dtype) { return dtype == kBF16 && tokens <= kTwoPartTokens ? 2 : 1; }

// The largest finite |dloss| of the tokens that count, in kScaleParts shares.
constexpr int kScaleParts = 64;
__global__ __launch_bounds__(kThreads) void k_loss_scale(LossProblem a, float* scale) {
    __shared__ float tmp[kThreads / 64];
    float top = 0.f;
    for (uint32_t n = blockIdx.x * kThreads + threadIdx.x; n < a.tokens; n += kScaleParts * kThreads) {
        const float f = fabsf(a.dloss[n]);
        if (counted(a, a.targets[n]) && f < INFINITY) top = fmaxf(top, f);
    }
    top = wave_max(top);
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 64; w++) top = fmaxf(top, tmp[w]);
        scale[blockIdx.x] = top;
    }
}

struct DPiece {
    char* hidden;     // the first piece: where the tokens' rows go for dweight; NULL: nowhere
    char* d;          // [parts][tokens] rows of ldv elements: the piece's d, each segment's padding zero
    float* acc;       // [splits][tokens][ldx]
    const float* scale;  // [kScaleParts], NULL: 1
    uint64_t ldv, ldx;
    uint32_t mt, nt;  // tiles of the launch
    uint32_t splits;  // workgroups that share one tile's sum over the piece
    int add;          // acc holds the earlier pieces' sum
};

// dweight reads a copy of hidden with rows of zeros for the tokens that are left
// out: their d is zero, but zero times what a padded row holds may be NaN.  The
// workgroups that form the first piece's d make it, each its share of the token
// tile's rows, without a launch of its own (4.8 us of 369 for 509 x 1000 fp32).
template <typename S>
__device__ __forceinline__ void copy_tokens(const LossProblem& a, uint32_t n0, uint32_t part, uint32_t parts, char* to) {
    const uint32_t units = a.hpitch / 16, rows = a.tokens - n0 < S::BN ? a.tokens - n0 : S::BN;
    for (uint32_t i = part * S::threads + threadIdx.x; i < rows * units; i += parts * S::threads) {
        const uint64_t n = n0 + i / units, at = n * a.hpitch + i % units * 16;
        const bool use = counted(a, a.targets[n]);
        *reinterpret_cast<u32x4*>(to + at) = use ? *reinterpret_cast<const u32x4*>(a.hidden + at) : u32x4{0, 0, 0, 0};
    }
}

// What d is relative to, 1 or more and less than 2 (the whole wave asks; the same
// value in every lane).
__device__ __forceinline__ float scale_of(const DPiece& p) {
    if (p.scale == nullptr) return 1.f;
    const float top = wave_max(p.scale[threadIdx.x & 63]);
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(top) & 0x7FFFFFu) | 0x3F800000u);
}

template <int DT, typename S, bool TAIL, int PARTS>
__global__ __launch_bounds__(S::threads) void k_loss_d(LossProblem a, Segments g, DPiece p) {
    typedef typename Elem<DT>::type T;
    uint32_t mt, nt;
    tile_of(blockIdx.x, g.tile[g.n], p.nt, mt, nt);
    const int sg = segment_of(g.tile, g.n, mt);
    const uint32_t m0 = (mt - g.tile[sg]) * S::BM, n0 = nt * S::BN;
    const uint32_t count = g.count[sg], padded = g.col[sg + 1] - g.col[sg];
    const uint32_t left = count > m0 ? count - m0 : 0;  // the last tile may lie in the padding alone
    f32x4 acc[S::MI][S::NI];
    const RowOperand<TAIL> A{g.weight[sg] + uint64_t(m0) * a.wpitch, left < S::BM ? left : S::BM, a.wpitch, a.hpitch,
                             a.cols * uint32_t(sizeof(typename Elem<DT>::type))};
    const RowOperand<false> B{a.hidden + uint64_t(n0) * a.hpitch, a.tokens - n0 < S::BN ? a.tokens - n0 : S::BN, a.hpitch, a.hpitch, a.hpitch};
    matrix_tile<DT, S, kRows, kRows>(A, B, 0, (a.hpitch + kStepBytes - 1) / kStepBytes, acc);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t mlane = (wave % S::GM) * S::WM + (lane >> 4) * 4;
    T* d = reinterpret_cast<T*>(p.d) + g.col[sg] + m0;
    const float scale = scale_of(p);
#pragma unroll
    for (int j = 0; j < S::NI; j++) {
        const uint32_t n = n0 + (wave / S::GM) * S::WN + j * 16 + (lane & 15);
        if (n >= a.tokens) continue;
        const int64_t t = a.targets[n];
        const float lse = a.lse[n];
        const bool use = counted(a, t);
        const float f = use ? a.dloss[n] / scale : 0.f;
        // d = p f; the target's row and the rows behind the shard's last one are mended below
#pragma unroll
        for (int i = 0; i < S::MI; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) acc[i][j][e] = exp_of(acc[i][j][e] - lse) * f;
        const int64_t at = t - int64_t(g.vocab[sg]) - int64_t(m0);
        const uint32_t hit = use && at >= 0 && at < S::BM ? uint32_t(at) : UINT32_MAX;  // the target's row in the tile
        if (__any(hit != UINT32_MAX) || left < S::BM) {
#pragma unroll
            for (int i = 0; i < S::MI; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const uint32_t m = mlane + i * 16 + e;
                    if (hit == m) acc[i][j][e] -= f;
                    if (m >= left) acc[i][j][e] = 0.f;
                }
        }
#pragma unroll
        for (int i = 0; i < S::MI; i++) {
            const uint32_t m = mlane + i * 16;
            // a part's width is a multiple of 4: the four are all inside it or all behind it
            if (m0 + m >= padded) continue;
            store_quad<DT>(d + uint64_t(n) * p.ldv + m, acc[i][j], use);
            if constexpr (PARTS > 1) {
                f32x4 rest;
#pragma unroll
                for (int e = 0; e < 4; e++) rest[e] = acc[i][j][e] - float(__bf16(acc[i][j][e]));
                store_quad<DT>(d + (uint64_t(a.tokens) + n) * p.ldv + m, rest, use);
            }
        }
    }
    if (p.hidden != nullptr) copy_tokens<S>(a, n0, mt, g.tile[g.n], p.hidden);
}

// The weight rows of a piece as the summed index: step by step through the
// segments, each of whole steps, zeros behind a segment's last row.  PARTS 2: all
// of them a second time.
template <int KR, int PARTS>
struct WeightOperand {
    const Segments& g;
    uint32_t pitch, skip, steps;
    mutable int sg;
    __device__ __forceinline__ rsrc_t at(uint32_t step, bool any) const {
        const bool second = PARTS > 1 && step >= steps;
        const uint32_t k = (second ? step - steps : step) * KR;
        if (PARTS > 1 && k < g.col[sg]) sg = 0;
        while (sg + 1 < g.n && k >= g.col[sg + 1]) sg++;
        const uint32_t row = k - g.col[sg], n = any && row < g.count[sg] ? g.count[sg] - row : 0;
        return scalar_rsrc(g.weight[sg] + uint64_t(row) * pitch + skip, n > 0 ? (n < KR ? n : KR) * pitch - skip : 0);
    }
    __device__ __forceinline__ uint32_t left(uint32_t) const { return UINT32_MAX; }
    __device__ __forceinline__ u32x4 cut(u32x4 v, uint32_t) const { return v; }
};

// acc[split][t][h] (+)= sum over the split's part of the piece of d[t][v] weight[v][h].
template <int DT, typename S, int PARTS>
__global__ __launch_bounds__(S::threads) void k_loss_dhidden(LossProblem a, Segments g, DPiece p) {
    typedef typename Elem<DT>::type T;
    constexpr int KR = kStepBytes / int(sizeof(T));
    uint32_t mt, nt;
    tile_of(blockIdx.x, p.mt, p.nt, mt, nt);
    const uint32_t m0 = mt * S::BM, n0 = nt * S::BN;
    const uint32_t pitch = uint32_t(p.ldv * sizeof(T)), steps = pitch / kStepBytes;
    // the first `more` splits take one step more than the others
    const uint32_t all = steps * PARTS, y = blockIdx.y;
    const uint32_t each = __builtin_amdgcn_readfirstlane(all / p.splits), more = all - each * p.splits;
    const uint32_t lo = y * each + (y < more ? y : more), hi = lo + each + (y < more ? 1 : 0);
    f32x4 acc[S::MI][S::NI];
    const WeightOperand<KR, PARTS> A{g, a.wpitch, m0 * uint32_t(sizeof(T)), steps, 0};
    const RowOperand<false> B{p.d + uint64_t(n0) * pitch, a.tokens - n0 < S::BN ? a.tokens - n0 : S::BN, pitch, pitch, pitch};
    if constexpr (PARTS > 1) matrix_tile<DT, S, kCols, kRows>(A, PartsOperand{B, steps, uint64_t(a.tokens) * pitch}, lo, hi, acc);
    else matrix_tile<DT, S, kCols, kRows>(A, B, lo, hi, acc);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float* to = p.acc + uint64_t(blockIdx.y) * a.tokens * p.ldx;
    const float scale = scale_of(p);
#pragma unroll
    for (int j = 0; j < S::NI; j++)
#pragma unroll
        for (int i = 0; i < S::MI; i++) {
            const uint32_t n = n0 + (wave / S::GM) * S::WN + j * 16 + (lane & 15);
            const uint32_t m = m0 + (wave % S::GM) * S::WM + i * 16 + (lane >> 4) * 4;
            if (n >= a.tokens || m >= p.ldx) continue;
            f32x4* o = reinterpret_cast<f32x4*>(to + uint64_t(n) * p.ldx + m);
            *o = p.add ? *o + acc[i][j] * scale : acc[i][j] * scale;
        }
}

// dweight[v][h] = sum_t d[t][v] hidden[t][h].
template <int DT, typename S, int PARTS>
__global__ __launch_bounds__(S::threads) void k_loss_dweight(LossProblem a, Segments g, DPiece p) {
    typedef typename Elem<DT>::type T;
    constexpr int KR = kStepBytes / int(sizeof(T));
    uint32_t mt, nt;
    tile_of(blockIdx.x, p.mt, g.tile[g.n], mt, nt);
    const int sg = segment_of(g.tile, g.n, nt);
    const uint32_t m0 = mt * S::BM, n0 = (nt - g.tile[sg]) * S::BN;
    f32x4 acc[S::MI][S::NI];
    constexpr uint32_t es = sizeof(T);
    const uint32_t skip = (g.col[sg] + n0) * es;
    const ColOperand<KR, PARTS> A{a.hidden + m0 * es, a.tokens, a.hpitch, m0 * es, 0};
    const ColOperand<KR, PARTS> B{p.d + skip, a.tokens, uint32_t(p.ldv * es), skip, a.tokens * p.ldv * es};
    matrix_tile<DT, S, kCols, kCols>(A, B, 0, (a.tokens + KR - 1) / KR * PARTS, acc);
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    T* out = reinterpret_cast<T*>(g.dweight[sg]);
    const float scale = scale_of(p);
    const bool quads = a.cols % 4 == 0 && reinterpret_cast<uintptr_t>(out) % (4 * sizeof(T)) == 0;
#pragma unroll
    for (int j = 0; j < S::NI; j++)
#pragma unroll
        for (int i = 0; i < S::MI; i++) {
            const uint32_t n = n0 + (wave / S::GM) * S::WN + j * 16 + (lane & 15);
            const uint32_t m = m0 + (wave % S::GM) * S::WM + i * 16 + (lane >> 4) * 4;
            if (n >= g.count[sg] || m >= a.cols) continue;
            T* to = out + uint64_t(n) * a.cols + m;
            if (quads) {
                store_quad<DT>(to, acc[i][j] * scale, true);
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (m + e < a.cols) to[e] = Elem<DT>::put(acc[i][j][e] * scale);
            }
        }
}

// Every rank's dhidden from the sums of the splits, in order, rounded once.
struct DHiddenOut {
    void* p[kMaxRanksHost];
    int nranks;
    int quads;   // rows are whole fours, aligned to them
};
template <int DT>
__global__ __launch_bounds__(kThreads) void k_loss_out(DHiddenOut o, const float* acc, uint32_t tokens, uint32_t cols,
                                                      uint64_t ldx, uint32_t splits) {
    typedef typename Elem<DT>::type T;
    const uint32_t n = blockIdx.x, c = (blockIdx.y * kThreads + threadIdx.x) * 4;
    if (c >= cols) return;
    const float* from = acc + uint64_t(n) * ldx + c;  // ldx is a multiple of 4
    const uint64_t next = uint64_t(tokens) * ldx;
    f32x4 s = *reinterpret_cast<const f32x4*>(from);
    for (uint32_t k0 = 1; k0 < splits; k0 += 8) {
        f32x4 v[8];  // eight splits' loads go out before the first is added
#pragma unroll
        for (int k = 0; k < 8; k++)
            if (k0 + k < splits) v[k] = *reinterpret_cast<const f32x4*>(from + (k0 + k) * next);
#pragma unroll
        for (int k = 0; k < 8; k++)
            if (k0 + k < splits) s += v[k];
    }
    for (int r = 0; r < o.nranks; r++) {
        T* to = static_cast<T*>(o.p[r]) + uint64_t(n) * cols + c;
        if (o.quads) {
            store_quad<DT>(to, s, true);
        } else {
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (c + e < cols) to[e] = Elem<DT>::put(s[e]);
        }
    }
}

// Rows of `cols` elements copied to rows of ld elements (a multiple of 16 bytes).
template <typename T>
__global__ __launch_bounds__(kThreads) void k_pad_rows(const T* src, T* dst, uint32_t cols, uint64_t ld) {
    const uint64_t row = blockIdx.x;
    for (uint32_t c = threadIdx.x; c < ld; c += kThreads) dst[row * ld + c] = c < cols ? src[row * cols + c] : T(0);
}

// hidden's rows of `cols` elements copied to rows of hpitch with zeros behind them,
// and rows of zeros for the tokens that are left out.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_loss_hidden(LossProblem a, const T* src, T* dst) {
    const uint64_t n = blockIdx.x, ld = a.hpitch / sizeof(T);
    const bool use = counted(a, a.targets[n]);
    for (uint32_t c = threadIdx.x; c < ld; c += kThreads) dst[n * ld + c] = use && c < a.cols ? src[n * a.cols + c] : T(0);
}

// -------------------------------------------------------------------- host --
uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }
uint32_t ceil_div(uint64_t n, uint64_t by) { return uint32_t((n + by - 1) / by); }
uint64_t esize(int dtype) { return dtype == kBF16 ? 2 : 4; }
uint64_t step_elems(int dtype) { return kStepBytes / esize(dtype); }

typedef Shape<256, 256, 2, 4> Wide;
typedef Shape<128, 128, 2, 2> Square;
typedef Shape<128, 64, 4, 1> Narrow;
typedef Shape<64, 64, 2, 2> Small;
typedef Shape<64, 16, 1, 1> Tiny;
enum Tile { kWide, kSquare, kNarrow, kSmall, kTiny };
constexpr uint32_t kTileM[] = {256, 128, 128, 64, 64}, kTileN[] = {256, 128, 64, 64, 16};

// The tile for an m x n product of `splits` sums: the largest that still
// fills the 256 CUs.
// tiny: for up to 16 tokens tiles of 16 of them, not to multiply mostly zeros
// (12 x 1088 fp32, 30000 rows: forward 45 -> 32 us, backward 182 -> 146; 1 x
// 4096 bf16, 131072 rows: backward 1250 -> 1090).  The forward pass in bf16 keeps
// tiles of 64 or 128 rows, whose maxima and sums are fewer (187 us, tiny ones 227).
Tile pick_tile(int dtype, uint64_t m, uint64_t n, bool tiny, uint32_t splits = 1) {
    if (tiny && n <= 16) return kTiny;
    const uint64_t square = uint64_t(ceil_div(m, 128)) * ceil_div(n, 128) * splits;
    if (dtype == kF32) return square >= 1024 ? kSquare : kSmall;
    if (n <= 64) return m >= 128 * 128 ? kNarrow : kSmall;
    if (uint64_t(ceil_div(m, 256)) * ceil_div(n, 256) * splits >= 224) return kWide;
    return square >= 192 ? kSquare : kSmall;
}
// launch(Shape) with the shape of `t`; TINY: where pick_tile may say so.
template <int DT, bool TINY, typename F>
void with_tile(Tile t, F&& launch) {
    if constexpr (TINY) {
        if (t == kTiny) return launch(Tiny());
    }
    if constexpr (DT == kBF16) {
        if (t == kWide) return launch(Wide());
        if (t == kNarrow) return launch(Narrow());
    }
    if (t == kSquare) launch(Square());
    else launch(Small());
}
// launch(Shape, TAIL): where weight's rows end inside a 16-byte chunk, the form
// that masks what follows them.
template <int DT, bool TINY, typename F>
void with_rows_of(Tile t, uint32_t wpitch, F&& launch) {
    with_tile<DT, TINY>(t, [&](auto shape) {
        if (wpitch % 16 != 0) launch(shape, std::true_type());
        else launch(shape, std::false_type());
    });
}

// The workspace's parts, each on a 256-byte boundary.
struct Parts {
    uint64_t at = 0;
    uint64_t take(uint64_t n) {
        const uint64_t here = at;
        at += up(n, 256);
        return here;
    }
};

// hidden is read where it is if its rows start and end on 16-byte boundaries;
// otherwise it is copied to such rows with zeros behind them (a small part of the
// call's bytes unless the vocabulary is small too).  weight may lie on any 4-byte boundaries; only bf16 rows of odd
// width, or at odd addresses, are copied, a piece at a time.
struct PadParts {
    uint64_t pitch, hidden, weight;
};
PadParts pad_parts(Parts& w, uint64_t tokens, uint64_t cols, uint64_t piece, int dtype) {
    PadParts b;
    b.pitch = up(cols * esize(dtype), 16);
    b.hidden = w.take(tokens * b.pitch);
    b.weight = dtype == kBF16 ? w.take(piece * b.pitch) : 0;
    return b;
}
bool hidden_direct(const LossArgs& a, int dtype) {
    return a.cols * esize(dtype) % 16 == 0 && reinterpret_cast<uintptr_t>(a.hidden) % 16 == 0;
}
bool weight_direct(const LossArgs& a, int dtype) {
    if (dtype == kF32) return true;
    if (a.cols % 2 != 0) return false;
    for (int r = 0; r < a.nranks; r++)
        if (reinterpret_cast<uintptr_t>(a.weight[r]) % 4 != 0) return false;
    return true;
}

LossProblem problem_of(const LossArgs& a) {
    LossProblem p = {};
    p.hidden = static_cast<const char*>(a.hidden);
    p.targets = a.targets;
    p.lse = a.lse_in;
    p.dloss = a.dloss;
    p.tokens = a.tokens;
    p.cols = a.cols;
    p.vocab = a.vocab.start[a.nranks];
    p.ignore_index = a.ignore_index;
    return p;
}

// Vocabulary rows [first, first + count) as segments; pad != NULL: their rows are in
// the workspace at *pad, one after the other.
Segments segments_of(const LossArgs& a, int dtype, uint32_t first, uint32_t count, const char* pad, uint64_t pitch) {
    Segments g = {};
    const uint64_t es = esize(dtype), row = uint64_t(a.cols) * es;
    for (int r = 0; r < a.nranks; r++) {
        const uint32_t lo = first > a.vocab.start[r] ? first : a.vocab.start[r];
        const uint32_t end = first + count, hi = end < a.vocab.start[r + 1] ? end : a.vocab.start[r + 1];
        if (lo >= hi) continue;
        const uint64_t local = lo - a.vocab.start[r];
        g.weight[g.n] = pad != nullptr ? pad + uint64_t(lo - first) * pitch : static_cast<const char*>(a.weight[r]) + local * row;
        g.dweight[g.n] = a.dweight[r] != nullptr ? static_cast<char*>(a.dweight[r]) + local * row : nullptr;
        g.count[g.n] = hi - lo;
        g.vocab[g.n] = lo;
        g.col[g.n + 1] = g.col[g.n] + uint32_t(up(hi - lo, step_elems(dtype)));
        g.n++;
    }
    return g;
}
void set_tiles(Segments& g, uint32_t rows_per_tile, bool padded) {
    for (int s = 0; s < g.n; s++)
        g.tile[s + 1] = g.tile[s] + ceil_div(padded ? g.col[s + 1] - g.col[s] : g.count[s], rows_per_tile);
}

template <typename T>
void pad_rows(const void* src, char* dst, uint32_t rows, uint32_t cols, uint64_t pitch, hipStream_t s) {
    if (rows > 0)
        hipLaunchKernelGGL(k_pad_rows<T>, dim3(rows), dim3(kThreads), 0, s, static_cast<const T*>(src), reinterpret_cast<T*>(dst),
                           cols, pitch / sizeof(T));
}
void pad_weight(const LossArgs& a, uint32_t first, uint32_t count, char* to, uint64_t pitch, hipStream_t s) {
    const Segments g = segments_of(a, kBF16, first, count, nullptr, pitch);
    for (int i = 0; i < g.n; i++) pad_rows<uint16_t>(g.weight[i], to + uint64_t(g.vocab[i] - first) * pitch, g.count[i], a.cols, pitch, s);
}

// hidden's place and pitch, and weight's pitch; where weight has to be copied
// piece by piece, the place for it.  leave_out: where hidden is copied, without the
// rows of the tokens that are left out (the forward pass gives their lse too).
template <typename T>
char* place_rows(const LossArgs& a, int dtype, const PadParts& pad, LossProblem& p, bool leave_out, hipStream_t s) {
    p.hpitch = uint32_t(pad.pitch);
    if (!hidden_direct(a, dtype)) {
        char* to = a.workspace + pad.hidden;
        if (!leave_out) pad_rows<T>(a.hidden, to, a.tokens, a.cols, pad.pitch, s);
        else if (a.tokens > 0)
            hipLaunchKernelGGL(k_loss_hidden<T>, dim3(a.tokens), dim3(kThreads), 0, s, p, static_cast<const T*>(a.hidden), reinterpret_cast<T*>(to));
        p.hidden = to;
    }
    const bool direct = weight_direct(a, dtype);
    p.wpitch = direct ? a.cols * uint32_t(sizeof(T)) : uint32_t(pad.pitch);
    return direct ? nullptr : a.workspace + pad.weight;
}

// Vocabulary rows of one launch of the forward pass: HIP counts a launch's
// threads in 32 bits, so it stays within 2^22 tiles of at most 512 threads.
// Never fewer than kLossPiece rows, for no more tokens than the call takes.
uint32_t stats_piece(uint32_t vocab, uint32_t tokens) {
    constexpr uint32_t most = 1 << 22;
    static_assert(most / (DT_MAX_LOSS_TOKENS / 128) * 128 >= kLossPiece, "stats_entries counts pieces of kLossPiece rows");
    const uint64_t rows = uint64_t(most / ceil_div(tokens, 128)) * 128;
    return uint32_t(rows < vocab ? rows : vocab);
}

uint64_t stats_entries(const RowTable& vocab, int nranks) {
    // at most one entry per 64 rows of a shard, and one per shard and piece end
    uint64_t n = 0;
    for (int r = 0; r < nranks; r++) n += ceil_div(vocab.start[r + 1] - vocab.start[r], 64);
    return n + 2 * ceil_div(vocab.start[nranks], kLossPiece);
}

template <int DT>
hipError_t forward(const LossArgs& a, hipStream_t s) {
    typedef typename Elem<DT>::type T;
    const uint32_t V = a.vocab.start[a.nranks];
    const bool direct = weight_direct(a, DT);
    const uint32_t piece = direct ? stats_piece(V, a.tokens) : loss_piece(a.vocab, a.nranks, a.tokens, a.cols, DT, 0);
    Parts parts;
    StatsArgs q = {};
    q.part = reinterpret_cast<float2*>(a.workspace + parts.take(stats_entries(a.vocab, a.nranks) * a.tokens * sizeof(float2)));
    q.target = reinterpret_cast<float*>(a.workspace + parts.take(uint64_t(a.tokens) * 4));
    LossProblem p = problem_of(a);
    const PadParts pad = pad_parts(parts, a.tokens, a.cols, loss_piece(a.vocab, a.nranks, a.tokens, a.cols, DT, 0), DT);
    char* wpad = place_rows<T>(a, DT, pad, p, false, s);
    const Tile t = pick_tile(DT, piece, a.tokens, DT == kF32);
    for (int pass = 0; pass < 2; pass++) {  // count the tiles, then launch
        q.entry = 0;
        for (uint32_t first = 0; first < V; first += piece) {
            const uint32_t count = V - first < piece ? V - first : piece;
            Segments g = segments_of(a, DT, first, count, wpad, p.wpitch);
            set_tiles(g, kTileM[t], false);
            if (pass == 1) {
                if (!direct) pad_weight(a, first, count, wpad, p.wpitch, s);
                with_rows_of<DT, DT == kF32>(t, p.wpitch, [&](auto shape, auto tail) {
                    typedef decltype(shape) S;
                    constexpr bool TAIL = decltype(tail)::value;
                    q.token_tiles = ceil_div(a.tokens, S::BN);
                    hipLaunchKernelGGL((k_loss_stats<DT, S, TAIL>), dim3(g.tile[g.n] * q.token_tiles), dim3(S::threads), 0, s, p, g, q);
                });
            }
            q.entry += g.tile[g.n];
        }
        q.entries = q.entry;
    }
    LossOut o = {};
    for (int r = 0; r < a.nranks; r++) {
        o.loss[r] = a.loss[r];
        o.lse[r] = a.lse[r];
    }
    o.nranks = a.nranks;
    hipLaunchKernelGGL(k_loss_join, dim3(ceil_div(a.tokens, kThreads / 64)), dim3(kThreads), 0, s, p, q, o);
    return hipGetLastError();
}

// launch(parts of d).  TOKENS: the tile's n counts tokens, so the tiles of up to
// 64 of them only meet d in two parts.
template <int DT, typename S, bool TOKENS, typename F>
void with_parts(uint64_t tokens, F&& launch) {
    constexpr bool few = std::is_same<S, Tiny>::value || std::is_same<S, Narrow>::value;
    if constexpr (DT == kBF16) {
        if (d_parts(tokens, DT) == 2) return launch(std::integral_constant<int, 2>());
    }
    if constexpr (DT != kBF16 || !TOKENS || !few) launch(std::integral_constant<int, 1>());
}

// Few tiles of dhidden: the sum over the piece is cut among workgroups, each
// with at least 4 steps of it.
uint32_t splits_of(uint64_t tokens, uint64_t cols, uint64_t ldv, int dtype) {
    const uint64_t tiles = uint64_t(ceil_div(cols, 64)) * ceil_div(tokens, 64);
    if (tiles == 0 || tiles >= 512) return 1;
    uint64_t want = ceil_div(1024, tiles);
    const uint64_t most = ldv / step_elems(dtype) / 4;
    if (want > most) want = most;
    return want < 1 ? 1 : want > 32 ? 32 : uint32_t(want);
}
struct BackwardParts {
    uint64_t ldv, ldx, d, acc, scale;
    uint32_t splits;
    PadParts pad;
    uint64_t bytes;
};
BackwardParts backward_parts(int nranks, uint64_t tokens, uint64_t cols, uint64_t piece, int dtype) {
    BackwardParts b;
    // a piece may hold parts of all ranks, each padded to a whole step
    b.ldv = up(piece, step_elems(dtype)) + (nranks - 1) * step_elems(dtype);
    b.ldx = up(cols, 4);
    b.splits = splits_of(tokens, cols, b.ldv, dtype);
    Parts w;
    b.d = w.take(d_parts(tokens, dtype) * tokens * b.ldv * esize(dtype));
    b.acc = w.take(b.splits * tokens * b.ldx * 4);
    b.scale = w.take(kScaleParts * sizeof(float));
    b.pad = pad_parts(w, tokens, cols, piece, dtype);
    b.bytes = w.at;
    return b;
}

template <int DT>
hipError_t backward(const LossArgs& a, hipStream_t s) {
    typedef typename Elem<DT>::type T;
    const uint32_t V = a.vocab.start[a.nranks];
    const BackwardParts b = backward_parts(a.nranks, a.tokens, a.cols, a.piece, DT);
    LossProblem q = problem_of(a);
    char* wpad = place_rows<T>(a, DT, b.pad, q, true, s);
    LossProblem left = q;  // hidden without the tokens that are left out
    left.hidden = a.workspace + b.pad.hidden;
    DPiece p = {};
    if (hidden_direct(a, DT)) p.hidden = a.workspace + b.pad.hidden;
    p.d = a.workspace + b.d;
    p.acc = reinterpret_cast<float*>(a.workspace + b.acc);
    p.ldx = b.ldx;
    p.splits = b.splits;
    if (DT == kBF16 && a.tokens > kTwoPartTokens) {
        float* scale = reinterpret_cast<float*>(a.workspace + b.scale);
        hipLaunchKernelGGL(k_loss_scale, dim3(kScaleParts), dim3(kThreads), 0, s, q, scale);
        p.scale = scale;
    }
    for (uint32_t first = 0; first < V; first += a.piece) {
        const uint32_t count = V - first < a.piece ? V - first : a.piece;
        Segments g = segments_of(a, DT, first, count, wpad, q.wpitch);
        p.ldv = g.col[g.n];
        if (a.tokens > 0) {
            if (wpad != nullptr) pad_weight(a, first, count, wpad, q.wpitch, s);
            const Tile t = pick_tile(DT, count, a.tokens, true);
            set_tiles(g, kTileM[t], true);
            with_rows_of<DT, true>(t, q.wpitch, [&](auto shape, auto tail) {
                typedef decltype(shape) S;
                constexpr bool TAIL = decltype(tail)::value;
                p.nt = ceil_div(a.tokens, S::BN);
                with_parts<DT, S, true>(a.tokens, [&](auto parts) {
                    hipLaunchKernelGGL((k_loss_d<DT, S, TAIL, decltype(parts)::value>), dim3(g.tile[g.n] * p.nt), dim3(S::threads), 0, s, q, g, p);
                });
            });
            with_tile<DT, true>(pick_tile(DT, a.cols, a.tokens, true, p.splits), [&](auto shape) {
                typedef decltype(shape) S;
                p.mt = ceil_div(a.cols, S::BM);
                p.nt = ceil_div(a.tokens, S::BN);
                with_parts<DT, S, true>(a.tokens, [&](auto parts) {
                    hipLaunchKernelGGL((k_loss_dhidden<DT, S, decltype(parts)::value>), dim3(p.mt * p.nt, p.splits), dim3(S::threads), 0, s, q, g, p);
                });
            });
            p.add = 1;
            p.hidden = nullptr;
        }
        const Tile t = pick_tile(DT, a.cols, count, false);
        set_tiles(g, kTileN[t], false);
        with_tile<DT, false>(t, [&](auto shape) {
            typedef decltype(shape) S;
            p.mt = ceil_div(a.cols, S::BM);
            with_parts<DT, S, false>(a.tokens, [&](auto parts) {
                hipLaunchKernelGGL((k_loss_dweight<DT, S, decltype(parts)::value>), dim3(p.mt * g.tile[g.n]), dim3(S::threads), 0, s, left, g, p);
            });
        });
    }
    if (a.tokens > 0) {
        DHiddenOut o = {};
        o.quads = a.cols % 4 == 0;
        for (int r = 0; r < a.nranks; r++) {
            o.p[r] = a.dhidden[r];
            if (reinterpret_cast<uintptr_t>(o.p[r]) % (4 * sizeof(T)) != 0) o.quads = 0;
        }
        o.nranks = a.nranks;
        hipLaunchKernelGGL(k_loss_out<DT>, dim3(a.tokens, ceil_div(a.cols, kThreads * 4)), dim3(kThreads), 0, s, o, static_cast<const float*>(p.acc), a.tokens,
                           a.cols, p.ldx, p.splits);
    }
    return hipGetLastError();
}

}  // namespace

uint64_t loss_workspace(const RowTable& vocab, int nranks, uint64_t tokens, uint64_t cols, int dtype) {
    Parts w;
    w.take(stats_entries(vocab, nranks) * tokens * sizeof(float2));
    w.take(tokens * 4);
    pad_parts(w, tokens, cols, loss_piece(vocab, nranks, tokens, cols, dtype, 0), dtype);
    return w.at;
}

// A piece's weight rows are read three times and its d four times.  kLossPiece
// rows, or more where those rows and their d stay below 64 MiB, and so in the
// 256 MiB of cache in front of the memory: fewer launches (2 tokens x 129 fp32,
// 60174 rows: 191 us with four pieces, 131 with one).
uint32_t loss_piece(const RowTable& vocab, int nranks, uint64_t tokens, uint64_t cols, int dtype, uint64_t asked) {
    constexpr uint64_t cached = 64 << 20;
    uint64_t want = asked;
    if (want == 0) {
        want = cached / ((cols + d_parts(tokens, dtype) * tokens) * esize(dtype)) / 64 * 64;
        if (want < kLossPiece) want = kLossPiece;
    }
    const uint64_t all = vocab.start[nranks];
    if (want > kMaxLossPiece) want = kMaxLossPiece;
    return uint32_t(want < all ? want : all);
}

uint64_t loss_backward_workspace(int nranks, uint64_t tokens, uint64_t cols, uint32_t piece, int dtype) {
    return backward_parts(nranks, tokens, cols, piece, dtype).bytes;
}

hipError_t launch_loss(const LossArgs& a, int dtype, hipStream_t s) {
    return dtype == kBF16 ? forward<kBF16>(a, s) : forward<kF32>(a, s);
}
hipError_t launch_loss_backward(const LossArgs& a, int dtype, hipStream_t s) {
    return dtype == kBF16 ? backward<kBF16>(a, s) : backward<kF32>(a, s);
}

}  // namespace dt
