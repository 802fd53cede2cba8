// dt_matrix.h -- the matrix products of the model-step operators, a tile of
// `out` at a time: out[n][m] = sum_k A(m, k) B(n, k), where an operand lies in
// memory either with k contiguous (kRows) or with m or n contiguous (kCols).
// The second kind is turned on the way from LDS to the registers, so nothing is
// stored transposed.
#pragma once

#include "dt_step_device.h"

namespace dt {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
#define DT_LDS __attribute__((address_space(3)))

constexpr int kChunks = 4;             // 16-byte chunks of the summed index per step
constexpr int kStepBytes = kChunks * 16;
// fp32: a sum runs over so many steps of 16 terms at most, and these sums are added
// up apart, so that its error does not grow with every term of a long one.
constexpr uint32_t kRunSteps = 32;
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
// behind its end, the next row's first values, is masked in the registers: where
// the other operand has zeros there, an infinity times zero would still be NaN.
template <bool TAIL>
struct RowOperand {
    static constexpr bool tail = TAIL;
    const char* p;     // the tile's first row
    uint32_t rows, pitch, bytes, valid, skip;   // skip: bytes of a row before p
    __device__ __forceinline__ rsrc_t at(uint32_t step, bool any) const {
        return scalar_rsrc(p + step * kStepBytes, any && rows > 0 ? rows * pitch - skip - step * kStepBytes : 0);
    }
    __device__ __forceinline__ uint32_t left(uint32_t step) const { return bytes - step * kStepBytes; }
    __device__ __forceinline__ uint32_t group_at(uint32_t group) const { return group * 16 * pitch; }  // 16 rows of the tile
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
template <int DT, int MODE, int R, typename OP>
__device__ __forceinline__ uint32_t load_place(const OP& op, uint32_t group, uint32_t lane) {
    if constexpr (MODE == kRows) {
        // 16 rows of 64 bytes: lane l brings row l / 4
        const uint32_t row = lane >> 2;
        return op.group_at(group) + row * op.pitch + ((lane & 3) ^ row_turn(row)) * 16;
    } else {
        typedef ColTile<DT, R> C;
        constexpr uint32_t slots = C::row_bytes / 16, per_unit = C::unit_bytes / 16;
        const uint32_t k = group * C::per_load + lane / slots, slot = lane % slots;
        return k * op.pitch + ((slot / per_unit) ^ C::f(k)) * C::unit_bytes + slot % per_unit * 16;
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
__device__ __forceinline__ uint32_t fragment_place(uint32_t at, uint32_t lane) {
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

// Waits until at most `loads` of this wave's loads (63: any number) and `reads`
// of its LDS reads (15: as many as the counter holds) are outstanding.
template <int loads, int reads>
__device__ __forceinline__ void wait() {
    static_assert(loads < 64 && reads < 16, "the counters hold 6 and 4 bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((loads & 15) | (loads >> 4) << 14 | 7 << 4 | reads << 8);
    asm volatile("" ::: "memory");
}

// The same, and then waits for the workgroup's other waves.
template <int loads, int reads>
__device__ __forceinline__ void arrive() {
    wait<loads, reads>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A wave's 16 x 16 part of the product of two fragments.
template <int DT>
__device__ __forceinline__ f32x4 multiply(const u32x4& a, const u32x4& b, f32x4 acc) {
    if constexpr (DT == kBF16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), acc, 0, 0, 0);
        return acc;
    }
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
    const uint32_t lane = threadIdx.x & 63;
    // the wave's shares of A's and B's groups of 1 KiB
    uint32_t pa[S::loads_a], pb[S::loads_b];
#pragma unroll
    for (int i = 0; i < S::loads_a; i++) pa[i] = load_place<DT, MA, S::BM>(A, wave * S::loads_a + i, lane);
#pragma unroll
    for (int i = 0; i < S::loads_b; i++) pb[i] = load_place<DT, MB, S::BN>(B, wave * S::loads_b + i, lane);
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
    uint32_t ra = fragment_place<DT, MA, S::BM>(wm, lane), rb = fragment_place<DT, MB, S::BN>(wn, lane);
#pragma unroll
    for (int i = 0; i < S::MI; i++) fa[i] = A.cut(fragment<DT, MA, S::BM>(s0, ra, i), lo);
#pragma unroll
    for (int j = 0; j < S::NI; j++) fb[0][j] = B.cut(fragment<DT, MB, S::BN>(s0 + S::BM * kChunks, rb, j), lo);
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
        for (int j = 0; j < S::NI; j++) next[j] = B.cut(fragment<DT, MB, S::BN>(following + S::BM * kChunks, rb, j), step + 1);
#pragma unroll
        for (int i = 0; i < S::MI; i++) {
#pragma unroll
            for (int j = 0; j < S::NI; j++) acc[i][j] = multiply<DT>(fa[i], now[j], acc[i][j]);
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

// The lane, without what the compiler knows of it: a loop over tiles would
// otherwise hold each address that it gives in a register through the products.
__device__ __forceinline__ uint32_t fresh_lane() {
    uint32_t lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    return lane;
}

// The tiles of a workgroup one after the other, as matrix_tile multiplies them, with
// the loads running on from tile to tile: the next tile's first three steps are on
// their way while the last ones of a tile are multiplied and while its sums leave
// the registers.
//   next(t)               the workgroup's next tile; false: there is none
//   operands(t, A, B)     sets its operands and returns its steps of the summed
//                         index; a row's pitch is the same in all tiles
//   rows(t)               its rows of B that are there: waves with none of them leave
//                         the matrix units to the others
//   done(t, acc, room)    what becomes of its sums, acc as matrix_tile leaves it; room:
//                         LDS of the wave's own
// A tile takes whole rounds of four steps, one at least, so the loads are never
// more than one tile ahead.
template <int DT, typename S, int MA, int MB, typename OA, typename OB, typename Tile, typename Next, typename Operands, typename Rows, typename Done>
__device__ __forceinline__ void matrix_walk(Next&& next, Operands&& operands, Rows&& rows, Done&& done) {
    __shared__ u32x4 s0[S::stage], s1[S::stage], s2[S::stage], s3[S::stage];
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Tile now, ahead;     // multiplied, loaded
    if (!next(ahead)) return;
    OA A, now_a;         // loaded; a row's end in the tile that is multiplied
    OB B, now_b;
    auto rounds = [](uint32_t n) { return n == 0 ? 4 : (n + 3) / 4 * 4; };
    uint32_t steps = operands(ahead, A, B), end = rounds(steps), step = 0;   // of the loads
    bool more = true;
    const uint32_t wm = (wave % S::GM) * S::WM, wn = (wave / S::GM) * S::WN, lane = fresh_lane();
    uint32_t pa[S::loads_a], pb[S::loads_b];
#pragma unroll
    for (int i = 0; i < S::loads_a; i++) pa[i] = load_place<DT, MA, S::BM>(A, wave * S::loads_a + i, lane);
#pragma unroll
    for (int i = 0; i < S::loads_b; i++) pb[i] = load_place<DT, MB, S::BN>(B, wave * S::loads_b + i, lane);
    auto load = [&](u32x4* to) {
        load_step<MA>(A, step, step < steps, pa, to + wave * S::loads_a * 64);
        load_step<MB>(B, step, step < steps, pb, to + S::BM * kChunks + wave * S::loads_b * 64);
        step++;
    };
    load(s0);
    load(s1);
    load(s2);
    arrive<2 * S::loads, 15>();
    u32x4 fa[S::MI], fb[2][S::NI];
    uint32_t ra = fragment_place<DT, MA, S::BM>(wm, lane), rb = fragment_place<DT, MB, S::BN>(wn, lane);
#pragma unroll
    for (int i = 0; i < S::MI; i++) fa[i] = A.cut(fragment<DT, MA, S::BM>(s0, ra, i), 0);
#pragma unroll
    for (int j = 0; j < S::NI; j++) fb[0][j] = B.cut(fragment<DT, MB, S::BN>(s0 + S::BM * kChunks, rb, j), 0);
    f32x4 acc[S::MI][S::NI];
    constexpr bool RUNS = DT == kF32;
    f32x4 total[RUNS ? S::MI : 1][RUNS ? S::NI : 1];
    // One step, as in matrix_tile.  settled: the bytes of the following step have
    // been waited for already, behind the tile before, and its stores need not be.
    constexpr int turn_reads = S::MI * (MA == kRows ? 1 : 2) + S::NI * (MB == kRows ? 1 : 2);
    bool active = wn < rows(ahead);   // the wave has rows in the tile that is multiplied
    auto turn = [&](uint32_t following_step, bool settled, u32x4* free, const u32x4* following, const u32x4 (&fn)[S::NI], u32x4 (&fnext)[S::NI]) {
        if (!settled) wait<S::loads, 15>();
        arrive<63, turn_reads < 15 ? turn_reads : 15>();
        load(free);
        // keeps the compiler from holding every fragment's address of every stage in a register
        asm volatile("" : "+v"(ra), "+v"(rb));
        wait<63, 0>();   // the last turn's reads, in waves without rows as well: their stage is loaded again in the next turn
        if (!active && following_step != 0) return;
        // the loads may be in the next tile already, whose rows may end elsewhere
        const OA& end_a = following_step == 0 ? A : now_a;
        const OB& end_b = following_step == 0 ? B : now_b;
#pragma unroll
        for (int j = 0; j < S::NI; j++) fnext[j] = end_b.cut(fragment<DT, MB, S::BN>(following + S::BM * kChunks, rb, j), following_step);
#pragma unroll
        for (int i = 0; i < S::MI; i++) {
#pragma unroll
            for (int j = 0; j < S::NI; j++) acc[i][j] = multiply<DT>(fa[i], fn[j], acc[i][j]);
            fa[i] = end_a.cut(fragment<DT, MA, S::BM>(following, ra, i), following_step);
        }
    };
    bool settled = false;
    while (true) {
        now = ahead;
        now_a = A;
        now_b = B;
        const uint32_t last = end;
#pragma unroll
        for (int i = 0; i < S::MI; i++)
#pragma unroll
            for (int j = 0; j < S::NI; j++) {
                acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
                if constexpr (RUNS) total[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
        for (uint32_t k = 0; k < last; k += 4) {
            if constexpr (RUNS) {
                if (k % kRunSteps == 0) {
#pragma unroll
                    for (int i = 0; i < S::MI; i++)
#pragma unroll
                        for (int j = 0; j < S::NI; j++) {
                            total[i][j] += acc[i][j];
                            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
                        }
                }
            }
            turn(k + 1, settled, s3, s1, fb[0], fb[1]);
            if (step == end) {   // three steps of this tile are left to be multiplied
                more = next(ahead);
                steps = more ? operands(ahead, A, B) : 0;
                end = rounds(steps);
                step = 0;
            }
            turn(k + 2, settled, s0, s2, fb[1], fb[0]);
            settled = false;
            turn(k + 3, false, s1, s3, fb[0], fb[1]);
            turn(k + 4 == last ? 0 : k + 4, false, s2, s0, fb[1], fb[0]);
        }
        // The loads that are on their way arrive before the stores go out, so that nothing waits for those; and s3,
        // loaded again behind the next barrier, is read no more.
        arrive<0, 0>();
        constexpr uint32_t room = S::stage / S::waves;
        static_assert(room * 16 >= 16 * S::WM * (DT == kBF16 ? 2 : 4) && room * 16 >= 16 * (S::WM < 64 ? S::WM : 64) * 4,
                      "the wave's room holds 16 rows of its features in the type, or of up to 64 of them in fp32");
        if constexpr (RUNS) {
#pragma unroll
            for (int i = 0; i < S::MI; i++)
#pragma unroll
                for (int j = 0; j < S::NI; j++) acc[i][j] += total[i][j];
        }
        if (active) done(now, acc, s3 + wave * room);
        if (!more) break;
        settled = true;
        active = wn < rows(ahead);
    }
    arrive<0, 0>();  // nothing is on its way into LDS when the workgroup ends
}

// 16 rows of W features, row lane % 16 in the lane's quads v[q] (features 16 q + 4
// (lane / 16) on), rounded to the type and turned through the wave's room in LDS:
// emit(row, feature, 16 bytes of them), so that stores are of whole lines where
// quads would touch 16 rows each.
template <int DT, int W, typename Emit>
__device__ __forceinline__ void turn_rows(u32x4* room, const f32x4 (&v)[W / 16], Emit&& emit) {
    constexpr uint32_t es = DT == kBF16 ? 2 : 4, per_row = W * es / 16, all = 16 * per_row;
    const uint32_t lane = fresh_lane(), n = lane & 15;
#pragma unroll
    for (int q = 0; q < W / 16; q++) {
        const uint32_t byte = (16 * q + (lane >> 4) * 4) * es, at = (n * per_row + ((byte / 16) ^ (n % per_row))) * 16 + byte % 16;
        store_quad<DT>(reinterpret_cast<typename Elem<DT>::type*>(reinterpret_cast<char*>(room) + at), v[q], true);
    }
#pragma unroll
    for (uint32_t k = 0; k < (all + 63) / 64; k++) {
        const uint32_t i = k * 64 + lane, row = i / per_row, vec = i % per_row;
        if (all % 64 != 0 && i >= all) continue;
        emit(row, vec * (16 / es), room[row * per_row + (vec ^ (row % per_row))]);
    }
}

// 16 bytes at byte `at` of a row of `bytes` bytes that starts and ends at any
// element: zeros behind the row's end, where nothing is read.
template <int ES>
__device__ __forceinline__ u32x4 read_loose(const char* row, uint32_t at, uint32_t bytes) {
    u32x4 x = {0, 0, 0, 0};
    if (at + 16 <= bytes) {
        x = *reinterpret_cast<const typename Loose<ES>::type*>(row + at);
    } else if (at < bytes) {
        typedef typename std::conditional<ES == 2, uint16_t, uint32_t>::type T;
        T t[16 / ES];
#pragma unroll
        for (int e = 0; e < 16 / ES; e++) t[e] = at + e * ES < bytes ? *reinterpret_cast<const T*>(row + at + e * ES) : T(0);
        __builtin_memcpy(&x, t, 16);
    }
    return x;
}

// Which of `total` tiles workgroup `id` takes: ids go round the 8 XCDs, and each XCD
// gets a run of neighbouring tiles.
__device__ __forceinline__ uint32_t share_of(uint32_t id, uint32_t total) {
    const uint32_t q = total / 8, rem = total % 8, x = id % 8;
    return x * q + (x < rem ? x : rem) + id / 8;
}
// Tile t of mt x nt, walked in bands of 8 rows of tiles.
__device__ __forceinline__ void band_tile(uint32_t t, uint32_t mt, uint32_t nt, uint32_t& m, uint32_t& n) {
    const uint32_t band = t / (8 * nt), first = band * 8, in = t - band * 8 * nt;
    const uint32_t high = mt - first < 8 ? mt - first : 8;
    // divisions run on the vector unit: back into scalar registers, where the buffer resources are built
    m = __builtin_amdgcn_readfirstlane(first + in % high);
    n = __builtin_amdgcn_readfirstlane(in / high);
}
// Tile `id` of mt x nt in an order that keeps an XCD's workgroups on neighbouring tiles.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t mt, uint32_t nt, uint32_t& m, uint32_t& n) {
    band_tile(share_of(id, mt * nt), mt, nt, m, n);
}

}  // namespace
}  // namespace dt
