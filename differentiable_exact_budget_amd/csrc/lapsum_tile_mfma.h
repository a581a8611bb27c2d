// The main loop of the 16-bit matrix kernels (gfx950): a workgroup of four waves
// forms the sums of a BM x BN tile, each wave a quarter of it, from operands
// that go from memory straight to a ring of LDS buffers.  What is done with the
// sums is the callers'.
#pragma once
#include "lapsum_expert_tile.h"

namespace lapsum {

constexpr int kStepK = 64;  // k of one LDS unit: two matrix instructions deep
constexpr int kRing = 5;    // LDS units, each of one operand
constexpr int kProductThreads = 256;

// 16 bytes a lane from buffer offset `off` to LDS, lane l at `lds` + 16 l.
// Written as an instruction so that the compiler's counters do not wait for
// it at the next LDS read: step_barrier does, when the data is wanted.  It
// has no register output.
LS_DEV void load_to_lds(u32x4 rsrc, uint32_t off, uint32_t lds) {
    asm volatile(
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %0, %1, 0 offen lds"
        :
        : "v"(off), "s"(rsrc), "s"(lds));
}

// This wave's loads but the last LEFT have landed and its LDS reads are done;
// then the workgroup meets.
template <int LEFT>
LS_DEV void step_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LEFT) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// One operand of a tile: R rows (of its own index) by kStepK of k, a unit.
//   k contiguous: row i is a line of 128 bytes, a whole one of memory too (two
//     steps of 64 bytes, each with a buffer of its own, asked for the line twice:
//     the loss' forward tiles 1 to 2 % slower, 8-bit products 2 to 6 %), whose chunk c of 16 bytes lies at c ^ fold(i).
//     LDS serves 256 bytes of 16-byte reads at a time, of the lanes 0-3, 12-15,
//     20-23 and 24-27, then of 4-11, 16-19 and 28-31, and the same from 32
//     (measured, by pairs of lanes): the even rows of each sixteen reads meet
//     eight places, and the odd.
//   own index contiguous: two steps as StepLds lays them out.
template <int R, bool KFAST, bool PAIRED>
struct Operand {
    using Step = StepLds<R, KFAST, PAIRED>;
    static constexpr int kBytes = 2 * Step::kBytes;
    static constexpr int kLoads = kBytes / (kProductThreads * 16);  // a wave's loads of a unit
    static constexpr int kChunks = KFAST ? 8 : R / 8;               // chunks of a memory row

    const char* base;       // of the tile's first row and k
    uint32_t rows;          // rows of the tile that exist (KFAST), else its k
    uint32_t ld;            // bytes between rows of memory
    uint32_t last;          // not KFAST: bytes of the tile's last memory row that exist
    uint32_t voff[kLoads];  // this lane's offsets
    uint32_t kcol;          // KFAST: first k of this lane's chunk of load 0

    static LS_DEV int fold(int i) {
        if (!KFAST) return Step::fold(i);
        return PAIRED ? (i >> 1 & 1) | (i >> 3 & 3) << 1 : i >> 1 & 7;
    }
    // x: element (0, 0) of the tile; own: rows left of its own index; K:
    // length of the sum; ld_: elements between memory rows
    template <class T>
    LS_DEV void init(const T* x, int own, int K, int ld_) {
        base = reinterpret_cast<const char*>(x);
        ld = (uint32_t)ld_ * 2u;
        rows = (uint32_t)(KFAST ? min(R, own) : K);
        last = (uint32_t)min(R, own) * 2u;
        const int l = lane_id(), w = uniform(threadIdx.x >> 6);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int row = (w * kLoads + i) * (64 / kChunks) + l / kChunks, c = (l % kChunks) ^ fold(row);
            voff[i] = (uint32_t)row * ld + (uint32_t)c * 16;
            if (i == 0) kcol = c * 8;
        }
    }
    // the unit of k0 .. (empty past K: its loads write zeros)
    LS_DEV u32x4 window(int k0, int K) const {
        const char* p = base + (KFAST ? (size_t)k0 * 2 : (size_t)k0 * ld);
        uint32_t n = KFAST ? rows * ld - (uint32_t)k0 * 2
                           : (min((uint32_t)kStepK, rows - (uint32_t)k0) - 1u) * ld + last;
        if (k0 >= K) n = 0;
        return u32x4{(uint32_t)(uintptr_t)p, (uint32_t)((uintptr_t)p >> 32), n, 0x00020000u};
    }
    // issues load i of the window into the LDS unit at byte address `lds`
    LS_DEV void load(const u32x4& win, uint32_t lds, int i, int k0, int K) const {
        const int w = uniform(threadIdx.x >> 6);
        // the last unit of a sum: what follows in memory is the next row
        // (load i's rows differ from load 0's in these bits of their fold)
        const int k = k0 + (int)(kcol ^ (PAIRED ? (i & 3) * 16 : (i & 1) * 32));
        const uint32_t off = KFAST && k >= K ? 0x80000000u : voff[i];
        load_to_lds(win, off, lds + (w * kLoads + i) * 1024);
    }
    // fragment f, of the rows from r0, of step q of a unit
    static LS_DEV s16x8 frag(const char* lds, int r0, int f, int q) {
        if (!KFAST) return Step::frag(lds + q * Step::kBytes, r0, f);
        const int l = lane_id(), i = l & 15;
        const int row = r0 + (PAIRED ? (f >> 1) * 32 + (i >> 2) * 8 + (f & 1) * 4 + (i & 3) : f * 16 + i);
        return *(const s16x8*)(lds + row * 128 + ((q * 4 + (l >> 4)) ^ fold(row)) * 16);
    }
};

// acc = the sums over k < K of a(i, k) b(j, k) for this wave's quarter of a BM x
// BN tile.  a, b: element (0, 0) of the tile; kA, kB: k is the contiguous index;
// own_a, own_b: rows (columns) that there are from there; lda, ldb: elements
// between memory rows.  All addresses and strides are on 16 bytes.
template <class T, bool kA, bool kB, int BM, int BN>
struct TileSums {
    static_assert(BM == BN);  // the operands' units take each other's place
    using OpA = Operand<BM, kA, false>;
    using OpB = Operand<BN, kB, true>;
    static constexpr int FM = BM / 32, FN = BN / 32;  // fragments of a wave
    static constexpr int kUnit = OpA::kBytes;
    static constexpr int kLds = kRing * kUnit;

    f32x4 acc[FM][FN] = {};

    LS_DEV void run(const T* a, int own_a, int lda, const T* b, int own_b, int ldb, int K, char* lds) {
        if (K <= 0) return;
        const int w = uniform(threadIdx.x >> 6);
        const int r0 = (w >> 1) * (BM / 2), c0 = (w & 1) * (BN / 2);
        OpA oa;
        OpB ob;
        oa.init(a, own_a, K, lda);
        ob.init(b, own_b, K, ldb);
        const uint32_t at = (uint32_t)(uintptr_t)(LS_LDS(char)*)lds;
        auto fetch = [&](const auto& op, const u32x4& win, int k0, int to, int from, int end) {
#pragma unroll
            for (int i = from; i < end; ++i) op.load(win, at + to, i, k0, K);
        };
        // the units of the k that are multiplied, of the next, and a free one
        int ua = 0, ub = kUnit, na = 2 * kUnit, nb = 3 * kUnit, spare = 4 * kUnit;
        fetch(oa, oa.window(0, K), 0, ua, 0, OpA::kLoads);
        fetch(ob, ob.window(0, K), 0, ub, 0, OpB::kLoads);
        fetch(oa, oa.window(kStepK, K), kStepK, na, 0, OpA::kLoads);
        fetch(ob, ob.window(kStepK, K), kStepK, nb, 0, OpB::kLoads);
        s16x8 fa[2][FM], fb[2][FN];
        step_barrier<OpA::kLoads + OpB::kLoads>();
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[0][j] = OpB::frag(lds + ub, c0, j, 0);
#pragma unroll
        for (int i = 0; i < FM; ++i) fa[0][i] = OpA::frag(lds + ua, r0, i, 0);
        // Step q multiplies the fragments of set q and reads the next step's into
        // the other.  Step 0 fetches A of two units on into the free unit.  Step 1,
        // when all waves have read the present units, waits for the next ones and
        // fetches B of two units on to where A was; where B was is free then.
        auto step = [&](auto qv, int k0) {
            constexpr int q = decltype(qv)::value;
            if (q) step_barrier<OpA::kLoads>();
            const char *sa = lds + (q ? na : ua), *sb = lds + (q ? nb : ub);
            constexpr int kReads = FM + FN, kReadIn = FM / 2;
            const int kf = k0 + 2 * kStepK;
            const u32x4 win = q ? ob.window(kf, K) : oa.window(kf, K);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                if (i < kReadIn) {
#pragma unroll
                    for (int r = i * kReads / kReadIn; r < (i + 1) * kReads / kReadIn; ++r) {
                        if (r < FN) fb[q ^ 1][r] = OpB::frag(sb, c0, r, q ^ 1);
                        else fa[q ^ 1][r - FN] = OpA::frag(sa, r0, r - FN, q ^ 1);
                    }
                }
                if (q) fetch(ob, win, kf, ua, i * OpB::kLoads / FM, (i + 1) * OpB::kLoads / FM);
                else fetch(oa, win, kf, spare, i * OpA::kLoads / FM, (i + 1) * OpA::kLoads / FM);
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mfma16<T>(fb[q][j], fa[q][i], acc[i][j]);
                // keeps the compiler from gathering the loads
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        for (int k0 = 0; k0 < K; k0 += kStepK) {
            step(std::integral_constant<int, 0>{}, k0);
            step(std::integral_constant<int, 1>{}, k0);
            const int free = ub;
            ub = nb, nb = ua, ua = na, na = spare, spare = free;
        }
        // the last loads, past K, still write zeros to LDS
        step_barrier<0>();
    }
    // f(row, column, eight sums from there) for what this lane holds: lane l has
    // row l % 16 of a fragment and, of a pair of fragments, columns
    // 8 (l / 16) .. + 7
    template <class F>
    LS_DEV void each8(F&& f) const {
        const int l = lane_id(), w = uniform(threadIdx.x >> 6);
        const int r0 = (w >> 1) * (BM / 2), c0 = (w & 1) * (BN / 2);
#pragma unroll
        for (int j = 0; j < FN; j += 2)
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                float v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) v[r] = acc[i][j + (r >> 2)][r & 3];
                f(r0 + i * 16 + (l & 15), c0 + j * 16 + (l >> 4) * 8, v);
            }
    }
};

// Which tile a workgroup forms.  Workgroups are dealt out to the eight XCDs
// in turn; 32 at a time (one per CU) an XCD takes neighbouring tiles, which
// share operands in its L2, and the XCDs' 32 follow one another, so that
// together they walk one expert or two at a time and what one XCD fetches the
// others find in the memory-side cache.  Tiles past the last whole round of
// 256 are cut into quarters when that fills the CUs better: a quarter takes
// about a third of a tile's time, so up to 128 of them are worth it.
constexpr int kXcds = 8, kXcdTiles = 32, kRound = kXcds * kXcdTiles;
constexpr int kCutTiles = 128;
struct Turn {
    int tile;     // -1: none
    int quarter;  // 0 .. 3, or -1: the whole tile
};
LS_DEV Turn take_turn(int block, int n, bool cut) {
    const int full = n / kRound * kRound;
    const int x = block % kXcds, i = block / kXcds;
    if (block < full) return {(i / kXcdTiles * kXcds + x) * kXcdTiles + i % kXcdTiles, -1};
    const int rest = n - full, r = i - full / kXcds;
    cut = cut && rest <= kCutTiles;
    const int work = cut ? rest * 4 : rest, per = (work + kXcds - 1) / kXcds, t = x * per + r;
    if (r >= per || t >= work) return {-1, -1};
    return cut ? Turn{full + t / 4, t & 3} : Turn{full + t, -1};
}
inline long long turns(long long n, bool cut) { return ceil_div(n + (cut ? 3 * kCutTiles : 0), kXcds) * kXcds + kXcds; }

}  // namespace lapsum
