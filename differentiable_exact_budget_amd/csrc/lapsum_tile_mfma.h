// The main loop of the 16-bit matrix kernels (gfx950): a workgroup of four waves
// forms the sums of a BM x BN tile, each wave a quarter of it, from operands
// that go from memory straight to a ring of LDS buffers.  What is done with the
// sums is the callers'.
#pragma once
#include "lapsum_expert_tile.h"

namespace lapsum {

constexpr int kStepK = 32;  // k of one LDS buffer
constexpr int kRing = 5;    // LDS buffers
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

// One operand of a tile: R rows (of its own index) by kStepK of k.
template <int R, bool KFAST, bool PAIRED>
struct Operand : StepLds<R, KFAST, PAIRED> {
    using Lds = StepLds<R, KFAST, PAIRED>;
    using Lds::fold;
    using Lds::kBytes;
    static constexpr int kLoads = kBytes / (kProductThreads * 16);  // a wave's loads per step
    static constexpr int kChunks = R / 8;                           // chunks of a k row (not KFAST)

    const char* base;       // of the tile's first row and k
    uint32_t rows;          // rows of the tile that exist (KFAST), else its k
    uint32_t ld;            // bytes between rows of memory
    uint32_t last;          // not KFAST: bytes of the tile's last memory row that exist
    uint32_t kcol;          // KFAST: first k of this lane's chunk
    uint32_t voff[kLoads];  // this lane's offsets

    // x: element (0, 0) of the tile; own: rows left of its own index; K:
    // length of the sum; ld_: elements between memory rows
    template <class T>
    LS_DEV void init(const T* x, int own, int K, int ld_) {
        base = reinterpret_cast<const char*>(x);
        ld = (uint32_t)ld_ * 2u;
        const int l = lane_id(), w = uniform(threadIdx.x >> 6);
        if (KFAST) {
            rows = (uint32_t)min(R, own);
            const int u = (l & 7) ^ fold(l >> 3), c = u & 3;
            kcol = c * 8;
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                voff[i] = (uint32_t)((w * kLoads + i) * 16 + (l >> 3) * 2 + (u >> 2)) * ld + c * 16;
        } else {
            rows = (uint32_t)K;
            last = (uint32_t)min(R, own) * 2u;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int k = (w * kLoads + i) * (64 / kChunks) + l / kChunks;
                voff[i] = (uint32_t)k * ld + (uint32_t)((l % kChunks) ^ fold(k)) * 16;
            }
        }
    }
    // the buffer of k0 .. k0 + 31 (empty past K: its loads write zeros)
    LS_DEV u32x4 window(int k0, int K) const {
        const char* p = base + (KFAST ? (size_t)k0 * 2 : (size_t)k0 * ld);
        uint32_t n = KFAST ? rows * ld - (uint32_t)k0 * 2
                           : (min((uint32_t)kStepK, rows - (uint32_t)k0) - 1u) * ld + last;
        if (k0 >= K) n = 0;
        return u32x4{(uint32_t)(uintptr_t)p, (uint32_t)((uintptr_t)p >> 32), n, 0x00020000u};
    }
    // issues load i of the window into the LDS buffer at byte address `lds`
    LS_DEV void load(const u32x4& win, uint32_t lds, int i, int k0, int K) const {
        const int w = uniform(threadIdx.x >> 6);
        // the last step of a sum: what follows in memory is the next row
        const uint32_t off = KFAST && k0 + (int)kcol >= K ? 0x80000000u : voff[i];
        load_to_lds(win, off, lds + (w * kLoads + i) * 1024);
    }
};

// acc = the sums over k < K of a(i, k) b(j, k) for this wave's quarter of a BM x
// BN tile.  a, b: element (0, 0) of the tile; kA, kB: k is the contiguous index;
// own_a, own_b: rows (columns) that there are from there; lda, ldb: elements
// between memory rows.  All addresses and strides are on 16 bytes.
template <class T, bool kA, bool kB, int BM, int BN>
struct TileSums {
    using OpA = Operand<BM, kA, false>;
    using OpB = Operand<BN, kB, true>;
    static constexpr int FM = BM / 32, FN = BN / 32;  // fragments of a wave
    static constexpr int kBuffer = OpA::kBytes + OpB::kBytes;
    static constexpr int kLds = kRing * kBuffer;

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
        // steps s and s + 1 of one operand, interleaved, loads [from, to)
        auto fetch = [&](const auto& op, const u32x4 (&win)[2], int k0, uint32_t to0, uint32_t to1, int from, int to) {
#pragma unroll
            for (int r = from; r < to; ++r) {
                if (r & 1) op.load(win[1], to1, r >> 1, k0 + kStepK, K);
                else op.load(win[0], to0, r >> 1, k0, K);
            }
        };
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
            const int k0 = q * kStepK;
            const u32x4 wa[2] = {oa.window(k0, K), oa.window(k0 + kStepK, K)};
            const u32x4 wb[2] = {ob.window(k0, K), ob.window(k0 + kStepK, K)};
            const uint32_t to = at + q * kBuffer;
            fetch(oa, wa, k0, to, to + kBuffer, 0, 2 * OpA::kLoads);
            fetch(ob, wb, k0, to + OpA::kBytes, to + OpA::kBytes + kBuffer, 0, 2 * OpB::kLoads);
        }
        s16x8 fa[2][FM], fb[2][FN];
        step_barrier<2 * (OpA::kLoads + OpB::kLoads)>();
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[0][j] = OpB::frag(lds + OpA::kBytes, c0, j);
#pragma unroll
        for (int i = 0; i < FM; ++i) fa[0][i] = OpA::frag(lds, r0, i);
        // the buffers of steps s - 2, s - 1, s and s + 1
        int prev2 = 0, prev = 4 * kBuffer, cur = 0, next = kBuffer;
        // Step s multiplies the fragments of set s % 2 and reads step s + 1
        // into the other.  An even step fetches A for s + 4 and s + 5, an odd
        // one B for s + 3 and s + 4, into the two buffers whose fragments are
        // all read.  An odd step waits for everything before the even step's
        // loads: the buffers that it and the following step read.
        auto step = [&](auto qv, int k0) {
            constexpr int q = decltype(qv)::value;
            step_barrier<q == 0 ? 63 : 2 * OpA::kLoads>();
            const char *sa = lds + next, *sb = sa + OpA::kBytes;
            constexpr int kReads = FM + FN, kReadIn = FM / 2;
            const int kf = k0 + (q == 0 ? 4 : 3) * kStepK;
            u32x4 win[2];
            if (q == 0) win[0] = oa.window(kf, K), win[1] = oa.window(kf + kStepK, K);
            else win[0] = ob.window(kf, K), win[1] = ob.window(kf + kStepK, K);
            const uint32_t to0 = at + (q == 0 ? prev : prev2 + OpA::kBytes);
            const uint32_t to1 = at + (q == 0 ? cur : prev + OpA::kBytes);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                if (i < kReadIn) {
#pragma unroll
                    for (int r = i * kReads / kReadIn; r < (i + 1) * kReads / kReadIn; ++r) {
                        if (r < FN) fb[q ^ 1][r] = OpB::frag(sb, c0, r);
                        else fa[q ^ 1][r - FN] = OpA::frag(sa, r0, r - FN);
                    }
                }
                if (q == 0) fetch(oa, win, kf, to0, to1, i * 2 * OpA::kLoads / FM, (i + 1) * 2 * OpA::kLoads / FM);
                else fetch(ob, win, kf, to0, to1, i * 2 * OpB::kLoads / FM, (i + 1) * 2 * OpB::kLoads / FM);
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mfma16<T>(fb[q][j], fa[q][i], acc[i][j]);
                // keeps the compiler from gathering the loads
                __builtin_amdgcn_sched_barrier(0);
            }
            prev2 = prev;
            prev = cur;
            cur = next;
            next = next == (kRing - 1) * kBuffer ? 0 : next + kBuffer;
        };
        for (int k0 = 0; k0 < K; k0 += 2 * kStepK) {
            step(std::integral_constant<int, 0>{}, k0);
            step(std::integral_constant<int, 1>{}, k0 + kStepK);
        }
        // the last steps' loads, past K, still write zeros to LDS
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
