// The experts' products on 16-bit rows whose widths are multiples of 8: tiles
// in LDS, 16-bit matrix instructions, fp32 sums.
//
// Mathematics: C(i, j) = sum over k of A(i, k) B(j, k), i over one expert's
// rows (or, for the weight gradient, its outputs), j over columns.  Each of A
// and B is stored with either k or its own index contiguous:
//   y  = act(xs W^T + b)   A = xs  (k contiguous)   B = W   (k contiguous)
//   dx = dz W              A = dz  (k contiguous)   B = W^T (j contiguous)
//   dW = dz^T xs           A = dz^T (i contiguous)  B = xs^T (j contiguous)
//
// A workgroup of four waves forms a BM x BN tile of C, each wave a quarter of
// it: with 256 x 256 a wave holds 128 x 128 fp32 sums in 256 registers, the
// most there is, so a byte that is brought to LDS is used as often as it can
// be.  The sum runs in steps of 32 k, one matrix instruction deep.
//  - Operands go from memory to LDS without passing through registers
//    (buffer_load ... lds, 16 bytes a lane) into a ring of five buffers.  Two
//    steps are fetched as one, alternately all of A and all of B, so that the
//    two halves of a 128-byte line are asked for together, and the loads are
//    spread evenly between the matrix instructions: a wave that issues many
//    at once stands still until the memory pipeline has taken them.
//  - While a step's fragments are multiplied, the next step's are read from
//    LDS into a second set of registers.
//  - Reads out of range return zero, which is all the masking that ragged
//    experts need: a tile's buffer ends with its expert's last row.
//
// 32768 rows, 8 experts 2048 -> 4096 in bf16 (0.55 TFLOP): y 0.50 ms, 1.1
// PFLOP/s; dx 0.47, dW 0.44.  What bounds it is the feed: the loads to LDS
// alone, without a product, take 0.41 / 0.38 / 0.37 ms; the matrix instructions
// alone would take 0.36.  By the counters the matrix pipes work 44 / 54 / 51 %
// of the time (y with silu, dx, dW) and 32 / 25 / 21 % of the requests miss the
// L2.  A tile's first loads and its epilogue stand alone, no products beside
// them: an activation adds what its instructions take (silu 16 us to y's 500,
// gelu 46), and short sums feel it most: 16384 rows, 16 experts 1024 -> 4096 in
// f16 (0.14 TFLOP, 96 us at a large product's rate) take 160 us without one,
// 169 with silu, 189 with gelu.
//
// A wave's direct-to-LDS store is 64 consecutive chunks of the step's layout
// in LDS, so the layout's permutation is made on the global side: each lane
// fetches the chunk that belongs at its place.  B's fragments come in pairs
// that share 32 columns, so a lane ends with 8 consecutive columns of a row of
// C, one 16-byte store.
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

// BM x BN of a piece, from its row i0 and column j0
template <class T, int FORM, int ACT, int BM, int BN>
LS_DEV void form_tile(const Piece<T>& p, int i0, int j0, char* lds) {
    constexpr bool kA = FORM != kFormDw, kB = FORM == kFormY;  // k contiguous?
    using OpA = Operand<BM, kA, false>;
    using OpB = Operand<BN, kB, true>;
    using Z = typename ZKeep<T>::type;
    constexpr int FM = BM / 32, FN = BN / 32;  // fragments of a wave
    constexpr int kBuffer = OpA::kBytes + OpB::kBytes;
    const int l = lane_id(), w = uniform(threadIdx.x >> 6);
    const int r0 = (w >> 1) * (BM / 2), c0 = (w & 1) * (BN / 2);
    const int M = p.M - i0, N = p.N - j0, K = p.K;

    f32x4 acc[FM][FN] = {};
    if (K > 0) {
        OpA oa;
        OpB ob;
        oa.init(p.a + (kA ? (long long)i0 * p.lda : i0), M, K, p.lda);
        ob.init(p.b + (kB ? (long long)j0 * p.ldb : j0), N, K, p.ldb);
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
    // lane l holds row l % 16 of a fragment and, of a pair of fragments,
    // columns 8 (l / 16) .. + 7
    struct __attribute__((aligned(16))) T8 { T v[8]; };
    struct __attribute__((aligned(16))) Z8 { Z v[8]; };
#pragma unroll
    for (int j = 0; j < FN; j += 2) {
        const int col = c0 + j * 16 + (l >> 4) * 8;
        if (col >= N) continue;
        float bj[8] = {};
        if (FORM == kFormY && p.bias) {
            const T8 v = *(const T8*)(p.bias + j0 + col);
#pragma unroll
            for (int r = 0; r < 8; ++r) bj[r] = to_f(v.v[r]);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int row = r0 + i * 16 + (l & 15);
            if (row >= M) continue;
            const long long to = (long long)(i0 + row) * p.ldc + j0 + col;
            T8 o;
            Z8 k;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const float v = acc[i][j + (r >> 2)][r & 3] + bj[r];
                if (FORM == kFormY && ACT != kActNone) k.v[r] = ZKeep<T>::template make<ACT>(v);
                o.v[r] = from_f<T>(act_of<ACT, T>(v));
            }
            *(T8*)(p.c + to) = o;
            if (FORM == kFormY && ACT != kActNone && p.z)  // not read before the backward pass
                __builtin_nontemporal_store(__builtin_bit_cast(u32x4, k), (u32x4*)(p.z + to));
        }
    }
}

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

template <class T, int FORM, int ACT, int BM, int BN>
__global__ __launch_bounds__(kProductThreads) void k_product(LinearArgs g) {
    constexpr int kGroup = 4;  // row tiles that walk the columns together: 4 x 8 tiles on an XCD at a time
    constexpr bool kCut = BM == 256;
    __shared__ __align__(1024) char lds[kRing * (BM + BN) * kStepK * 2];
    const int cols = ((FORM == kFormY ? g.out : g.in) + BN - 1) / BN;
    Place<T> at;
    int quarter;
    if constexpr (FORM == kFormDw) {
        const Turn t = take_turn(blockIdx.x, (g.out + BM - 1) / BM * g.E * cols, kCut);
        if (t.tile < 0) return;
        at = dw_place<T, BM>(g, t.tile, cols);
        quarter = t.quarter;
    } else {
        RowTiles<BM> rows(g.off, g.E, g.P);
        const Turn t = take_turn(blockIdx.x, rows.count() * cols, kCut);
        if (t.tile < 0) return;
        at = row_place<T, FORM, BM>(g, rows, t.tile, cols);
        quarter = t.quarter;
    }
    const int first = at.q / (kGroup * cols) * kGroup, n = min(kGroup, at.rows - first);
    const int in = at.q - first * cols;
    int i0 = (first + in % n) * BM, j0 = in / n * BN;
    if constexpr (kCut) {
        if (quarter >= 0) {
            i0 += (quarter >> 1) * (BM / 2);
            j0 += (quarter & 1) * (BN / 2);
            if (i0 < at.p.M && j0 < at.p.N) form_tile<T, FORM, ACT, BM / 2, BN / 2>(at.p, i0, j0, lds);
            return;
        }
    }
    form_tile<T, FORM, ACT, BM, BN>(at.p, i0, j0, lds);
}

template <class T, int B>
static void launch_tiles(int form, const LinearArgs& g, hipStream_t st) {
    const int N = form == kFormY ? g.out : g.in;
    const long long cols = ceil_div(N, B);
    const long long tiles = cols * (form == kFormDw ? ceil_div(g.out, B) * g.E : max_row_tiles<B>(g.P, g.E));
    const dim3 grid((unsigned)turns(tiles, B == 256)), block(kProductThreads);
    if (form == kFormDw)
        hipLaunchKernelGGL((k_product<T, kFormDw, kActNone, B, B>), grid, block, 0, st, g);
    else if (form == kFormDx)
        hipLaunchKernelGGL((k_product<T, kFormDx, kActNone, B, B>), grid, block, 0, st, g);
    else
        with_act(g.act, [&](auto av) {
            hipLaunchKernelGGL((k_product<T, kFormY, decltype(av)::value, B, B>), grid, block, 0, st, g);
        });
}

bool expert_mfma_takes(int form, int dtype, const LinearArgs& g) {
    if (dtype == kF32 || g.in % 8 || g.out % 8 || g.in > (1 << 20) || g.out > (1 << 20)) return false;
    if (!aligned16(g.a) || !aligned16(g.b) || !aligned16(g.c) || !aligned16(g.bias) || !aligned16(g.z)) return false;
    // one tile a workgroup, whatever its side
    const long long tiles = form == kFormDw ? ceil_div(g.out, 64) * ceil_div(g.in, 64) * g.E
                                            : ceil_div(form == kFormY ? g.out : g.in, 64) *
                                                  max_row_tiles<64>(g.P, g.E);
    return tiles < kGridMax;
}

// The tile's side, by what was measured (bf16, 64 / 128 / 256, us; R: rows of
// an expert on average; tiles: of 256, the row forms' taken as half filled at
// each expert's end):
//   y, 64 experts 2048 -> 1024, R = 1:      30 / 32 / 48    (few rows: more
//                               R = 16:     45 / 46 / 53    workgroups stream
//                               R = 64:     85 / 64 / 68    the weights)
//   y, 8 experts 2048 -> 2048, 160 tiles:   69 / 55 / 58
//                              288 tiles:  124 / 84 / 81
//   y, 64 experts 512 -> 1024, 384 tiles:   47 / 37 / 49    (a short sum)
//   dx, 8 experts 2048 -> 1024, 32 tiles:   20 / 23 / 29
//   dW, 8 experts, 512 x 512, 32 tiles:     17 / 21 / 21
//       8 experts, 2048 x 1024, 256 tiles:  21 / 19 / 18
//       64 experts, 1024 x 2048, R = 1:     79 / 65 / 73
// R takes the experts without rows in, so rows that are all one expert's among
// many get too small a tile: 4096 rows 1024 -> 128, y 58 us as one of 1024
// experts and 8 as the only one.  And dW's sum is never split over workgroups:
// 65536 rows of 4 experts 64 -> 64 take 83 us on 4 of them, their bytes 3.
static int tile_side(int form, const LinearArgs& g) {
    const long long per = g.P / g.E;
    if (form == kFormDw) {
        if (per > 16 && ceil_div(g.out, 256) * ceil_div(g.in, 256) * g.E >= 256) return 256;
        return ceil_div(g.out, 128) * ceil_div(g.in, 128) * g.E >= 256 ? 128 : 64;
    }
    const int N = form == kFormY ? g.out : g.in, K = form == kFormY ? g.in : g.out;
    if (per >= 96 && K >= 1024 && (g.P / 256 + g.E / 2) * ceil_div(N, 256) >= 256) return 256;
    return per > 32 && (g.P / 128 + g.E / 2) * ceil_div(N, 128) >= 128 ? 128 : 64;
}

void launch_expert_mfma(int form, int dtype, const LinearArgs& g, hipStream_t st) {
    // Few rows for each expert, or few at all: without LDS.  64-wide tiles / few,
    // us, weights in the memory-side cache and from memory: 64 experts
    // 2048 -> 1024, 1 row of an expert 27 / 29 and 44 / 33, 2 rows 35 / 36 and
    // 57 / 42, 4 rows 38 / 43 and 64 / 51, 8 rows 40 / 51 and 65 / 62; 8 experts
    // 2048 -> 4096, 2 rows 20 / 18 and 31 / 21; 64 experts 512 -> 1024, 4 rows
    // 13 / 15 and 15 / 18; 16 experts 512 -> 512, 4 rows 5.7 / 4.1 and 6.8 / 4.4.
    const bool few = (g.in >= 1024 && g.P <= 4 * g.E) || g.P * ceil_div(g.out, 64) < 1024;
    if (form == kFormY && few && expert_few_takes(g)) {
        launch_expert_few(dtype, g, st);
        return;
    }
    const int side = tile_side(form, g);
    with_dtype(dtype, [&](auto tv) {
        using T = decltype(tv);
        if constexpr (sizeof(T) == 2) {
            if (side == 256) launch_tiles<T, 256>(form, g, st);
            else if (side == 128) launch_tiles<T, 128>(form, g, st);
            else launch_tiles<T, 64>(form, g, st);
        }
    });
}

}  // namespace lapsum
