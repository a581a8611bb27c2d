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
// be.  The main loop (lapsum_tile_mfma.h) takes 64 of k of one operand as a unit,
// two steps of one matrix instruction each.
//  - Operands go from memory to LDS without passing through registers
//    (buffer_load ... lds, 16 bytes a lane) into a ring of five units: those of A
//    and B that are multiplied, the next ones, and a free one.  A step fetches one
//    operand's unit, whole 128-byte lines of it where k is contiguous, and the
//    loads are spread evenly between the matrix instructions: a wave that issues
//    many at once stands still until the memory pipeline has taken them.
//  - While a step's fragments are multiplied, the next step's are read from
//    LDS into a second set of registers.  The waves meet once in two steps.
//  - Reads out of range return zero, which is all the masking that ragged
//    experts need: a tile's buffer ends with its expert's last row.
//
// 32768 rows, 8 experts 2048 -> 4096 in bf16 (0.55 TFLOP): y 0.45 ms, 1.2
// PFLOP/s; dx 0.43, dW 0.43.  Feed and products bound it together: the loads to
// LDS alone, without reads and products, take 0.36 / 0.30 / 0.30 ms (with what
// the tiles write), all but the loads 0.31 / 0.34 / 0.33.  By the counters the
// matrix pipes work 46 / 57 / 53 % of the time (y with silu, dx, dW) and 32 / 25 /
// 21 % of the requests miss the L2.  A tile's first loads and its epilogue stand
// alone, no products beside them: an activation adds what its instructions take
// (silu 16 us to y's 453, gelu 48), and short sums feel it most: 16384 rows, 16
// experts 1024 -> 4096 in f16 (0.14 TFLOP, 96 us at a large product's rate) take
// 138 us without one, 150 with silu, 166 with gelu.
//
// A wave's direct-to-LDS store is 64 consecutive chunks of a unit's layout
// in LDS, so the layout's permutation is made on the global side: each lane
// fetches the chunk that belongs at its place.  B's fragments come in pairs
// that share 32 columns, so a lane ends with 8 consecutive columns of a row of
// C, one 16-byte store.
#include "lapsum_tile_mfma.h"

namespace lapsum {

// BM x BN of a piece, from its row i0 and column j0
template <class T, int FORM, int ACT, int BM, int BN>
LS_DEV void form_tile(const Piece<T>& p, int i0, int j0, char* lds) {
    constexpr bool kA = FORM != kFormDw, kB = FORM == kFormY;  // k contiguous?
    using Tile = TileSums<T, kA, kB, BM, BN>;
    using Z = typename ZKeep<T>::type;
    constexpr int FM = Tile::FM, FN = Tile::FN;
    const int l = lane_id(), w = uniform(threadIdx.x >> 6);
    const int r0 = (w >> 1) * (BM / 2), c0 = (w & 1) * (BN / 2);
    const int M = p.M - i0, N = p.N - j0;

    Tile tile;
    tile.run(p.a + (kA ? (long long)i0 * p.lda : i0), M, p.lda, p.b + (kB ? (long long)j0 * p.ldb : j0), N, p.ldb, p.K,
             lds);
    auto& acc = tile.acc;
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

template <class T, int FORM, int ACT, int BM, int BN>
__global__ __launch_bounds__(kProductThreads) void k_product(LinearArgs g) {
    constexpr int kGroup = 4;  // row tiles that walk the columns together: 4 x 8 tiles on an XCD at a time
    constexpr bool kCut = BM == 256;
    __shared__ __align__(1024) char lds[kRing * BM * kStepK * 2];
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
// an expert on average, here of each):
//   y, 64 experts 2048 -> 1024, R = 1:      39 / 40 / 45    (few rows: more
//                               R = 16:     39 / 41 / 46    workgroups stream
//                               R = 64:     54 / 48 / 53    the weights)
//   y, 8 experts 2048 -> 2048, R = 512:     56 / 34 / 43
//                              R = 1024:   106 / 64 / 56
//   y, 64 experts 512 -> 1024, R = 256:     38 / 27 / 26    (a short sum)
//   dx, 8 experts 2048 -> 1024, R = 25:    9.3 / 11 / 15
//                               R = 512:    33 / 22 / 30
//   dW, 8 experts, 512 x 512, R = 512:     6.1 / 7.7 / 9.2
//       8 experts, 2048 x 1024, R = 512:    33 / 24 / 23
//       64 experts, 1024 x 2048, R = 1:     83 / 69 / 73
// R takes the experts without rows in, so rows that are all one expert's among
// many get too small a tile: 4096 rows 1024 -> 128, y 58 us as one of 1024
// experts and 8 as the only one.  And dW's sum is never split over workgroups:
// 65536 rows of 4 experts 64 -> 64 take 58 us on 4 of them, their bytes 3.
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
    // us, weights in the memory-side cache (as far as it holds them) and from
    // memory, every expert with rows: 64 experts 2048 -> 1024, 1 row of an expert
    // 38 / 39 and 63 / 46, 2 rows 39 / 41 and 63 / 48, 4 rows 39 / 44 and 64 / 52, 8
    // rows 39 / 50 and 64 / 62; 8 experts 2048 -> 4096, 2 rows 21 / 22 and 33 / 26;
    // 64 experts 512 -> 1024, 4 rows 12 / 15 and 15 / 19; 16 experts 512 -> 512, 4
    // rows 5.5 / 4.0 and 8.1 / 4.8.
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
