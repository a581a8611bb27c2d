// The experts' products on rows and weights in 8 bits: e4m3 values in blocks of
// 128 along the sum, each under a power of two.
//
// Mathematics: y(i, j) = act(sum over blocks b of 2^(ea(i, b) + eb(j, b)) times
// the sum over k of b of qa(i, k) qb(j, k), + bias(j)), i over one expert's
// rows.  The matrix instruction v_mfma_scale_f32_32x32x64_f8f6f4 takes the two
// powers of two of each row from registers and multiplies them in, so the
// blocks' sums run on in one fp32 accumulator.
//
// The tiles are those of the 16-bit products (lapsum_tile_mfma.h): four waves,
// a quarter of a B x B tile each, operands straight from memory to a ring of
// five LDS units, a block (128 bytes of k, a line of memory) of one operand
// each.  A step is one matrix instruction deep (64 k), two steps are a block,
// and a row is whole blocks, so no load is masked along the sum.
//  - Scales stay in registers, 16 blocks' of each row that a lane multiplies,
//    shifted on by a byte a block; the next 16 are fetched after 2048 k.
//  - A weight fragment's rows are dealt out so that a lane's 16 sums of one
//    row are 16 consecutive columns.
//
// 32768 rows, 8 experts 2048 -> 4096, bf16 results: 306 to 315 us (1.77 PFLOP/s; a
// library's product of one such size, unscaled, 264), with silu 332 to 342, where
// the 16-bit product takes 459 and 480; 4096 -> 4096: 524 us (2.1 PFLOP/s).  Of a
// tile's 39 us the loop takes 30, its first loads 3.5 and its results 5.5: all CUs
// write theirs at once, 33 MB, and memory bounds that.  The loop is bound by its
// feed, 10 TB/s: a sum of 32768 for 4096 x 4096 takes 448 us, 446 with a quarter of
// its matrix instructions, 408 with all of them and operands that L2 always
// holds (22 % of the requests miss it), 310 without loads (the matrix pipes' own
// time, at 1.9 GHz).  More loads in flight, a third unit's, did not help: 508.
// 64 rows at 41 of 64 experts 2048 -> 1024, 86 MB: 17 us.
//
// Accuracy.  Of eight neighbouring products that instruction drops what is 2^14
// and more below the largest (measured: a product of 2^-13 of the largest is
// kept, one of 2^-14 is not; between groups of eight, and into the accumulator,
// fp32), which leaves sums of random rows 1.5e-5 off in the 2-norm, whatever
// their length: a thirtieth of fp16's rounding.  Results in fp32 take the bf16
// instruction instead, on values expanded in registers, scales and all: e4m3
// fits bf16 down to 2^-126 (below, a value keeps bf16's nearest multiple of
// 2^-133), so the products are exact and the sums fp32's own: 32768 rows, 8 experts
// 2048 -> 4096 529 us, 4096 -> 4096 946, 64 rows over 64 experts 2048 -> 1024 23.4 (bf16
// results 309, 523 and 21.5).
#include "lapsum_layer_ops.h"
#include "lapsum_tile_mfma.h"

namespace lapsum {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(1)));

// One operand of a tile: R rows by a block of k, 128 bytes of each.  COLS: its
// rows are the product's columns, dealt out to a fragment as above.
template <int R, bool COLS>
struct Operand8 {
    static constexpr int kBytes = R * kBlock8;
    static constexpr int kLoads = kBytes / (kProductThreads * 16);  // a wave's loads per block

    const char* base;  // the tile's first row
    uint32_t bytes;    // of the rows that exist
    uint32_t voff[kLoads];

    // A row is a line of 128 bytes, whose chunk c of 16 lies at c ^ fold(row).
    // LDS serves 256 bytes of such reads at a time: of the lanes 0-3, 12-15, 20-23
    // and 24-27, then of 4-11, 16-19 and 28-31, and the same from 32 (measured, by
    // pairs of lanes).  Of each sixteen the even rows have eight folds, and the odd.
    static LS_DEV int fold(int row) { return row >> 1 & 7; }

    LS_DEV void init(const uint8_t* x, int own, uint32_t ld) {
        base = reinterpret_cast<const char*>(x);
        bytes = (uint32_t)min(R, own) * ld;
        const int l = lane_id(), w = uniform(threadIdx.x >> 6);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int row = (w * kLoads + i) * 8 + (l >> 3);
            voff[i] = (uint32_t)row * ld + ((l & 7) ^ fold(row)) * 16;
        }
    }
    // the buffer of block b (empty past the last: its loads write zeros)
    LS_DEV u32x4 window(int b, int blocks) const {
        const char* p = base + (size_t)b * kBlock8;
        return u32x4{(uint32_t)(uintptr_t)p, (uint32_t)((uintptr_t)p >> 32),
                     b < blocks ? bytes - (uint32_t)b * kBlock8 : 0u, 0x00020000u};
    }
    LS_DEV void load(const u32x4& win, uint32_t lds, int i) const {
        load_to_lds(win, voff[i], lds + (uniform(threadIdx.x >> 6) * kLoads + i) * 1024);
    }
    // the row of the operand that lane l has of fragment f of the rows from r0
    static LS_DEV int row(int r0, int f) {
        const int s = lane_id() & 31;
        return r0 + f * 32 + (COLS ? (s >> 2 & 1) * 16 + (s >> 3) * 4 + (s & 3) : s);
    }
    // half h of it in step q of the block: chunk 4 q + 2 (l / 32) + h of its row
    static LS_DEV u32x4 half(const char* lds, int r0, int f, int q, int h) {
        const int r = row(r0, f), c = q * 4 + (lane_id() >> 5) * 2 + h;
        return *(const u32x4*)(lds + r * kBlock8 + (c ^ fold(r)) * 16);
    }
};

// 16 blocks' scales of a row from block b, of an array with `left` bytes from
// the row's first; bytes past the row are never used
LS_DEV u32x4 scales16(const uint8_t* row, int b, long long left) {
    if (b + 16 <= left) return *reinterpret_cast<const u32x4u*>(row + b);
    uint64_t v[2] = {};
#pragma unroll 1
    for (int i = 0; b + i < left; ++i) {
        const uint64_t x = (uint64_t)row[b + i] << (i & 7) * 8;
        if (i < 8) v[0] |= x;
        else v[1] |= x;
    }
    return u32x4{(uint32_t)v[0], (uint32_t)(v[0] >> 32), (uint32_t)v[1], (uint32_t)(v[1] >> 32)};
}

// 16 values (a half of a fragment) under the power of two of scale byte 0, in bf16
LS_DEV void expand(bf16x8 (&o)[2], u32x4 v, uint32_t scale) {
    const float by = __uint_as_float((scale & 255u) << 23);  // the exponent is all that counts
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[w], by, false);
        const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[w], by, true);
        const int at = (w & 1) * 4;
        o[w >> 1][at] = lo[0], o[w >> 1][at + 1] = lo[1], o[w >> 1][at + 2] = hi[0], o[w >> 1][at + 3] = hi[1];
    }
}

// EXACT: by the bf16 instruction
template <int B, bool EXACT>
struct TileSums8 {
    using OpA = Operand8<B, false>;
    using OpB = Operand8<B, true>;
    static constexpr int F = B / 64;  // fragments of a wave, of rows and of columns
    static constexpr int kUnit = OpA::kBytes;
    static constexpr int kLds = kRing * kUnit;

    f32x16 acc[F][F] = {};

    // a, as: the tile's first row and its scales, M rows from there; b, bs, N
    // the same of its columns; left_a, left_b: scales from there to the array's end
    LS_DEV void run(const uint8_t* a, const uint8_t* as, int M, long long left_a, const uint8_t* b, const uint8_t* bs,
                    int N, long long left_b, int blocks, char* lds) {
        const int K = blocks * kBlock8, w = uniform(threadIdx.x >> 6);
        const int r0 = (w >> 1) * (B / 2), c0 = (w & 1) * (B / 2);
        OpA oa;
        OpB ob;
        oa.init(a, M, (uint32_t)K);
        ob.init(b, N, (uint32_t)K);
        u32x4 sa[F], sb[F];
        auto scales = [&](int blk) {
#pragma unroll
            for (int i = 0; i < F; ++i) {
                const long long at = (long long)min(OpA::row(r0, i), M - 1) * blocks;
                sa[i] = scales16(as + at, blk, left_a - at);
            }
#pragma unroll
            for (int j = 0; j < F; ++j) {
                const long long at = (long long)min(OpB::row(c0, j), N - 1) * blocks;
                sb[j] = scales16(bs + at, blk, left_b - at);
            }
        };
        const uint32_t at = (uint32_t)(uintptr_t)(LS_LDS(char)*)lds;
        auto fetch = [&](const auto& op, const u32x4& win, int to, int from, int end) {
#pragma unroll
            for (int i = from; i < end; ++i) op.load(win, at + to, i);
        };
        // the units of the block that is multiplied, of the next, and a free one
        int ua = 0, ub = kUnit, na = 2 * kUnit, nb = 3 * kUnit, spare = 4 * kUnit;
        fetch(oa, oa.window(0, blocks), ua, 0, OpA::kLoads);
        fetch(ob, ob.window(0, blocks), ub, 0, OpB::kLoads);
        fetch(oa, oa.window(1, blocks), na, 0, OpA::kLoads);
        fetch(ob, ob.window(1, blocks), nb, 0, OpB::kLoads);
        u32x4 fa[2][F][2], fb[2][F][2];
        step_barrier<OpA::kLoads + OpB::kLoads>();
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                fb[0][f][h] = OpB::half(lds + ub, c0, f, 0, h);
                fa[0][f][h] = OpA::half(lds + ua, r0, f, 0, h);
            }
        auto whole = [](const u32x4 (&f)[2]) {
            return __builtin_bit_cast(i32x8, __builtin_shufflevector(f[0], f[1], 0, 1, 2, 3, 4, 5, 6, 7));
        };
        // Step q of block b multiplies the fragments of set q and reads the next
        // step's into the other.  Step 0 fetches A of block b + 2 into the free
        // unit.  Step 1, when all waves have read block b, waits for block b + 1
        // and fetches B of block b + 2 to where A of b was; where its B was is free
        // then.
        auto step = [&](auto qv, int blk) {
            constexpr int q = decltype(qv)::value;
            if (q) step_barrier<OpA::kLoads>();
            const char *pa = lds + (q ? na : ua), *pb = lds + (q ? nb : ub);
            constexpr int kReads = 4 * F, kReadIn = F > 1 ? F / 2 : 1;
            const u32x4 win = q ? ob.window(blk + 2, blocks) : oa.window(blk + 2, blocks);
#pragma unroll
            for (int i = 0; i < F; ++i) {
                if (i < kReadIn) {
#pragma unroll
                    for (int r = i * kReads / kReadIn; r < (i + 1) * kReads / kReadIn; ++r) {
                        const int f = r >> 1;
                        if (f < F) fb[q ^ 1][f][r & 1] = OpB::half(pb, c0, f, q ^ 1, r & 1);
                        else fa[q ^ 1][f - F][r & 1] = OpA::half(pa, r0, f - F, q ^ 1, r & 1);
                    }
                }
                if (q) fetch(ob, win, ua, i * OpB::kLoads / F, (i + 1) * OpB::kLoads / F);
                else fetch(oa, win, spare, i * OpA::kLoads / F, (i + 1) * OpA::kLoads / F);
                if constexpr (EXACT) {
                    bf16x8 a[2][2];
                    expand(a[0], fa[q][i][0], sa[i][0]);
                    expand(a[1], fa[q][i][1], sa[i][0]);
#pragma unroll
                    for (int j = 0; j < F; ++j) {
                        bf16x8 b[2][2];
                        expand(b[0], fb[q][j][0], sb[j][0]);
                        expand(b[1], fb[q][j][1], sb[j][0]);
#pragma unroll
                        for (int h = 0; h < 4; ++h)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[h >> 1][h & 1], a[h >> 1][h & 1],
                                                                                acc[i][j], 0, 0, 0);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < F; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                            whole(fb[q][j]), whole(fa[q][i]), acc[i][j], 0, 0, 0, (int)sb[j][0], 0, (int)sa[i][0]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        auto on = [](u32x4& s) {  // to the next block's scale
            s[0] = __builtin_amdgcn_alignbyte(s[1], s[0], 1);
            s[1] = __builtin_amdgcn_alignbyte(s[2], s[1], 1);
            s[2] = __builtin_amdgcn_alignbyte(s[3], s[2], 1);
            s[3] >>= 8;
        };
        // (the inner loop has no branch: past one the compiler would sink the
        // products, and the loads would stand together)
        for (int b0 = 0; b0 < blocks; b0 += 16) {
            scales(b0);
            const int end = min(b0 + 16, blocks);
            for (int blk = b0; blk < end; ++blk) {
                step(std::integral_constant<int, 0>{}, blk);
                step(std::integral_constant<int, 1>{}, blk);
#pragma unroll
                for (int f = 0; f < F; ++f) on(sa[f]), on(sb[f]);
                const int free = ub;
                ub = nb, nb = ua, ua = na, na = spare, spare = free;
            }
        }
        // the last steps' loads, past the last block, still write zeros to LDS
        step_barrier<0>();
    }
};

typedef uint32_t Words8 __attribute__((ext_vector_type(4), aligned(2)));  // 16 bytes at any element

struct Piece8 {
    const uint8_t *a, *as, *b, *bs;
    long long left_a, left_b;
    const void* bias;
    void* c;
    int M, N, blocks;  // blocks: 0 for unused rows
};
template <class T, int ACT, int B>
LS_DEV void tile8(const Piece8& p, int i0, int j0, char* lds) {
    using Tile = TileSums8<B, sizeof(T) == 4>;
    Tile tile;
    const int M = p.M - i0, N = p.N - j0;
    if (p.blocks > 0) {
        const long long a = (long long)i0 * p.blocks, b = (long long)j0 * p.blocks;
        tile.run(p.a + a * kBlock8, p.as + a, M, p.left_a - a, p.b + b * kBlock8, p.bs + b, N, p.left_b - b, p.blocks,
                 lds);
    }
    // A wave's quarter leaves through its own part of LDS, kPass rows at a time:
    // in registers a lane has 16 columns of 32 rows, from LDS it takes 16 bytes
    // of a row, its neighbours the next, so bias and activation are a short loop
    // and the stores are whole lines (unrolled over the registers: the same time
    // from ten times the code).
    constexpr int WR = B / 2, WC = B / 2, V = 16 / (int)sizeof(T);
    constexpr int kLine = WC * 4 + 16;  // bytes of a row: neighbouring rows meet other banks
    constexpr int kPass = WR < 64 ? WR : 64;
    static_assert(4 * kPass * kLine <= Tile::kLds);
    constexpr int kLanes = WC / V, kRows = 64 / kLanes;  // lanes of a row, rows at a time
    const int l = lane_id(), w = uniform(threadIdx.x >> 6);
    const int r0 = i0 + (w >> 1) * WR, c0 = j0 + (w & 1) * WC;
    const int col = c0 + l % kLanes * V;
    char* own = lds + w * kPass * kLine;
    struct Chunk { T v[V]; };
    Chunk bias{};
    const bool whole = col + V <= p.N;
    if (p.bias && whole) {
        bias = __builtin_bit_cast(Chunk, *reinterpret_cast<const Words8*>((const T*)p.bias + col));
    } else if (p.bias) {
#pragma unroll
        for (int r = 0; r < V; ++r)
            if (col + r < p.N) bias.v[r] = ((const T*)p.bias)[col + r];
    }
#pragma unroll
    for (int pass = 0; pass < WR; pass += kPass) {
        // (a wave's own LDS operations are served in order)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int i = 0; i < kPass / 32; ++i)
#pragma unroll
            for (int j = 0; j < Tile::F; ++j)
#pragma unroll
                for (int q = 0; q < 16; q += 4) {
                    const f32x16& a = tile.acc[pass / 32 + i][j];
                    *(f32x4*)(own + (i * 32 + (l & 31)) * kLine + (j * 32 + (l >> 5) * 16 + q) * 4) =
                        f32x4{a[q], a[q + 1], a[q + 2], a[q + 3]};
                }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        // kAhead rows' reads in flight at a time
        constexpr int kTimes = kPass / kRows, kAhead = kTimes < 8 ? kTimes : 8;
        static_assert(kTimes % kAhead == 0);
#pragma unroll 1
        for (int t = 0; t < kTimes; t += kAhead) {
            f32x4 v[kAhead][V / 4];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const f32x4* at = (const f32x4*)(own + ((t + u) * kRows + l / kLanes) * kLine + l % kLanes * V * 4);
#pragma unroll
                for (int q = 0; q < V / 4; ++q) v[u][q] = at[q];
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int row = r0 + pass + (t + u) * kRows + l / kLanes;
                Chunk o;
#pragma unroll
                for (int q = 0; q < V; ++q) o.v[q] = from_f<T>(act_of<ACT, T>(v[u][q / 4][q % 4] + to_f(bias.v[q])));
                if (row >= p.M) continue;
                T* c = (T*)p.c + (long long)row * p.N + col;
                if (whole) {
                    *reinterpret_cast<Words8*>(c) = __builtin_bit_cast(u32x4, o);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (col + e < p.N) c[e] = o.v[e];
                }
            }
        }
    }
}

template <class T, int ACT, int B>
__global__ __launch_bounds__(kProductThreads) void k_linear8(Linear8Args g) {
    constexpr int kGroup = 4;  // row tiles that walk the columns together
    constexpr bool kCut = B == 256;
    __shared__ __align__(1024) char lds[TileSums8<B, false>::kLds];
    const int cols = (g.out + B - 1) / B;
    RowTiles<B> rows(g.off, g.E, g.P);
    const Turn t = take_turn(blockIdx.x, rows.count() * cols, kCut);
    if (t.tile < 0) return;
    const RowTile at = rows.find(t.tile / cols);
    const bool used = at.e < g.E;
    const long long e = used ? at.e : 0, row = (long long)g.blocks, mat = (long long)g.out * g.blocks;
    Piece8 p;
    p.M = at.ehi - at.elo;
    p.N = g.out;
    p.blocks = used ? g.blocks : 0;  // unused rows: zeros
    p.a = g.a + at.elo * row * kBlock8;
    p.as = g.as + at.elo * row;
    p.left_a = (g.P - at.elo) * row;
    p.b = g.b + e * mat * kBlock8;
    p.bs = g.bs + e * mat;
    p.left_b = (g.E - e) * mat;
    p.bias = g.bias && used ? (const T*)g.bias + e * g.out : nullptr;
    p.c = (T*)g.c + (long long)at.elo * g.out;
    const int q = t.tile - at.first * cols, tiles = (p.M + B - 1) / B;
    const int first = q / (kGroup * cols) * kGroup, n = min(kGroup, tiles - first), in = q - first * cols;
    int i0 = (first + in % n) * B, j0 = in / n * B;
    if constexpr (kCut) {
        if (t.quarter >= 0) {
            i0 += (t.quarter >> 1) * (B / 2);
            j0 += (t.quarter & 1) * (B / 2);
            if (i0 < p.M && j0 < p.N) tile8<T, ACT, B / 2>(p, i0, j0, lds);
            return;
        }
    }
    tile8<T, ACT, B>(p, i0, j0, lds);
}

void launch_expert_linear8(int dtype, const Linear8Args& g, hipStream_t st) {
    if (g.P < 1 || g.out < 1) return;
    with_dtype(dtype, [&](auto tv) {
        using T = decltype(tv);
        with_act(g.act, [&](auto av) {
            auto launch = [&](auto bv) {
                constexpr int B = bv.value;
                const long long tiles = max_row_tiles<B>(g.P, g.E) * ceil_div(g.out, B);
                hipLaunchKernelGGL((k_linear8<T, decltype(av)::value, B>), dim3((unsigned)turns(tiles, B == 256)),
                                   dim3(kProductThreads), 0, st, g);
            };
            const long long per = g.P / g.E;
            // one tile a workgroup, whose threads a launch counts in 32 bits
            const bool many = max_row_tiles<64>(g.P, g.E) * ceil_div(g.out, 64) >= kGridMax;
            // (fp32's expanded fragments leave no registers for the widest)
            const bool widest = sizeof(T) == 2 && per >= 96 && (g.P / 256 + g.E / 2) * ceil_div(g.out, 256) >= 256;
            if (many || widest) launch(std::integral_constant<int, 256>{});
            else if (per > 32 && (g.P / 128 + g.E / 2) * ceil_div(g.out, 128) >= 128)
                launch(std::integral_constant<int, 128>{});
            else launch(std::integral_constant<int, 64>{});
        });
    });
}

}  // namespace lapsum
