// What the experts' matrix kernels share: the 16-bit matrix instruction and
// how a step's operand lies in LDS (gfx950).
//
// A step is 64 bytes of k of R rows, laid out against bank conflicts in the
// reads below (which lanes' reads meet: lapsum_tile_mfma.h).  The counters of
// the 256-wide tiles show none where k is contiguous in both operands, and
// conflicts in a third of the cycles that LDS indexes with one transposed
// operand, in half of them with two:
//   k contiguous: row i has 4 chunks of 16 bytes, two rows to a line of 128;
//     chunk c lies at c ^ fold(line) within its row's half.  A fragment is one
//     16-byte read a lane.
//   own index contiguous: row k has R elements; chunk c lies at c ^ fold(k).
//     16-bit fragments are two transposing 8-byte reads (ds_read_b64_tr_b16).
#pragma once
#include <type_traits>

#include "lapsum_expert_ops.h"

namespace lapsum {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

#define LS_LDS(T) __attribute__((address_space(3))) T

template <class T>
LS_DEV f32x4 mfma16(s16x8 a, s16x8 b, f32x4 c) {
    if constexpr (std::is_same_v<T, __bf16>)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

// KFAST: k is contiguous.  PAIRED: fragments 2 j and 2 j + 1 share the rows
// 32 j .. + 31, row 8 q + 4 (f & 1) + r being row 4 q + r of fragment f, so
// that a lane that holds both has 8 consecutive rows of them; else fragment f
// has the rows 16 f .. + 15.
template <int R, bool KFAST, bool PAIRED>
struct StepLds {
    static constexpr int kBytes = R * 64;
    static LS_DEV int fold(int q) {
        if (KFAST) return PAIRED ? (q & 1) | (q >> 1 & 2) : q & 3;
        // k rows of 64 and 128 bytes differ in banks by themselves
        if (R == 32) return 0;
        return PAIRED ? (R == 64 ? (q >> 1 & 1) << 2 : (q & 3) << 2) : (q & 3) << 1;
    }
    // 16-bit fragment f of the rows from r0: lane l has row l % 16 of it, k
    // 8 (l / 16) .. + 7
    static LS_DEV s16x8 frag(const char* lds, int r0, int f) {
        const int l = lane_id(), g = l >> 4, i = l & 15;
        if (KFAST) {
            const int r = PAIRED ? (f >> 1) * 32 + (i >> 2) * 8 + (f & 1) * 4 + (i & 3) : f * 16 + i;
            const int u = ((i & 1) * 4 + g) ^ fold(r >> 1 & 7);
            return *(const s16x8*)(lds + ((r0 + r) >> 1) * 128 + u * 16);
        }
        // the read gives lane l column l % 16 of 16, taken 4 columns at a time
        // from the places that lanes 4 q + b name: row q, block b
        // (the fold changes a chunk's low three or four bits, so at most four
        // addresses serve all fragments)
        const int k = g * 8 + (i >> 2), b = i & 3;
        const int c = PAIRED ? ((r0 >> 3) + b) ^ fold(k) ^ (f >> 1) << 2
                             : ((r0 >> 3) + (f & 3) * 2 + (b >> 1) ^ fold(k)) + (f >> 2) * 8;
        const char* p = lds + k * (R * 2) + c * 16 + (PAIRED ? f & 1 : b & 1) * 8;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LS_LDS(s16x4)*)p);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LS_LDS(s16x4)*)(p + 4 * R * 2));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    // fp32 fragment f of 32 rows: lane l has row l % 32, k 8 b + 4 (l / 32) .. + 3
    static LS_DEV f32x4 frag32(const char* lds, int r0, int f, int b) {
        const int l = lane_id(), r = r0 + f * 32 + (l & 31);
        if (KFAST) {
            const int u = ((r & 1) * 4 + b * 2 + (l >> 5)) ^ fold(r >> 1 & 7);
            return *(const f32x4*)(lds + (r >> 1) * 128 + u * 16);
        }
        f32x4 v;
        const float* p = (const float*)lds + (b * 8 + (l >> 5) * 4) * R + r;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = p[e * R];
        return v;
    }
};

// What a tile is cut from: A's and B's element (0, 0), C's row 0, the rows
// and columns there are, and the length of the sum.
template <class T>
struct Piece {
    const T *a, *b, *bias;
    T* c;
    typename ZKeep<T>::type* z;
    int M, N, K, lda, ldb, ldc;
};
// A piece, the number of its row tiles, and a tile's number in it.
template <class T>
struct Place {
    Piece<T> p;
    int q, rows;
};

// The piece of tile t of a row form, in tiles of BM rows and `cols` columns.
// I: int, or long long where a launch may count 2^31 tiles (their number is
// only bounded, by one more for each expert; a piece has fewer).
template <class T, int FORM, int BM, class I>
LS_DEV Place<T> row_place(const LinearArgs& g, RowTiles<BM>& tiles, I t, int cols) {
    Place<T> r;
    Piece<T>& p = r.p;
    const RowTile at = tiles.find((int)(t / cols));
    const bool used = at.e < g.E;
    p.M = at.ehi - at.elo;
    p.N = FORM == kFormY ? g.out : g.in;
    p.K = !used ? 0 : FORM == kFormY ? g.in : g.out;  // unused rows: zeros
    p.lda = FORM == kFormY ? g.in : g.out;
    p.ldb = g.in;
    p.ldc = p.N;
    p.a = (const T*)g.a + (long long)at.elo * p.lda;
    p.b = (const T*)g.b + (long long)(used ? at.e : 0) * g.out * g.in;
    p.c = (T*)g.c + (long long)at.elo * p.N;
    p.bias = FORM == kFormY && g.bias && used ? (const T*)g.bias + (long long)at.e * g.out : nullptr;
    p.z = FORM == kFormY && g.z && used ? (typename ZKeep<T>::type*)g.z + (long long)at.elo * p.N : nullptr;
    r.rows = (p.M + BM - 1) / BM;
    r.q = (int)(t - (I)at.first * cols);
    return r;
}
// the same of the weight gradient
template <class T, int BM, class I>
LS_DEV Place<T> dw_place(const LinearArgs& g, I t, int cols) {
    Place<T> r;
    Piece<T>& p = r.p;
    r.rows = (g.out + BM - 1) / BM;
    const int e = (int)(t / (r.rows * cols));
    r.q = (int)(t % (r.rows * cols));
    const int lo = uniform(row_at(g.off, e, g.P));
    p.M = g.out;
    p.N = g.in;
    p.K = max(uniform(row_at(g.off, e + 1, g.P)) - lo, 0);
    p.lda = g.out;
    p.ldb = g.in;
    p.ldc = g.in;
    p.a = (const T*)g.a + (long long)lo * g.out;
    p.b = (const T*)g.b + (long long)lo * g.in;
    p.c = (T*)g.c + (long long)e * g.out * g.in;
    p.bias = nullptr;
    p.z = nullptr;
    return r;
}

}  // namespace lapsum
