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
// A workgroup forms a BM x BN tile of C, 64 steps of k at a time.  The steps'
// operands go from memory to LDS without passing through registers
// (buffer_load ... lds, 16 bytes a lane), into one of two buffers while the
// other is multiplied.  Reads out of range return zero, which is all the
// masking that ragged experts need: a tile's buffer ends with its expert's
// last row.
//
// LDS layout, free of bank conflicts for the fragment reads below:
//   k contiguous: row i has 64 k = 8 chunks of 16 bytes; chunk c lies at
//     c ^ (i & 7).  A fragment is one 16-byte read a lane.
//   own index contiguous: row k has BM (BN) elements; the pair of chunks q
//     (16 elements) lies at q ^ ((k & 3) | (k >> 3 & 1) << 2).  A fragment is
//     two transposing 8-byte reads (ds_read_b64_tr_b16).
// A wave's direct-to-LDS store is 64 consecutive chunks, so the permutation
// is made on the global side: each lane fetches the chunk that belongs at its
// place.
#include "lapsum_expert_ops.h"

namespace lapsum {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

#define LS_LDS(T) __attribute__((address_space(3))) T

constexpr int kStepK = 64;  // k of one LDS buffer

template <class T>
LS_DEV f32x4 mfma16(s16x8 a, s16x8 b, f32x4 c);
template <>
LS_DEV f32x4 mfma16<__bf16>(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}
template <>
LS_DEV f32x4 mfma16<_Float16>(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

// 16 bytes a lane from buffer offset `off` to LDS, lane l at `lds` + 16 l.
// Written as an instruction so that the compiler's counters do not wait for
// it at the next LDS read: step_barrier does, one step later.  It has no
// register output.
LS_DEV void load_to_lds(u32x4 rsrc, uint32_t off, uint32_t lds) {
    asm volatile(
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %0, %1, 0 offen lds"
        :
        : "v"(off), "s"(rsrc), "s"(lds)
        : "memory");
}

// One operand of a tile: R rows (of its own index) by kStepK of k.
// KFAST: k is contiguous in memory.
template <int R, bool KFAST, int WAVES>
struct Operand {
    static constexpr int kBytes = R * kStepK * 2;
    static constexpr int kLoads = kBytes / (WAVES * 1024);  // a wave's loads per step
    static_assert(kLoads * WAVES * 1024 == kBytes, "whole waves of loads");

    const char* base;  // of the tile's first row and k
    uint32_t rows;     // rows of the tile that exist (KFAST), else its k
    uint32_t ld;       // bytes between rows of memory
    uint32_t voff[kLoads];
    uint32_t kcol;     // KFAST: first k of this lane's chunk
    uint32_t last;     // else: bytes of the tile's last memory row that exist

    // x: element (0, 0) of the tile; own: rows left (its own index); K: length
    // of the sum; ld: elements between memory rows
    template <class T>
    LS_DEV void init(const T* x, long long own, int K, int ld_) {
        base = reinterpret_cast<const char*>(x);
        ld = (uint32_t)ld_ * 2u;
        const int l = lane_id(), w = uniform(threadIdx.x >> 6);
        if (KFAST) {
            rows = (uint32_t)min((long long)R, own);
            const int c = (l & 7) ^ (l >> 3);
            kcol = c * 8;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) voff[i] = (uint32_t)((w * kLoads + i) * 8 + (l >> 3)) * ld + c * 16;
        } else {
            rows = (uint32_t)K;
            last = (uint32_t)min((long long)R, own) * 2u;
            constexpr int kChunks = R / 8;          // chunks of a k row
            constexpr int kPer = 64 / kChunks;      // k rows of one load
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int k = (w * kLoads + i) * kPer + l / kChunks;
                const int f = (k & 3) | ((k >> 3) & 1) << 2;
                voff[i] = (uint32_t)k * ld + (uint32_t)((l % kChunks) ^ (f << 1)) * 16;
            }
        }
    }
    // issues the loads of k0 .. k0 + 63 into LDS from byte address `lds`
    LS_DEV void load(uint32_t lds, int k0, int K) const {
        const int w = uniform(threadIdx.x >> 6);
        const char* p;
        uint32_t n;
        bool on = true;
        if (KFAST) {
            p = base + (size_t)k0 * 2;
            n = rows * ld - (uint32_t)k0 * 2;
            on = k0 + (int)kcol < K;  // the last step: what follows in memory is the next row
        } else {
            p = base + (size_t)k0 * ld;
            n = (min((uint32_t)kStepK, rows - (uint32_t)k0) - 1u) * ld + last;
        }
        const u32x4 rs = {(uint32_t)(uintptr_t)p, (uint32_t)((uintptr_t)p >> 32), n, 0x00020000u};
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            load_to_lds(rs, KFAST ? (on ? voff[i] : 0x80000000u) : voff[i], lds + (w * kLoads + i) * 1024);
    }
    // fragment f (16 rows from r0 + 16 f) of k kk * 32 .. + 31: lane l has row
    // l % 16, k 8 (l / 16) .. + 7
    static LS_DEV s16x8 frag(const char* lds, int r0, int f, int kk) {
        const int l = lane_id(), g = l >> 4, i = l & 15;
        if (KFAST) {
            const int c = (kk * 4 + g) ^ (i & 7);
            return *(const s16x8*)(lds + (r0 + f * 16 + i) * 128 + c * 16);
        }
        const int s = (i >> 2) | (g & 1) << 2;
        const char* p = lds + (kk * 32 + g * 8 + (i >> 2)) * (R * 2) + ((((r0 >> 4) + f) ^ s) << 5) + (i & 3) * 8;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LS_LDS(s16x4)*)p);
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LS_LDS(s16x4)*)(p + 4 * R * 2));
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// every wave's loads have landed and its reads are done; then the workgroup meets
LS_DEV void step_barrier() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Tile `t` of `n` such that the workgroups of one XCD (they are dealt out in
// turn) take neighbouring tiles, which share operands in its L2.  Returns -1
// past the end; the grid has at least 8 ceil(n / 8) workgroups' worth.
LS_DEV int xcd_tile(int block, int n) {
    const int per = (n + 7) >> 3;
    const int t = (block & 7) * per + (block >> 3);
    return (block >> 3) < per && t < n ? t : -1;
}

// BM x BN tile by WM x WN waves
template <class T, int FORM, int ACT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64) void k_product(LinearArgs g) {
    constexpr int kWaves = WM * WN;
    constexpr bool kA = FORM != kFormDw, kB = FORM == kFormY;  // k contiguous?
    using OpA = Operand<BM, kA, kWaves>;
    using OpB = Operand<BN, kB, kWaves>;
    using Z = typename ZKeep<T>::type;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // fragments of a wave
    constexpr int kGroup = 4;                            // row tiles that walk the columns together
    constexpr int kBuffer = OpA::kBytes + OpB::kBytes;
    __shared__ __align__(1024) char lds[2 * kBuffer];

    const int l = lane_id(), w = uniform(threadIdx.x >> 6);
    const int r0 = w / WN * (BM / WM), c0 = w % WN * (BN / WN);
    const int N = FORM == kFormY ? g.out : g.in;
    const int cols = (N + BN - 1) / BN;

    // the tile: rows [0, M) at c, columns [j0, N)
    const T *a = (const T*)g.a, *b = (const T*)g.b;
    T* c = (T*)g.c;
    Z* z = nullptr;
    const T* bias = nullptr;
    int M, K, j0, lda, ldb;
    if (FORM == kFormDw) {
        const int rows = (g.out + BM - 1) / BM, per = rows * cols;
        const int t = xcd_tile(blockIdx.x, per * g.E);
        if (t < 0) return;
        const int e = t / per, q = t % per;
        const int grp = q / (kGroup * cols), first = grp * kGroup, n = min(kGroup, rows - first);
        const int in = q - first * cols, i0 = (first + in % n) * BM;
        j0 = in / n * BN;
        const int lo = uniform(row_at(g.off, e, g.P));
        K = max(uniform(row_at(g.off, e + 1, g.P)) - lo, 0);
        M = g.out - i0, lda = g.out, ldb = g.in;
        a += (long long)lo * lda + i0;
        b += (long long)lo * ldb;
        c += ((long long)e * g.out + i0) * g.in;
    } else {
        const int t = xcd_tile(blockIdx.x, count_row_tiles<BM>(g.off, g.E, g.P) * cols);
        if (t < 0) return;
        // the expert whose tiles hold t / cols, then the place among its tiles
        const RowTile at = find_row_tile<BM>(g.off, g.E, g.P, t / cols);
        const int lo = uniform(row_at(g.off, at.e, g.P));
        const int hi = at.e < g.E ? max(uniform(row_at(g.off, at.e + 1, g.P)), lo) : g.P;
        const int rows = (hi - lo + BM - 1) / BM, q = t - at.first * cols;
        const int grp = q / (kGroup * cols), first = grp * kGroup, n = min(kGroup, rows - first);
        const int in = q - first * cols, i0 = lo + (first + in % n) * BM;
        j0 = in / n * BN;
        M = hi - i0;
        K = FORM == kFormY ? g.in : g.out;
        lda = K, ldb = g.in;
        a += (long long)i0 * lda;
        c += (long long)i0 * N;
        if (at.e < g.E) {
            b += (long long)at.e * g.out * g.in;
            if (FORM == kFormY && g.bias) bias = (const T*)g.bias + (long long)at.e * g.out;
            if (FORM == kFormY && g.z) z = (Z*)g.z + (long long)i0 * N;
        } else {
            K = 0;
        }
    }
    b += FORM == kFormY ? (long long)j0 * ldb : j0;

    f32x4 acc[FM][FN] = {};
    if (K > 0) {
        OpA oa;
        OpB ob;
        oa.init(a, M, K, lda);
        ob.init(b, N - j0, K, ldb);
        const uint32_t at = (uint32_t)(uintptr_t)(LS_LDS(char)*)lds;
        oa.load(at, 0, K);
        ob.load(at + OpA::kBytes, 0, K);
        int buf = 0;
        for (int k0 = 0; k0 < K; k0 += kStepK) {
            step_barrier();
            if (k0 + kStepK < K) {
                const uint32_t to = at + (kBuffer - buf);
                oa.load(to, k0 + kStepK, K);
                ob.load(to + OpA::kBytes, k0 + kStepK, K);
            }
            const char *sa = lds + buf, *sb = sa + OpA::kBytes;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                s16x8 fa[FM], fb[FN];
#pragma unroll
                for (int j = 0; j < FN; ++j) fb[j] = OpB::frag(sb, c0, j, kk);
#pragma unroll
                for (int i = 0; i < FM; ++i) fa[i] = OpA::frag(sa, r0, i, kk);
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j) acc[i][j] = mfma16<T>(fb[j], fa[i], acc[i][j]);
            }
            buf = kBuffer - buf;
        }
    }
    // lane l holds row l % 16 of a fragment, columns 4 (l / 16) .. + 3
    struct __attribute__((aligned(8))) T4 { T v[4]; };
    struct __attribute__((aligned(8))) Z4 { Z v[4]; };
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const int col = j0 + c0 + j * 16 + (l >> 4) * 4;
        if (col >= N) continue;
        float bj[4] = {};
        if (FORM == kFormY && bias) {
            const T4 v = *(const T4*)(bias + col);
#pragma unroll
            for (int r = 0; r < 4; ++r) bj[r] = to_f(v.v[r]);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int row = r0 + i * 16 + (l & 15);
            if (row >= M) continue;
            T4 o;
            Z4 k;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float v = acc[i][j][r] + bj[r];
                if (FORM == kFormY && ACT != kActNone) k.v[r] = ZKeep<T>::make(v);
                o.v[r] = from_f<T>(act_of<ACT>(v));
            }
            *(T4*)(c + (long long)row * N + col) = o;
            if (FORM == kFormY && ACT != kActNone && z) *(Z4*)(z + (long long)row * N + col) = k;
        }
    }
}

template <class T, int BM, int BN, int WM, int WN>
static void launch_tiles(int form, const LinearArgs& g, hipStream_t st) {
    const int N = form == kFormY ? g.out : g.in;
    const long long cols = ceil_div(N, BN);
    const long long tiles = cols * (form == kFormDw ? ceil_div(g.out, BM) * g.E : max_row_tiles<BM>(g.P, g.E));
    const dim3 grid((unsigned)(ceil_div(tiles, 8) * 8)), block(WM * WN * 64);
    if (form == kFormDw)
        hipLaunchKernelGGL((k_product<T, kFormDw, kActNone, BM, BN, WM, WN>), grid, block, 0, st, g);
    else if (form == kFormDx)
        hipLaunchKernelGGL((k_product<T, kFormDx, kActNone, BM, BN, WM, WN>), grid, block, 0, st, g);
    else
        with_act(g.act, [&](auto av) {
            hipLaunchKernelGGL((k_product<T, kFormY, decltype(av)::value, BM, BN, WM, WN>), grid, block, 0, st, g);
        });
}

bool expert_mfma_takes(int form, int dtype, const LinearArgs& g) {
    if (dtype == kF32 || g.in % 8 || g.out % 8 || g.in > (1 << 20) || g.out > (1 << 20)) return false;
    if (!aligned16(g.a) || !aligned16(g.b) || !aligned16(g.c) || !aligned16(g.bias) || !aligned16(g.z)) return false;
    // tiles counted in 32 bits
    const long long tiles = form == kFormDw ? ceil_div(g.out, 128) * ceil_div(g.in, 128) * g.E
                                            : ceil_div(form == kFormY ? g.out : g.in, 128) *
                                                  max_row_tiles<128>(g.P, g.E);
    return tiles < kGridMax;
}

void launch_expert_mfma(int form, int dtype, const LinearArgs& g, hipStream_t st) {
    with_dtype(dtype, [&](auto tv) {
        using T = decltype(tv);
        if constexpr (sizeof(T) == 2) launch_tiles<T, 256, 256, 2, 4>(form, g, st);
    });
}

}  // namespace lapsum
