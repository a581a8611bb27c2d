// The main loop of the matrix kernels for every type, size and alignment
// (gfx950).  Operands go from memory through registers to LDS, 16 bytes a lane
// at any element's address (the hardware takes those), only the ends of rows
// element by element.  What is done with the sums is the callers'.
#pragma once
#include "lapsum_expert_tile.h"

namespace lapsum {

constexpr int kAnyThreads = 256;

// steps of 64 bytes of k in a buffer (split, 513 x 2 rows of 257 -> 1001 in
// fp32, one / two: y 16.6 / 21.6 us, dx 18.6 / 18.6, dW 14.1 / 19.5: 32 KB of
// LDS leave room for five workgroups on a CU, 64 KB for two)
constexpr int any_steps(bool split) { return split ? 1 : 2; }

typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));  // 16 bytes at any element

// One operand: R rows by one step of k, dealt out to NT threads in chunks.
template <class T, int R, bool KFAST, bool PAIRED, int NT>
struct AnyOperand : StepLds<R, KFAST, PAIRED> {
    using Lds = StepLds<R, KFAST, PAIRED>;
    static constexpr int kPer = 16 / (int)sizeof(T);      // elements of a chunk
    static constexpr int kStepK = 64 / (int)sizeof(T);    // k of a step
    static constexpr int kLoads = R * 64 / (NT * 16);     // a thread's chunks per step
    static constexpr int kRow = KFAST ? 4 : R / kPer;     // chunks of a row of memory

    // Where a thread's chunks of k = 0 lie, for fetch(): rows past `own` are
    // the last one's copies, a chunk that starts past a row's end starts at
    // its last element.  What they bring goes into sums that nobody stores.
    const T* at[kLoads];
    LS_DEV void place(const T* __restrict__ x, long long ld, int own, int tid) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int q = i * NT + tid, line = q / kRow, c = q % kRow * kPer;
            at[i] = KFAST ? x + min(line, own - 1) * ld + c : x + line * ld + min(c, own - 1);
        }
    }
    // whether fetch() stays inside: k0 .. k0 + n - 1 are in the sum (of K
    // terms), and where a chunk may pass a row's end another row follows
    static LS_DEV bool inside(long long ld, int k0, int n, int K) {
        return KFAST ? k0 + n <= K : k0 + n < K && ld >= kPer;
    }
    LS_DEV void fetch(u32x4 (&r)[kLoads], long long ld, int k0) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) r[i] = *reinterpret_cast<const Words*>(at[i] + (KFAST ? k0 : k0 * ld));
    }
    // chunks of k0 .. of X (row i, k: x[i * ld + k], or x[k * ld + i]), zeros
    // past `own` rows and K
    static LS_DEV void get(u32x4 (&r)[kLoads], const T* __restrict__ x, long long ld, int own, int k0, int K, int tid) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int q = i * NT + tid, line = q / kRow, at = q % kRow * kPer;
            const int row = KFAST ? line : k0 + line, col = KFAST ? k0 + at : at;
            const int left = row < (KFAST ? own : K) ? (KFAST ? K : own) - col : 0;
            const T* p = x + row * ld + col;
            if (left >= kPer) {
                r[i] = *reinterpret_cast<const Words*>(p);
            } else {
                struct { T v[kPer]; } e = {};
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (j < left) e.v[j] = p[j];
                r[i] = __builtin_bit_cast(u32x4, e);
            }
        }
    }
    static LS_DEV void put(const u32x4 (&r)[kLoads], char* lds, int tid) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int q = i * NT + tid, line = q / kRow, c = q % kRow;
            int at;
            if (KFAST) at = (line >> 1) * 128 + (((line & 1) * 4 + c) ^ Lds::fold(line >> 1 & 7)) * 16;
            else at = line * (R * (int)sizeof(T)) + (sizeof(T) == 2 ? c ^ Lds::fold(line) : c) * 16;
            *(u32x4*)(lds + at) = r[i];
        }
    }
};

// whether an output takes the sums of a shared tile with cell() (below)
template <class P, class = void>
struct HasCell : std::false_type {};
template <class P>
struct HasCell<P, std::void_t<decltype(&P::cell)>> : std::true_type {};

// whether a 16-bit output also wants sums over the rows (below)
template <class P, class = void>
struct HasColumns : std::false_type {};
template <class P>
struct HasColumns<P, std::void_t<decltype(&P::columns)>> : std::true_type {};

// The sums over k < K of a(i, k) b(j, k) of a B x B tile; SPLIT: the waves share
// the sum.  a, b: element (0, 0) of the tile; kA, kB: k is the contiguous index;
// M, N: rows and columns that there are from there (1 and more); lda, ldb:
// elements between memory rows.  put.one(i, j, v) takes a sum of the M x N,
// put.eight(i, j, v) eight of a row, whose columns may pass N.  With SPLIT,
// put.cell(i, j, v, on), if there is one, takes every place of the tile, B
// neighbouring lanes a row of it, `on` where it is one of the M x N.  put.columns,
// if there is one, takes sums over rows of what put.value(i, j, v) makes of those
// (and stores): columns(part, j, s), column j's over the rows of part 0 or 1 of the
// tile, or with SPLIT 0 .. 3.
template <class T, bool kA, bool kB, int B, bool SPLIT, class Put>
LS_DEV void any_sums(const T* a, int M, int lda, const T* b, int N, int ldb, int K_, char* lds, const Put& put) {
    constexpr bool k16 = sizeof(T) == 2;
    constexpr int NT = SPLIT ? 64 : kAnyThreads;
    using OpA = AnyOperand<T, B, kA, false, NT>;
    using OpB = AnyOperand<T, B, kB, k16, NT>;
    constexpr int kAnySteps = any_steps(SPLIT);
    constexpr int kStepK = OpA::kStepK, kDeep = kAnySteps * kStepK;
    constexpr int kBuffer = kAnySteps * (OpA::kBytes + OpB::kBytes);
    constexpr int W = SPLIT ? B : B / 2;         // a wave's rows and columns
    constexpr int FR = k16 ? 16 : 32, F = W / FR;  // fragments
    const int l = lane_id(), w = uniform(threadIdx.x >> 6);
    const int r0 = SPLIT ? 0 : (w >> 1) * W, c0 = SPLIT ? 0 : (w & 1) * W;
    const int tid = SPLIT ? l : (int)threadIdx.x;
    int k0 = 0, K = K_;
    if (SPLIT) {  // this wave's share of the sum, in whole buffers
        const int deep = (K + kDeep - 1) / kDeep;
        k0 = w * deep / 4 * kDeep;
        K = min(K, (w + 1) * deep / 4 * kDeep);
        lds += w * 2 * kBuffer;
    }
    using Acc = std::conditional_t<k16, f32x4, f32x16>;
    Acc acc[F][F] = {};
    u32x4 ra[kAnySteps][OpA::kLoads], rb[kAnySteps][OpB::kLoads];
    OpA oa;
    OpB ob;
    oa.place(a, lda, M, tid);
    ob.place(b, ldb, N, tid);
    auto get = [&](int k) {
        if (k + kDeep <= K && OpA::inside(lda, k, kDeep, K_) && OpB::inside(ldb, k, kDeep, K_)) {
#pragma unroll
            for (int h = 0; h < kAnySteps; ++h) {
                oa.fetch(ra[h], lda, k + h * kStepK);
                ob.fetch(rb[h], ldb, k + h * kStepK);
            }
            return;
        }
#pragma unroll
        for (int h = 0; h < kAnySteps; ++h) {
            OpA::get(ra[h], a, lda, M, k + h * kStepK, K, tid);
            OpB::get(rb[h], b, ldb, N, k + h * kStepK, K, tid);
        }
    };
    if (k0 < K) get(k0);
    int buf = 0;
    for (; k0 < K; k0 += kDeep) {
        char* s = lds + buf;
#pragma unroll
        for (int h = 0; h < kAnySteps; ++h) {
            OpA::put(ra[h], s + h * OpA::kBytes, tid);
            OpB::put(rb[h], s + kAnySteps * OpA::kBytes + h * OpB::kBytes, tid);
        }
        // (a wave's own LDS operations are served in order)
        if (SPLIT) __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        else __syncthreads();
        if (k0 + kDeep < K) get(k0 + kDeep);
#pragma unroll
        for (int h = 0; h < kAnySteps; ++h) {
            const char *sa = s + h * OpA::kBytes, *sb = s + kAnySteps * OpA::kBytes + h * OpB::kBytes;
            if constexpr (k16) {
                s16x8 fa[F], fb[F];
#pragma unroll
                for (int i = 0; i < F; ++i) {
                    fb[i] = OpB::frag(sb, c0, i);
                    fa[i] = OpA::frag(sa, r0, i);
                }
#pragma unroll
                for (int i = 0; i < F; ++i)
#pragma unroll
                    for (int j = 0; j < F; ++j) acc[i][j] = mfma16<T>(fb[j], fa[i], acc[i][j]);
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    f32x4 fa[F], fb[F];
#pragma unroll
                    for (int i = 0; i < F; ++i) {
                        fa[i] = OpA::frag32(sa, r0, i, q);
                        fb[i] = OpB::frag32(sb, c0, i, q);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int i = 0; i < F; ++i)
#pragma unroll
                            for (int j = 0; j < F; ++j)
                                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[i][e], fb[j][e], acc[i][j], 0, 0, 0);
                }
            }
        }
        buf = kBuffer - buf;
    }
    // Where a lane's sums lie: 16-bit, row l % 16 of fragment i and columns
    // 8 (l / 16) + 4 (j & 1) + r of the pair j / 2; fp32, rows
    // 8 (r / 4) + 4 (l / 32) + r % 4 and column l % 32
    if constexpr (k16 && !SPLIT && HasColumns<Put>::value) {
#pragma unroll
        for (int j = 0; j < F; j += 2) {
            const int col = c0 + j * 16 + (l >> 4) * 8;
            float s[8] = {};
#pragma unroll
            for (int i = 0; i < F; ++i) {
                const int row = r0 + i * 16 + (l & 15);
                if (row >= M) continue;
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (col + r < N) s[r] += put.value(row, col + r, acc[i][j + (r >> 2)][r & 3]);
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {  // over the 16 lanes of a column
                s[r] += __uint_as_float(xor_lane<8>(__float_as_uint(s[r])));
                s[r] += __uint_as_float(xor_lane<4>(__float_as_uint(s[r])));
                s[r] += __uint_as_float(xor_lane<2>(__float_as_uint(s[r])));
                s[r] += __uint_as_float(xor_lane<1>(__float_as_uint(s[r])));
                if ((l & 15) == 0 && col + r < N) put.columns(w >> 1, col + r, s[r]);
            }
        }
        return;
    } else if constexpr (k16 && !SPLIT) {
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F; j += 2) {
                const int row = r0 + i * 16 + (l & 15), col = c0 + j * 16 + (l >> 4) * 8;
                float v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) v[r] = acc[i][j + (r >> 2)][r & 3];
                if (row < M) put.eight(row, col, v);
            }
        return;
    }
    auto each = [&](auto&& f) {
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F; ++j)
#pragma unroll
                for (int r = 0; r < (k16 ? 4 : 16); ++r) {
                    if constexpr (k16)
                        f(r0 + i * 16 + (l & 15), c0 + (j >> 1) * 32 + (l >> 4) * 8 + (j & 1) * 4 + r, acc[i][j][r]);
                    else
                        f(r0 + i * 32 + 8 * (r >> 2) + 4 * (l >> 5) + (r & 3), c0 + j * 32 + (l & 31), acc[i][j][r]);
                }
    };
    if constexpr (SPLIT) {
        __syncthreads();
        constexpr int kPad = B + 1;
        float* part = reinterpret_cast<float*>(lds - w * 2 * kBuffer);
        each([&](int i, int j, float v) { part[(w * B + i) * kPad + j] = v; });
        __syncthreads();
        static_assert(kAnyThreads % B == 0);  // a thread has one column
        float s = 0.0f;
        for (int q = threadIdx.x; q < B * B; q += kAnyThreads) {
            const int i = q / B, j = q % B;
            float v = part[i * kPad + j];
#pragma unroll
            for (int o = 1; o < 4; ++o) v += part[(o * B + i) * kPad + j];
            if constexpr (HasCell<Put>::value) {
                put.cell(i, j, v, i < M && j < N);
            } else if (i < M && j < N) {
                if constexpr (HasColumns<Put>::value) s += put.value(i, j, v);
                else put.one(i, j, v);
            }
        }
        if constexpr (HasColumns<Put>::value) {
            static_assert(B == 32);
            s += __uint_as_float(xor_lane<32>(__float_as_uint(s)));
            if (l < B && l < N) put.columns(w, l, s);
        }
    } else {
        each([&](int i, int j, float v) {
            if (i < M && j < N) put.one(i, j, v);
        });
    }
}

}  // namespace lapsum
