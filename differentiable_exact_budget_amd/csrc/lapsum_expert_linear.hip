// The experts' products for every type, size and alignment, and dz with the
// bias gradient.
//
// k_product_any takes what the 16-bit tile kernels do not: fp32 rows, and
// 16-bit rows whose widths or addresses are off 16 bytes.  Operands go from
// memory through registers to LDS, 16 bytes a lane at any element's address
// (the hardware takes those), only the ends of rows element by element.  16-bit
// rows are multiplied by the 16-bit matrix instruction, fp32 rows by the fp32
// one (v_mfma_f32_32x32x2_f32), which bounds them.
//  - Many tiles: 128 x 128 a workgroup, 64 x 64 a wave; two LDS buffers of two
//    steps each, the next two steps' loads in flight while two are multiplied.
//  - Few tiles: 32 x 32 a workgroup, and its four waves split the sum, each on
//    its own in its own part of LDS; their results are added in wave order.
// 32768 x 2047 rows -> 4095 in bf16: y 1.07 ms (0.51 PFLOP/s), dx 0.91 (0.59),
// dW 0.82 (0.65), bound by the way through registers; 32768 x 2048 -> 4096 in
// fp32: y 4.76 ms (116 TFLOP/s), dx 4.72, dW 4.41, the matrix instruction's
// rate being 157.
#include <algorithm>

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

// One row's element (i, j) of a piece from its sum
template <class T, int FORM, int ACT>
LS_DEV void put_any(const Piece<T>& p, long long i, int j, float v) {
    if (FORM == kFormY && p.bias) v += to_f(p.bias[j]);
    if (FORM == kFormY && ACT != kActNone && p.z) p.z[i * p.ldc + j] = ZKeep<T>::template make<ACT>(v);
    p.c[i * p.ldc + j] = from_f<T>(act_of<ACT, T>(v));
}

// eight of a row's elements of 16 bits
template <class T, int FORM, int ACT>
LS_DEV void put_any8(const Piece<T>& p, long long i, int j, const float (&v)[8]) {
    if (j + 8 > p.N) {
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (j + r < p.N) put_any<T, FORM, ACT>(p, i, j + r, v[r]);
        return;
    }
    struct { T v[8]; } c, b = {};
    struct { typename ZKeep<T>::type v[8]; } z;
    if (FORM == kFormY && p.bias) b = __builtin_bit_cast(decltype(b), *reinterpret_cast<const Words*>(p.bias + j));
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const float x = FORM == kFormY ? v[r] + to_f(b.v[r]) : v[r];
        if (FORM == kFormY && ACT != kActNone) z.v[r] = ZKeep<T>::template make<ACT>(x);
        c.v[r] = from_f<T>(act_of<ACT, T>(x));
    }
    if (FORM == kFormY && ACT != kActNone && p.z)
        *reinterpret_cast<Words*>(p.z + i * p.ldc + j) = __builtin_bit_cast(u32x4, z);
    *reinterpret_cast<Words*>(p.c + i * p.ldc + j) = __builtin_bit_cast(u32x4, c);
}

// B x B of a piece from row i0 and column j0; SPLIT: the waves share the sum
template <class T, int FORM, int ACT, int B, bool SPLIT>
LS_DEV void any_tile(const Piece<T>& p, int i0, int j0, char* lds) {
    constexpr bool kA = FORM != kFormDw, kB = FORM == kFormY;
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
    const T* a = p.a + (kA ? (long long)i0 * p.lda : i0);
    const T* b = p.b + (kB ? (long long)j0 * p.ldb : j0);
    const int M = p.M - i0, N = p.N - j0;
    int k0 = 0, K = p.K;
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
    oa.place(a, p.lda, M, tid);
    ob.place(b, p.ldb, N, tid);
    auto get = [&](int k) {
        if (k + kDeep <= K && OpA::inside(p.lda, k, kDeep, p.K) && OpB::inside(p.ldb, k, kDeep, p.K)) {
#pragma unroll
            for (int h = 0; h < kAnySteps; ++h) {
                oa.fetch(ra[h], p.lda, k + h * kStepK);
                ob.fetch(rb[h], p.ldb, k + h * kStepK);
            }
            return;
        }
#pragma unroll
        for (int h = 0; h < kAnySteps; ++h) {
            OpA::get(ra[h], a, p.lda, M, k + h * kStepK, K, tid);
            OpB::get(rb[h], b, p.ldb, N, k + h * kStepK, K, tid);
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
    if constexpr (k16 && !SPLIT) {
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F; j += 2) {
                const int row = r0 + i * 16 + (l & 15), col = c0 + j * 16 + (l >> 4) * 8;
                float v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) v[r] = acc[i][j + (r >> 2)][r & 3];
                if (row < M) put_any8<T, FORM, ACT>(p, i0 + row, j0 + col, v);
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
        for (int q = threadIdx.x; q < B * B; q += kAnyThreads) {
            const int i = q / B, j = q % B;
            float v = part[i * kPad + j];
#pragma unroll
            for (int o = 1; o < 4; ++o) v += part[(o * B + i) * kPad + j];
            if (i < M && j < N) put_any<T, FORM, ACT>(p, i0 + i, j0 + j, v);
        }
    } else {
        each([&](int i, int j, float v) {
            if (i < M && j < N) put_any<T, FORM, ACT>(p, i0 + i, j0 + j, v);
        });
    }
}

template <class T, int FORM, int ACT, int B, bool SPLIT>
__global__ __launch_bounds__(kAnyThreads) void k_product_any(LinearArgs g, long long tiles, int cols) {
    __shared__ __align__(128) char lds[2 * any_steps(SPLIT) * 2 * B * 64 * (SPLIT ? 4 : 1)];
    for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
        // tiles past the last (their number is only bounded here) have no rows
        Place<T> at;
        if constexpr (FORM == kFormDw) {
            at = dw_place<T, B>(g, t, cols);
        } else {
            RowTiles<B> rows(g.off, g.E, g.P);
            at = row_place<T, FORM, B>(g, rows, t, cols);
        }
        if (at.rows > 0 && at.q < at.rows * cols)
            any_tile<T, FORM, ACT, B, SPLIT>(at.p, at.q / cols * B, at.q % cols * B, lds);
        __syncthreads();
    }
}

template <class T, int B, bool SPLIT>
static void launch_any(int form, const LinearArgs& g, hipStream_t st) {
    const int N = form == kFormY ? g.out : g.in;
    const long long cols = ceil_div(N, B);
    const long long tiles = cols * (form == kFormDw ? ceil_div(g.out, B) * g.E : max_row_tiles<B>(g.P, g.E));
    const dim3 grid(grid_of(tiles)), block(kAnyThreads);
    if (form == kFormDw)
        hipLaunchKernelGGL((k_product_any<T, kFormDw, kActNone, B, SPLIT>), grid, block, 0, st, g, tiles, (int)cols);
    else if (form == kFormDx)
        hipLaunchKernelGGL((k_product_any<T, kFormDx, kActNone, B, SPLIT>), grid, block, 0, st, g, tiles, (int)cols);
    else
        with_act(g.act, [&](auto av) {
            hipLaunchKernelGGL((k_product_any<T, kFormY, decltype(av)::value, B, SPLIT>), grid, block, 0, st, g, tiles,
                               (int)cols);
        });
}

void launch_expert_product(int form, int dtype, const LinearArgs& g, hipStream_t st) {
    const int N = form == kFormY ? g.out : g.in;
    if (N < 1 || (form == kFormDw ? g.out : g.P) < 1) return;
    if (expert_mfma_takes(form, dtype, g)) {
        launch_expert_mfma(form, dtype, g, st);
        return;
    }
    // 128 x 128 tiles where there are enough of them, for 16-bit rows every
    // second CU's, for fp32, whose tiles take eight times as long, more than
    // one for each CU (128 / 32 wide, us, tiles counted as below: bf16 y, 95
    // tiles 28.0 / 27.8, 120 tiles 29 / 29, 152 tiles 29 / 39, 280 tiles
    // 36 / 63; fp32 y, 152 tiles 88 / 68, 280 tiles 145 / 118; fp32 dW, 512
    // tiles 91 / 110, 896 tiles 59 / 77)
    const long long tiles = ceil_div(N, 128) * (form == kFormDw ? ceil_div(g.out, 128) * g.E : g.P / 128 + g.E / 2);
    with_dtype(dtype, [&](auto tv) {
        using T = decltype(tv);
        if (tiles >= (sizeof(T) == 2 ? 128 : 384)) launch_any<T, 128, false>(form, g, st);
        else launch_any<T, 32, true>(form, g, st);
    });
}

// ---------------------------------------------------------------------------
// dz = dy act'(z) and the column sums of dz per expert
// ---------------------------------------------------------------------------
// A workgroup takes kDzRows rows of one expert and 64 V columns, a wave a
// quarter of the rows; the waves' sums are added in wave order, one partial
// row per tile of rows, and k_dbias adds an expert's partials in their order.
//
// dz is rounded to the rows' type, once: the products that follow take their
// operands in it, and two 16-bit parts of dz would double them.  It is what
// 16-bit gradients lose beyond their own rounding: dx and dW of 32768 rows
// 2048 -> 4096 in bf16 with silu are 2.35e-3 off in the 2-norm, against 1.66e-3
// with dz in fp32, and 1.66e-3 off the formula that has this rounding; in fp16
// 3.0e-4 against 2.1e-4, a tenth of the excess by z's fp16.
//
// With V = 16 bytes a lane takes them at any element's address; where that
// leaves fewer than two workgroups for a CU it takes one element of 16 rows
// instead (16 bytes / one element, silu and the sums, us: 1026 rows of 1001 in
// fp32 11.7 / 7.8, 4096 of 1024 in bf16 18.2 / 9.9, 8192 of 1024 20.5 / 16.5,
// 16384 of 1024 25.2 / 24.1, 8192 of 2001 27.7 / 35.2, 32768 of 4095 164 /
// 222).  Memory bounds it: 32768 rows of 4096 in bf16, 805 MB: 149 us.
template <class T, int ACT, int V>
LS_DEV void dz_tile(const void* __restrict__ zp, const T* __restrict__ dy, const int32_t* __restrict__ off, int P,
                    int E, int N, T* __restrict__ dz, float* __restrict__ part, int ti, int tj,
                    float (*s)[64 * V]) {
    using Z = typename ZKeep<T>::type;
    const RowTile t = find_row_tile<kDzRows>(off, E, P, ti);
    if (t.lo >= t.hi || t.e >= E) return;
    const int l = lane_id(), w = threadIdx.x >> 6;
    // the lane's columns; at a row's end the last V of the row, which other
    // lanes have in part too: both write the same values
    const bool on = (long long)tj * (64 * V) + l * V < N;
    const long long c = min((long long)tj * (64 * V) + l * V, (long long)max(N - V, 0));
    float sum[V] = {};
    constexpr int U = V == 1 ? 16 : 4;  // rows whose loads are in flight at a time
    struct PT {
        T v[V];
    };
    struct __attribute__((packed, aligned(sizeof(T)))) Loose {  // at any element
        PT p;
    };
    struct PZ {
        Z v[V];
    };
    static_assert(V == 1 || (sizeof(PT) == 16 && sizeof(PZ) == 16));
    // whole: rows have V columns and more
    auto run = [&](auto whole) {
        // what is read once goes past the caches, which dz is to fill
        auto load = [&](auto& x, const auto* p) {
            if constexpr (decltype(whole)::value) {
                x = __builtin_bit_cast(std::decay_t<decltype(x)>,
                                       __builtin_nontemporal_load(reinterpret_cast<const Words*>(p)));
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) x.v[i] = p[min(i, N - 1)];
            }
        };
        for (int r0 = t.lo + w; r0 < t.hi; r0 += 4 * U) {
            PT g[U];
            PZ z[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const long long at = (long long)min(r0 + 4 * u, t.hi - 1) * N + c;
                load(g[u], dy + at);
                if (ACT != kActNone) load(z[u], (const Z*)zp + at);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + 4 * u;
                if (r >= t.hi) break;
                PT o;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float d = to_f(g[u].v[i]);
                    if (ACT != kActNone) {
                        const float zi = ZKeep<T>::value(z[u].v[i]);
                        // relu drops dy where its slope is 0, inf and NaN too
                        d = ACT == kActRelu ? (zi > 0.0f ? d : 0.0f) : d * slope_of<ACT, T>(zi);
                        o.v[i] = from_f<T>(d);
                    }
                    sum[i] += d;
                }
                if (ACT == kActNone) continue;
                T* to = dz + (long long)r * N + c;
                if constexpr (decltype(whole)::value) {
                    reinterpret_cast<Loose*>(to)->p = o;
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (i < N) to[i] = o.v[i];
                }
            }
        }
    };
    if (on) {
        if (V > 1 && N >= V) run(std::bool_constant<(V > 1)>{});
        else run(std::false_type{});
    }
    if (!part) return;
#pragma unroll
    for (int i = 0; i < V; ++i) s[w][i * 64 + l] = sum[i];
    __syncthreads();
    if (w != 0 || !on) return;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (c + i < N)
            part[(long long)ti * N + c + i] = (s[0][i * 64 + l] + s[1][i * 64 + l]) +
                                                  (s[2][i * 64 + l] + s[3][i * 64 + l]);
}

template <class T, int ACT, int V>
__global__ __launch_bounds__(256) void k_dz(const void* __restrict__ zp, const T* __restrict__ dy,
                                            const int32_t* __restrict__ off, int P, int E, int N, T* __restrict__ dz,
                                            float* __restrict__ part, long long tiles, int cols) {
    __shared__ float s[4][64 * V];
    for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
        dz_tile<T, ACT, V>(zp, dy, off, P, E, N, dz, part, (int)(t / cols), (int)(t % cols), s);
        __syncthreads();
    }
}

// An expert's partial sums, 64 columns a workgroup: a wave adds every fourth
// tile's, eight loads in flight, and the waves' sums are added in wave order
// (4096 columns of 8 experts, 520 partial rows: 5.5 us).
//
// `tiles` rows of partial sums there are.  Offsets that a sort made need at
// most so many; of offsets that run back, experts' rows overlap and would count
// more, so an expert's first row and its number are held to them.
template <class T>
__global__ __launch_bounds__(256) void k_dbias(const float* __restrict__ part, const int32_t* __restrict__ off, int P,
                                               int E, int N, int tiles, long long c0, T* __restrict__ dbias) {
    __shared__ float s[4][64];
    const int e = blockIdx.y, l = lane_id(), w = uniform(threadIdx.x >> 6);
    // the expert's first tile of rows: those of the experts before it
    int first = 0;
    for (int i = l; i < e; i += 64)
        first += (max(row_at(off, i + 1, P) - row_at(off, i, P), 0) + kDzRows - 1) / kDzRows;
    // (a lane adds up at most 16 experts' tiles, below 2^29, and 64 lanes of at
    // most `tiles` stay below 2^32)
    const uint32_t before = wave_inclusive_scan((uint32_t)min(first, tiles));
    first = (int)min((uint32_t)__builtin_amdgcn_readlane((int)before, 63), (uint32_t)tiles);
    const int n = min((max(row_at(off, e + 1, P) - row_at(off, e, P), 0) + kDzRows - 1) / kDzRows, tiles - first);
    const long long c = c0 + (long long)blockIdx.x * 64 + l;
    float sum = 0.0f;
    if (c < N) {
        const float* p = part + (long long)first * N + c;
#pragma unroll 8
        for (int i = w; i < n; i += 4) sum += p[(long long)i * N];
    }
    s[w][l] = sum;
    __syncthreads();
    if (w == 0 && c < N) dbias[(long long)e * N + c] = from_f<T>((s[0][l] + s[1][l]) + (s[2][l] + s[3][l]));
}

void launch_expert_dz(const void* z, const void* dy, int dtype, int act, const int32_t* off, int P, int E, int out,
                      void* dz, float* part, hipStream_t st) {
    if (P < 1 || out < 1 || (act == kActNone && !part)) return;
    with_dtype(dtype, [&](auto tv) {
        using T = decltype(tv);
        with_act(act, [&](auto av) {
            constexpr int A = decltype(av)::value;
            auto launch = [&](auto vv) {
                constexpr int V = decltype(vv)::value;
                const int cols = (int)ceil_div(out, 64 * V);
                const long long tiles = max_row_tiles<kDzRows>(P, E) * cols;
                hipLaunchKernelGGL((k_dz<T, A, V>), dim3(grid_of(tiles)), dim3(256), 0, st, z, (const T*)dy, off, P,
                                   E, out, (T*)dz, part, tiles, cols);
            };
            constexpr int W = 16 / (int)sizeof(T);
            if (max_row_tiles<kDzRows>(P, E) * ceil_div(out, 64 * W) >= 512) launch(std::integral_constant<int, W>{});
            else launch(std::integral_constant<int, 1>{});
        });
    });
}

void launch_expert_dbias(const float* part, int dtype, const int32_t* off, int P, int E, int out, void* dbias,
                         hipStream_t st) {
    if (out < 1) return;
    with_dtype(dtype, [&](auto tv) {
        using T = decltype(tv);
        // one launch up to a grid's columns, 262144 of 1024 experts (walking
        // on by the grid in the kernel: 0.2 us more for every call)
        const long long most = kGridMax / E * 64;
        for (long long c0 = 0; c0 < out; c0 += most)
            hipLaunchKernelGGL(k_dbias<T>, dim3((unsigned)ceil_div(std::min(out - c0, most), 64), (unsigned)E),
                               dim3(256), 0, st, part, off, P, E, out, (int)max_row_tiles<kDzRows>(P, E), c0,
                               (T*)dbias);
    });
}

}  // namespace lapsum
