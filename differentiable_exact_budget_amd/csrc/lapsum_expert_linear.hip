// The experts' products: every expert's weights against its own rows, forward
// and both gradients, in matrix instructions.
//
// k_product_any takes every type, size and alignment: a workgroup forms a
// 64 x 64 tile of one expert's result, staging 32 steps of the sum at a time
// in LDS as fp32 and multiplying with the fp32 matrix instruction
// (v_mfma_f32_32x32x2_f32), so 16-bit rows lose nothing on the way.
#include "lapsum_expert_ops.h"

namespace lapsum {

constexpr int kAnyTile = 64;
constexpr int kAnyK = 32;
constexpr int kAnyThreads = 256;
constexpr int kAnyPad = kAnyTile + 4;

typedef float f32x16 __attribute__((ext_vector_type(16)));

// One tile of the operand X(i, k), i < n, k < K, into s[k][i]; zeros outside.
// KFAST: k is the contiguous index (X[i * ld + k]), else i (X[k * ld + i]).
template <class T, bool KFAST>
struct AnyLoad {
    static constexpr int kN = kAnyTile * kAnyK / kAnyThreads;
    float r[kN];
    LS_DEV void get(const T* __restrict__ x, long long ld, long long i0, long long n, long long k0, long long K) {
#pragma unroll
        for (int q = 0; q < kN; ++q) {
            const int at = q * kAnyThreads + threadIdx.x;
            const long long i = i0 + (KFAST ? at / kAnyK : at % kAnyTile);
            const long long k = k0 + (KFAST ? at % kAnyK : at / kAnyTile);
            r[q] = i < n && k < K ? to_f(x[KFAST ? i * ld + k : k * ld + i]) : 0.0f;
        }
    }
    LS_DEV void put(float (*s)[kAnyPad]) const {
#pragma unroll
        for (int q = 0; q < kN; ++q) {
            const int at = q * kAnyThreads + threadIdx.x;
            s[KFAST ? at % kAnyK : at / kAnyTile][KFAST ? at / kAnyK : at % kAnyTile] = r[q];
        }
    }
};

// tile `ti` of the rows (or of expert and output), `tj` of the columns
template <class T, int FORM, int ACT>
LS_DEV void product_any(const LinearArgs& g, int ti, int tj, float (*sa)[kAnyPad], float (*sb)[kAnyPad]) {
    using Z = typename ZKeep<T>::type;
    // this workgroup's part of the result: rows i0.. of M (from C row c0),
    // columns j0.. of N; the sum runs over K
    const long long j0 = (long long)tj * kAnyTile;
    long long M, N, K, i0, lda, ldb;
    const T *a = (const T*)g.a, *b = (const T*)g.b;
    T* c = (T*)g.c;
    const T* bias = nullptr;
    Z* z = nullptr;
    if (FORM == kFormDw) {
        const int to = (g.out + kAnyTile - 1) / kAnyTile;
        const int e = ti / to;
        const int lo = row_at(g.off, e, g.P), hi = max(row_at(g.off, e + 1, g.P), lo);
        i0 = (long long)(ti % to) * kAnyTile;
        M = g.out, N = g.in, K = hi - lo, lda = g.out, ldb = g.in;
        a += lo * lda;
        b += lo * ldb;
        c += (long long)e * g.out * g.in;
    } else {
        const RowTile t = find_row_tile<kAnyTile>(g.off, g.E, g.P, ti);
        if (t.lo >= t.hi) return;
        const bool unused = t.e >= g.E;
        i0 = 0, M = t.hi - t.lo;
        K = FORM == kFormY ? g.in : g.out;
        N = FORM == kFormY ? g.out : g.in;
        lda = K, ldb = g.in;
        a += t.lo * lda;
        c += t.lo * N;
        if (unused) {
            K = 0;
        } else {
            b += (long long)t.e * g.out * g.in;
            if (FORM == kFormY && g.bias) bias = (const T*)g.bias + (long long)t.e * g.out;
            if (FORM == kFormY && g.z) z = (Z*)g.z + t.lo * N;
        }
    }
    const int l = lane_id(), w = threadIdx.x >> 6;
    const int wi = (w >> 1) * 32, wj = (w & 1) * 32;
    f32x16 acc = {};
    AnyLoad<T, FORM != kFormDw> la;
    AnyLoad<T, FORM == kFormY> lb;
    la.get(a, lda, i0, M, 0, K);
    lb.get(b, ldb, j0, N, 0, K);
    for (long long k0 = 0; k0 < K; k0 += kAnyK) {
        la.put(sa);
        lb.put(sb);
        __syncthreads();
        if (k0 + kAnyK < K) {
            la.get(a, lda, i0, M, k0 + kAnyK, K);
            lb.get(b, ldb, j0, N, k0 + kAnyK, K);
        }
#pragma unroll
        for (int k = 0; k < kAnyK; k += 2)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(sa[k + (l >> 5)][wi + (l & 31)],
                                                       sb[k + (l >> 5)][wj + (l & 31)], acc, 0, 0, 0);
        __syncthreads();
    }
    // lane l holds column l % 32, rows 8 (r / 4) + 4 (l / 32) + r % 4
    const long long j = j0 + wj + (l & 31);
    if (j >= N) return;
    const float bj = bias ? to_f(bias[j]) : 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const long long i = i0 + wi + 8 * (r >> 2) + 4 * (l >> 5) + (r & 3);
        if (i >= M) continue;
        const float v = acc[r] + bj;
        if (z) z[i * N + j] = ZKeep<T>::template make<ACT>(v);
        c[i * N + j] = from_f<T>(act_of<ACT, T>(v));
    }
}

template <class T, int FORM, int ACT>
__global__ __launch_bounds__(kAnyThreads) void k_product_any(LinearArgs g, long long tiles, int cols) {
    __shared__ float sa[kAnyK][kAnyPad], sb[kAnyK][kAnyPad];
    for (long long t = blockIdx.x; t < tiles; t += gridDim.x)
        product_any<T, FORM, ACT>(g, (int)(t / cols), (int)(t % cols), sa, sb);
}

void launch_expert_product(int form, int dtype, const LinearArgs& g, hipStream_t st) {
    const int N = form == kFormY ? g.out : g.in;
    if (N < 1 || (form == kFormDw ? g.out : g.P) < 1) return;
    if (expert_mfma_takes(form, dtype, g)) {
        launch_expert_mfma(form, dtype, g, st);
        return;
    }
    const long long cols = ceil_div(N, kAnyTile);
    const long long tiles =
        cols * (form == kFormDw ? ceil_div(g.out, kAnyTile) * g.E : max_row_tiles<kAnyTile>(g.P, g.E));
    const dim3 grid(grid_of(tiles)), block(kAnyThreads);
    with_dtype(dtype, [&](auto tv) {
        using T = decltype(tv);
        if (form == kFormDw)
            hipLaunchKernelGGL((k_product_any<T, kFormDw, kActNone>), grid, block, 0, st, g, tiles, (int)cols);
        else if (form == kFormDx)
            hipLaunchKernelGGL((k_product_any<T, kFormDx, kActNone>), grid, block, 0, st, g, tiles, (int)cols);
        else
            with_act(g.act, [&](auto av) {
                hipLaunchKernelGGL((k_product_any<T, kFormY, decltype(av)::value>), grid, block, 0, st, g, tiles,
                                   (int)cols);
            });
    });
}

// ---------------------------------------------------------------------------
// dz = dy act'(z) and the column sums of dz per expert
// ---------------------------------------------------------------------------
// A workgroup takes kDzRows rows of one expert and 64 V columns, a wave a
// quarter of the rows; the waves' sums are added in wave order, one partial
// row per tile of rows, and k_dbias adds an expert's partials in their order.
template <class R>
LS_DEV R once(const void* p) {
    if constexpr (sizeof(R) == 16) {
        typedef uint32_t Words __attribute__((ext_vector_type(4)));
        return __builtin_bit_cast(R, __builtin_nontemporal_load(reinterpret_cast<const Words*>(p)));
    } else {
        return *reinterpret_cast<const R*>(p);
    }
}

template <class T, int ACT, int V>
LS_DEV void dz_tile(const void* __restrict__ zp, const T* __restrict__ dy, const int32_t* __restrict__ off, int P,
                    int E, int N, T* __restrict__ dz, float* __restrict__ part, int ti, int tj, float (*s)[64 * V]) {
    using Z = typename ZKeep<T>::type;
    const RowTile t = find_row_tile<kDzRows>(off, E, P, ti);
    if (t.lo >= t.hi || t.e >= E) return;
    const int l = lane_id(), w = threadIdx.x >> 6;
    const long long c = (long long)tj * (64 * V) + l * V;
    float sum[V] = {};
    // four rows' loads are in flight at a time
    constexpr int U = 4;
    struct __attribute__((aligned(sizeof(T) * V))) PT {
        T v[V];
    };
    struct __attribute__((aligned(sizeof(Z) * V))) PZ {
        Z v[V];
    };
    if (c < N) {
        for (int r0 = t.lo + w; r0 < t.hi; r0 += 4 * U) {
            PT g[U];
            PZ z[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const long long at = (long long)min(r0 + 4 * u, t.hi - 1) * N + c;
                // read once: past the caches, which dz is to fill
                g[u] = once<PT>(dy + at);
                if (ACT != kActNone) z[u] = once<PZ>((const Z*)zp + at);
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
                if (ACT != kActNone) *reinterpret_cast<PT*>(dz + (long long)r * N + c) = o;
            }
        }
    }
    if (!part) return;
#pragma unroll
    for (int i = 0; i < V; ++i) s[w][i * 64 + l] = sum[i];
    __syncthreads();
    if (w != 0 || c >= N) return;
#pragma unroll
    for (int i = 0; i < V; ++i)
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
// tile's, eight loads in flight, and the waves' sums are added in wave order.
template <class T>
__global__ __launch_bounds__(256) void k_dbias(const float* __restrict__ part, const int32_t* __restrict__ off, int P,
                                               int E, int N, T* __restrict__ dbias) {
    __shared__ float s[4][64];
    const int e = blockIdx.y, l = lane_id(), w = uniform(threadIdx.x >> 6);
    // the expert's first tile of rows: those of the experts before it
    int first = 0;
    for (int i = l; i < e; i += 64)
        first += (max(row_at(off, i + 1, P) - row_at(off, i, P), 0) + kDzRows - 1) / kDzRows;
    first = __builtin_amdgcn_readlane((int)wave_inclusive_scan((uint32_t)first), 63);
    const int n = (max(row_at(off, e + 1, P) - row_at(off, e, P), 0) + kDzRows - 1) / kDzRows;
    const long long c = (long long)blockIdx.x * 64 + l;
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
            constexpr int W = 16 / (int)sizeof(T);
            const bool wide = out % W == 0 && aligned16(z) && aligned16(dy) && aligned16(dz);
            const int cols = (int)ceil_div(out, wide ? 64 * W : 64);
            const long long tiles = max_row_tiles<kDzRows>(P, E) * cols;
            if (wide)
                hipLaunchKernelGGL((k_dz<T, A, W>), dim3(grid_of(tiles)), dim3(256), 0, st, z, (const T*)dy, off, P, E,
                                   out, (T*)dz, part, tiles, cols);
            else
                hipLaunchKernelGGL((k_dz<T, A, 1>), dim3(grid_of(tiles)), dim3(256), 0, st, z, (const T*)dy, off, P, E,
                                   out, (T*)dz, part, tiles, cols);
        });
    });
}

void launch_expert_dbias(const float* part, int dtype, const int32_t* off, int P, int E, int out, void* dbias,
                         hipStream_t st) {
    if (out < 1) return;
    with_dtype(dtype, [&](auto tv) {
        using T = decltype(tv);
        hipLaunchKernelGGL(k_dbias<T>, dim3((unsigned)ceil_div(out, 64), (unsigned)E), dim3(256), 0, st, part, off, P,
                           E, out, (T*)dbias);
    });
}

}  // namespace lapsum
