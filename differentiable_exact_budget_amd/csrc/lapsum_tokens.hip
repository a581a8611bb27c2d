// Token rows to their experts' places and back.
//
// Every kernel gives a token, or a stretch of its columns, to one wave: it
// reads the token's row (or sums into it) and touches the row of each of its
// slots, so a token's row is read from memory once however many slots it has,
// and every sum runs in the order of the slots.  They are copies with a
// little arithmetic: HBM bounds them where there are many tokens, and the
// latency of one load behind another where there are few.  So a wave keeps
// several 16-byte loads in flight (U stretches of 64 lanes), and with few
// tokens a row is spread over many waves instead (U = 1).
//
// 16384 tokens of 2048 in bf16: dispatch to 2 slots 34 us and its gradient
// 35 us for 201 MB each, 5.9 TB/s; combine of 4 slots with a residual 67 us for
// 389 MB, 5.8 TB/s; its gradient 96 to 120 us for 590 MB, 4.9 to 6.1 TB/s.
//
// Rows need not start on 16 bytes: the hardware takes 16-byte loads and stores
// at any element's address, and only a row's last elements go one by one.
//
// A slot's place is read from its lane (readlane) only where the whole wave
// is active: loops over a row's columns run to the wave's end and mask their
// loads and stores instead.
#include <initializer_list>

#include "lapsum_rows.h"

namespace lapsum {

constexpr int kTokWaves = 4;
constexpr int kTokThreads = kTokWaves * 64;

// positions of a token's slots, slot j in lane j; -1 for empty ones
LS_DEV int slot_place(const int32_t* __restrict__ place, long long t, int m, long long P) {
    const int l = lane_id();
    const int pos = l < m ? place[t * m + l] : -1;
    return (unsigned long long)(long long)pos < (unsigned long long)P ? pos : -1;
}

// zeros in the columns from c of the rows past offsets[E], dealt out over the
// tokens
template <class T, int U>
LS_DEV void zero_unused(T* __restrict__ rows, const int32_t* __restrict__ off, int E, long long P, long long D,
                        long long t, long long T_, long long c) {
    const long long used = min(max((long long)off[E], 0ll), P);
    for (long long r = used + t; r < P; r += T_)
#pragma unroll
        for (int u = 0; u < U; ++u) st<T>(rows + r * D, c + u * 64 * Pack<T>::V, D, Pack<T>{});
}

// A wave's work: token t, columns from c0.  `stretches` = ceil(D / (64 V U)).
struct Task {
    long long t, c0;
};
template <class T, int U>
LS_DEV Task task_of(long long i, int stretches) {
    const long long t = i / stretches;
    return {t, (i - t * stretches) * (64 * Pack<T>::V * U)};
}

template <class T, int U>
__global__ __launch_bounds__(kTokThreads) void k_dispatch(const T* __restrict__ x, long long T_, int m, long long D,
                                                           int E, int stretches, const int32_t* __restrict__ off,
                                                           const int32_t* __restrict__ place, T* __restrict__ xs) {
    constexpr int V = Pack<T>::V;
    const long long P = T_ * m;
    for (long long i = (long long)blockIdx.x * kTokWaves + uniform(threadIdx.x >> 6); i < T_ * stretches;
         i += (long long)gridDim.x * kTokWaves) {
        const Task a = task_of<T, U>(i, stretches);
        const int pos = slot_place(place, a.t, m, P);
        const long long c = a.c0 + lane_id() * V;
        Pack<T> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = ld<false>(x + a.t * D, c + u * 64 * V, D);
        for (int j = 0; j < m; ++j) {
            const int p = __builtin_amdgcn_readlane(pos, j);
            if (p < 0) continue;
#pragma unroll
            for (int u = 0; u < U; ++u) st<T>(xs + (long long)p * D, c + u * 64 * V, D, v[u]);
        }
        zero_unused<T, U>(xs, off, E, P, D, a.t, T_, c);
    }
}

// out = residual + sum of w rows (weights null: 1)
template <class T, int U>
__global__ __launch_bounds__(kTokThreads) void k_combine(const T* __restrict__ ys, const float* __restrict__ w,
                                                          const T* __restrict__ residual, long long T_, int m,
                                                          long long D, int stretches,
                                                          const int32_t* __restrict__ place, T* __restrict__ out) {
    constexpr int V = Pack<T>::V;
    const int l = lane_id();
    for (long long i = (long long)blockIdx.x * kTokWaves + uniform(threadIdx.x >> 6); i < T_ * stretches;
         i += (long long)gridDim.x * kTokWaves) {
        const Task a = task_of<T, U>(i, stretches);
        const int pos = slot_place(place, a.t, m, T_ * m);
        const float wt = w && l < m ? w[a.t * m + l] : 1.0f;
        const long long c = a.c0 + l * V;
        float acc[U][V] = {};
        if (residual) {
            Pack<T> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = ld<true>(residual + a.t * D, c + u * 64 * V, D);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int q = 0; q < V; ++q) acc[u][q] = to_f(v[u].v[q]);
        }
        // two slots' rows in flight
        for (int j = 0; j < m; j += 2) {
            const int p0 = __builtin_amdgcn_readlane(pos, j), p1 = j + 1 < m ? __builtin_amdgcn_readlane(pos, j + 1) : -1;
            const float w0 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wt), j));
            const float w1 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wt), min(j + 1, m - 1)));
            Pack<T> v0[U] = {}, v1[U] = {};
            if (p0 >= 0)
#pragma unroll
                for (int u = 0; u < U; ++u) v0[u] = ld<true>(ys + (long long)p0 * D, c + u * 64 * V, D);
            if (p1 >= 0)
#pragma unroll
                for (int u = 0; u < U; ++u) v1[u] = ld<true>(ys + (long long)p1 * D, c + u * 64 * V, D);
            if (p0 >= 0)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int q = 0; q < V; ++q) acc[u][q] = fmaf(w0, to_f(v0[u].v[q]), acc[u][q]);
            if (p1 >= 0)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int q = 0; q < V; ++q) acc[u][q] = fmaf(w1, to_f(v1[u].v[q]), acc[u][q]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Pack<T> o;
#pragma unroll
            for (int q = 0; q < V; ++q) o.v[q] = from_f<T>(acc[u][q]);
            st<T>(out + a.t * D, c + u * 64 * V, D, o);
        }
    }
}

// A wave takes a whole token (dw is a sum over the row), U stretches at a time,
// whatever the number of tokens: with few, the latencies of its slots one behind
// another bound it (4 or 64 tokens of 4096 x 8 slots in bf16: 17 us a call, dys
// alone 9 to 10, where 64 tokens' bytes take 2; 1024 tokens 31, their bytes 29).
template <class T, int U>
__global__ __launch_bounds__(kTokThreads) void k_combine_vjp(const T* __restrict__ ys, const float* __restrict__ w,
                                                              const T* __restrict__ dout, long long T_, int m,
                                                              long long D, int E, const int32_t* __restrict__ off,
                                                              const int32_t* __restrict__ place, T* __restrict__ dys,
                                                              float* __restrict__ dw) {
    constexpr int V = Pack<T>::V;
    const int l = lane_id();
    const long long P = T_ * m;
    for (long long t = (long long)blockIdx.x * kTokWaves + uniform(threadIdx.x >> 6); t < T_;
         t += (long long)gridDim.x * kTokWaves) {
        const int pos = slot_place(place, t, m, P);
        const float wt = l < m ? w[t * m + l] : 0.0f;
        float mine = 0.0f;  // slot l's dw
        for (long long c0 = 0; c0 < D; c0 += 64 * V * U) {
            const long long c = c0 + l * V;
            Pack<T> g[U];
#pragma unroll
            for (int u = 0; u < U; ++u) g[u] = ld<true>(dout + t * D, c + u * 64 * V, D);
            for (int j = 0; j < m; ++j) {
                const int p = __builtin_amdgcn_readlane(pos, j);
                if (p < 0) continue;
                const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wt), j));
                Pack<T> y[U];
                if (dw)
#pragma unroll
                    for (int u = 0; u < U; ++u) y[u] = ld<true>(ys + (long long)p * D, c + u * 64 * V, D);
                if (dys)
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        Pack<T> o;
#pragma unroll
                        for (int q = 0; q < V; ++q) o.v[q] = from_f<T>(wj * to_f(g[u].v[q]));
                        st<T>(dys + (long long)p * D, c + u * 64 * V, D, o);
                    }
                if (dw) {
                    float dot = 0.0f;
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int q = 0; q < V; ++q) dot = fmaf(to_f(g[u].v[q]), to_f(y[u].v[q]), dot);
                    dot = wave_sum_f32(dot);
                    mine += l == j ? dot : 0.0f;
                }
            }
            if (dys) zero_unused<T, U>(dys, off, E, P, D, t, T_, c);
        }
        if (dw && l < m) dw[t * m + l] = mine;
    }
}

// Calls f with an element type and U.  Several stretches a wave where that
// still leaves enough waves for the chip's 1024 SIMDs, else one (combine's
// kernel, 4 tokens of 4096 x 8 slots in bf16: 17.3 us with a wave a token, 4.2
// with U = 1; 65536 x 4 rows at U = 1 and 4 within 2%).
template <class F>
static void with_stretches(int dtype, long long T, long long D, F&& f) {
    with_dtype(dtype, [&](auto v) {
        using S = decltype(v);
        constexpr int kLanes = 64 * Pack<S>::V;
        if (T * ceil_div(D, 4 * kLanes) >= 4096) f(v, std::integral_constant<int, 4>{}, (int)ceil_div(D, 4 * kLanes));
        else f(v, std::integral_constant<int, 1>{}, (int)ceil_div(D, kLanes));
    });
}
static dim3 wave_grid(long long waves) { return dim3(grid_of(ceil_div(waves, kTokWaves))); }

void launch_dispatch(const void* x, int dtype, long long T, int m, long long D, int E, const int32_t* offsets,
                     const int32_t* place, void* xs, hipStream_t st) {
    if (T < 1 || D < 1) return;
    with_stretches(dtype, T, D, [&](auto tv, auto uv, int n) {
        using S = decltype(tv);
        constexpr int U = decltype(uv)::value;
        hipLaunchKernelGGL((k_dispatch<S, U>), wave_grid(T * n), dim3(kTokThreads), 0, st, (const S*)x, T, m, D, E, n,
                           offsets, place, (S*)xs);
    });
}

void launch_dispatch_vjp(const void* dxs, int dtype, long long T, int m, long long D, const int32_t* place, void* dx,
                         hipStream_t st) {
    launch_combine(dxs, nullptr, nullptr, dtype, T, m, D, place, dx, st);
}

void launch_combine(const void* ys, const float* w, const void* residual, int dtype, long long T, int m, long long D,
                    const int32_t* place, void* out, hipStream_t st) {
    if (T < 1 || D < 1) return;
    with_stretches(dtype, T, D, [&](auto tv, auto uv, int n) {
        using S = decltype(tv);
        constexpr int U = decltype(uv)::value;
        hipLaunchKernelGGL((k_combine<S, U>), wave_grid(T * n), dim3(kTokThreads), 0, st, (const S*)ys, w,
                           (const S*)residual, T, m, D, n, place, (S*)out);
    });
}

void launch_combine_vjp(const void* ys, const float* w, const void* dout, int dtype, long long T, int m, long long D,
                        int E, const int32_t* offsets, const int32_t* place, void* dys, float* dw, hipStream_t st) {
    if (T < 1) return;
    with_dtype(dtype, [&](auto tv) {
        using S = decltype(tv);
        hipLaunchKernelGGL((k_combine_vjp<S, 4>), wave_grid(T), dim3(kTokThreads), 0, st, (const S*)ys, w,
                           (const S*)dout, T, m, D, E, offsets, place, (S*)dys, dw);
    });
}

}  // namespace lapsum
