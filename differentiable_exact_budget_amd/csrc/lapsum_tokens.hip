// Token rows to their experts' places and back.
//
// Every kernel gives a token to one wave: it reads the token's row (or sums
// into it) and touches the row of each of its slots, so a token's row is read
// from memory once however many slots it has, and every sum runs in the order
// of the slots.  They are copies with a little arithmetic: HBM bounds them.
//
// A slot's place is read from its lane (readlane) only where the whole wave
// is active: loops over a row's columns run to the wave's end and mask their
// loads and stores instead.
#include <initializer_list>

#include "lapsum_expert_ops.h"

namespace lapsum {

constexpr int kTokWaves = 4;
constexpr int kTokThreads = kTokWaves * 64;

// V elements of a row in one load
template <class T, int V>
struct __attribute__((aligned(sizeof(T) * V))) Pack {
    T v[V];
};
template <class T, int V>
LS_DEV Pack<T, V> ld(const T* p) {
    return *reinterpret_cast<const Pack<T, V>*>(p);
}
template <class T, int V>
LS_DEV void st(T* p, const Pack<T, V>& x) {
    *reinterpret_cast<Pack<T, V>*>(p) = x;
}

// positions of a token's slots, slot j in lane j; -1 for empty ones
LS_DEV int slot_place(const int32_t* __restrict__ place, long long t, int m, long long P) {
    const int l = lane_id();
    const int pos = l < m ? place[t * m + l] : -1;
    return (unsigned long long)(long long)pos < (unsigned long long)P ? pos : -1;
}

// zeros in the rows past offsets[E], dealt out over the tokens' waves
template <class T, int V>
LS_DEV void zero_unused(T* __restrict__ rows, const int32_t* __restrict__ off, int E, long long P, long long D,
                        long long t, long long T_) {
    const long long used = min(max((long long)off[E], 0ll), P);
    Pack<T, V> z{};
    for (long long r = used + t; r < P; r += T_)
        for (long long c = (long long)lane_id() * V; c < D; c += 64 * V) st<T, V>(rows + r * D + c, z);
}

template <class T, int V>
__global__ __launch_bounds__(kTokThreads) void k_dispatch(const T* __restrict__ x, long long T_, int m, long long D,
                                                           int E, const int32_t* __restrict__ off,
                                                           const int32_t* __restrict__ place, T* __restrict__ xs) {
    for (long long t = (long long)blockIdx.x * kTokWaves + uniform(threadIdx.x >> 6); t < T_;
         t += (long long)gridDim.x * kTokWaves) {
        const long long P = T_ * m;
        const int pos = slot_place(place, t, m, P);
        for (long long c0 = 0; c0 < D; c0 += 64 * V) {
            const long long c = c0 + lane_id() * V;
            const bool on = c < D;
            Pack<T, V> v{};
            if (on) v = ld<T, V>(x + t * D + c);
            for (int j = 0; j < m; ++j) {
                const int p = __builtin_amdgcn_readlane(pos, j);
                if (p >= 0 && on) st<T, V>(xs + (long long)p * D + c, v);
            }
        }
        zero_unused<T, V>(xs, off, E, P, D, t, T_);
    }
}

// out = residual + sum of w rows (weights null: 1)
template <class T, int V>
__global__ __launch_bounds__(kTokThreads) void k_combine(const T* __restrict__ ys, const float* __restrict__ w,
                                                          const T* __restrict__ residual, long long T_, int m,
                                                          long long D, const int32_t* __restrict__ place,
                                                          T* __restrict__ out) {
    for (long long t = (long long)blockIdx.x * kTokWaves + uniform(threadIdx.x >> 6); t < T_;
         t += (long long)gridDim.x * kTokWaves) {
        const int l = lane_id();
        const int pos = slot_place(place, t, m, T_ * m);
        const float wt = w && l < m ? w[t * m + l] : 1.0f;
        for (long long c0 = 0; c0 < D; c0 += 64 * V) {
            const long long c = c0 + l * V;
            const bool on = c < D;
            float acc[V] = {};
            if (residual && on) {
                const Pack<T, V> v = ld<T, V>(residual + t * D + c);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = to_f(v.v[i]);
            }
            for (int j = 0; j < m; ++j) {
                const int p = __builtin_amdgcn_readlane(pos, j);
                if (p < 0) continue;
                const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wt), j));
                Pack<T, V> v{};
                if (on) v = ld<T, V>(ys + (long long)p * D + c);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = fmaf(wj, to_f(v.v[i]), acc[i]);
            }
            Pack<T, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) o.v[i] = from_f<T>(acc[i]);
            if (on) st<T, V>(out + t * D + c, o);
        }
    }
}

template <class T, int V>
__global__ __launch_bounds__(kTokThreads) void k_combine_vjp(const T* __restrict__ ys, const float* __restrict__ w,
                                                              const T* __restrict__ dout, long long T_, int m,
                                                              long long D, int E, const int32_t* __restrict__ off,
                                                              const int32_t* __restrict__ place, T* __restrict__ dys,
                                                              float* __restrict__ dw) {
    for (long long t = (long long)blockIdx.x * kTokWaves + uniform(threadIdx.x >> 6); t < T_;
         t += (long long)gridDim.x * kTokWaves) {
        const int l = lane_id();
        const long long P = T_ * m;
        const int pos = slot_place(place, t, m, P);
        const float wt = l < m ? w[t * m + l] : 0.0f;
        float mine = 0.0f;
        for (int j = 0; j < m; ++j) {
            const int p = __builtin_amdgcn_readlane(pos, j);
            if (p < 0) continue;
            const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wt), j));
            float dot = 0.0f;
            for (long long c = (long long)l * V; c < D; c += 64 * V) {
                const Pack<T, V> g = ld<T, V>(dout + t * D + c);
                if (dw) {
                    const Pack<T, V> y = ld<T, V>(ys + (long long)p * D + c);
#pragma unroll
                    for (int i = 0; i < V; ++i) dot = fmaf(to_f(g.v[i]), to_f(y.v[i]), dot);
                }
                if (dys) {
                    Pack<T, V> o;
#pragma unroll
                    for (int i = 0; i < V; ++i) o.v[i] = from_f<T>(wj * to_f(g.v[i]));
                    st<T, V>(dys + (long long)p * D + c, o);
                }
            }
            if (dw) {
                dot = wave_sum_f32(dot);
                if (l == j) mine = dot;
            }
        }
        if (dw && l < m) dw[t * m + l] = mine;
        if (dys) zero_unused<T, V>(dys, off, E, P, D, t, T_);
    }
}

// calls f with an element type and the elements of a 16-byte load when every
// row starts on 16 bytes, else one element at a time
template <class F>
static void with_pack(int dtype, long long D, std::initializer_list<const void*> ptrs, F&& f) {
    bool wide = D * (long long)dtype_size(dtype) % 16 == 0;
    for (const void* p : ptrs) wide = wide && aligned16(p);
    with_dtype(dtype, [&](auto v) {
        using T = decltype(v);
        if (wide) f(v, std::integral_constant<int, 16 / (int)sizeof(T)>{});
        else f(v, std::integral_constant<int, 1>{});
    });
}
static dim3 tok_grid(long long T) { return dim3(grid_of(ceil_div(T, kTokWaves))); }

void launch_dispatch(const void* x, int dtype, long long T, int m, long long D, int E, const int32_t* offsets,
                     const int32_t* place, void* xs, hipStream_t st) {
    if (T < 1 || D < 1) return;
    with_pack(dtype, D, {x, xs}, [&](auto tv, auto vv) {
        using S = decltype(tv);
        constexpr int V = decltype(vv)::value;
        hipLaunchKernelGGL((k_dispatch<S, V>), tok_grid(T), dim3(kTokThreads), 0, st, (const S*)x, T, m, D, E, offsets,
                           place, (S*)xs);
    });
}

void launch_dispatch_vjp(const void* dxs, int dtype, long long T, int m, long long D, const int32_t* place, void* dx,
                         hipStream_t st) {
    launch_combine(dxs, nullptr, nullptr, dtype, T, m, D, place, dx, st);
}

void launch_combine(const void* ys, const float* w, const void* residual, int dtype, long long T, int m, long long D,
                    const int32_t* place, void* out, hipStream_t st) {
    if (T < 1 || D < 1) return;
    with_pack(dtype, D, {ys, residual, out}, [&](auto tv, auto vv) {
        using S = decltype(tv);
        constexpr int V = decltype(vv)::value;
        hipLaunchKernelGGL((k_combine<S, V>), tok_grid(T), dim3(kTokThreads), 0, st, (const S*)ys, w,
                           (const S*)residual, T, m, D, place, (S*)out);
    });
}

void launch_combine_vjp(const void* ys, const float* w, const void* dout, int dtype, long long T, int m, long long D,
                        int E, const int32_t* offsets, const int32_t* place, void* dys, float* dw, hipStream_t st) {
    if (T < 1) return;
    with_pack(dtype, D, {ys, dout, dys}, [&](auto tv, auto vv) {
        using S = decltype(tv);
        constexpr int V = decltype(vv)::value;
        hipLaunchKernelGGL((k_combine_vjp<S, V>), tok_grid(T), dim3(kTokThreads), 0, st, (const S*)ys, w,
                           (const S*)dout, T, m, D, E, offsets, place, (S*)dys, dw);
    });
}

}  // namespace lapsum
