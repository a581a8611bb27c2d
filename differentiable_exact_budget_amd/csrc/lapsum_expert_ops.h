// Shared by the expert operators' kernels and their host code (gfx950,
// wave64): element types, activations, the search of a row tile among the
// experts, and the launchers (each defined next to its kernels).
#pragma once
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cstddef>

#include "lapsum_device.h"

namespace lapsum {

enum Dtype : int { kF32 = 0, kBF16 = 1, kF16 = 2 };
enum Act : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };

constexpr int kExpertsMax = 1024;
constexpr int kSlotsMax = 64;

// rows of dz that one workgroup sums for the bias gradient
constexpr int kDzRows = 64;

inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
// workgroups of a launch: kernels walk on by the grid where there is more work
// (a grid holds fewer than 2^32 threads)
constexpr long long kGridMax = 1 << 22;
inline unsigned grid_of(long long n) { return (unsigned)(n < kGridMax ? n : kGridMax); }
inline size_t dtype_size(int d) { return d == kF32 ? 4 : 2; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// calls f with a value of the element type
template <class F>
inline void with_dtype(int d, F&& f) {
    if (d == kF32) f(float{});
    else if (d == kBF16) f(__bf16{});
    else f(_Float16{});
}

template <class F>
inline void with_act(int act, F&& f) {
    if (act == kActRelu) f(std::integral_constant<int, kActRelu>{});
    else if (act == kActSilu) f(std::integral_constant<int, kActSilu>{});
    else if (act == kActGelu) f(std::integral_constant<int, kActGelu>{});
    else f(std::integral_constant<int, kActNone>{});
}

// lapsum_route.hip
// sums (null: no normalization): per row the sum that the weights are divided by
void launch_expert_topk(const float* gates, long long T, int E, int m, float floor, int32_t* ids, float* w,
                        float* sums, hipStream_t st);
void launch_expert_topk_vjp(const int32_t* ids, const float* w, const float* dw, const float* sums, long long T,
                            int E, int m, float* dgates, hipStream_t st);
size_t expert_sort_scratch(long long P, int E);
void launch_expert_sort(const int32_t* ids, long long P, int E, int32_t* offsets, int32_t* order, int32_t* place,
                        uint32_t* scratch, hipStream_t st);

// lapsum_tokens.hip
void launch_dispatch(const void* x, int dtype, long long T, int m, long long D, int E, const int32_t* offsets,
                     const int32_t* place, void* xs, hipStream_t st);
void launch_dispatch_vjp(const void* dxs, int dtype, long long T, int m, long long D, const int32_t* place, void* dx,
                         hipStream_t st);
void launch_combine(const void* ys, const float* w, const void* residual, int dtype, long long T, int m, long long D,
                    const int32_t* place, void* out, hipStream_t st);
void launch_combine_vjp(const void* ys, const float* w, const void* dout, int dtype, long long T, int m, long long D,
                        int E, const int32_t* offsets, const int32_t* place, void* dys, float* dw, hipStream_t st);

// lapsum_expert_linear.hip
// One product over all experts.  kFormY: C[rows, out] = A[rows, in] W_e^T;
// kFormDx: C[rows, in] = A[rows, out] W_e; kFormDw: C_e[out, in] = A^T B over
// the rows of e (A = dz[rows, out], B = xs[rows, in]).
enum Form : int { kFormY = 0, kFormDx = 1, kFormDw = 2 };
struct LinearArgs {
    const void* a;
    const void* b;
    const void* bias;   // kFormY, may be null
    void* c;
    void* z;            // kFormY, may be null
    const int32_t* off;
    int P, E, in, out;
    int act;            // kFormY
};
void launch_expert_product(int form, int dtype, const LinearArgs& g, hipStream_t st);
// lapsum_expert_mfma.hip: the products that the 16-bit matrix instructions take
bool expert_mfma_takes(int form, int dtype, const LinearArgs& g);
void launch_expert_mfma(int form, int dtype, const LinearArgs& g, hipStream_t st);
// lapsum_expert_few.hip: kFormY with few rows an expert, for what expert_mfma_takes
bool expert_few_takes(const LinearArgs& g);
void launch_expert_few(int dtype, const LinearArgs& g, hipStream_t st);
// dz (may be null: dz = dy, not written) and per-chunk column sums (may be
// null) of dz; then the sums per expert
void launch_expert_dz(const void* z, const void* dy, int dtype, int act, const int32_t* off, int P, int E, int out,
                      void* dz, float* part, hipStream_t st);
void launch_expert_dbias(const float* part, int dtype, const int32_t* off, int P, int E, int out, void* dbias,
                         hipStream_t st);

#if defined(__HIPCC__)

LS_DEV int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
template <class T>
LS_DEV T* uniform(T* p) {
    const uintptr_t u = reinterpret_cast<uintptr_t>(p);
    const uint32_t lo = (uint32_t)uniform((int)(uint32_t)u), hi = (uint32_t)uniform((int)(uint32_t)(u >> 32));
    return reinterpret_cast<T*>((uintptr_t)hi << 32 | lo);
}
LS_DEV float wave_sum_f32(float v) {
    v += __uint_as_float(xor_lane<32>(__float_as_uint(v)));
    v += __uint_as_float(xor_lane<16>(__float_as_uint(v)));
    v += __uint_as_float(xor_lane<8>(__float_as_uint(v)));
    v += __uint_as_float(xor_lane<4>(__float_as_uint(v)));
    v += __uint_as_float(xor_lane<2>(__float_as_uint(v)));
    v += __uint_as_float(xor_lane<1>(__float_as_uint(v)));
    return v;
}

// offsets[e] as a row number: a plan from elsewhere is kept in bounds
LS_DEV int row_at(const int32_t* __restrict__ off, int e, int P) { return min(max(off[e], 0), P); }

// The rows cut into tiles of BM that never cross an expert, the experts' tiles
// in order and those of the unused rows (e = E) behind them.  Lane l holds
// expert e0 + l of 64 experts; with more, find() goes through them again.
// Every lane of a wave calls these with one tile.
struct RowTile {
    int e;         // expert, or E
    int lo, hi;    // the tile's rows; a tile past the last has lo = hi = P
    int first;     // the expert's first tile
    int elo, ehi;  // the expert's rows
};
template <int BM>
struct RowTiles {
    const int32_t* off;
    int E, P;
    int lo, hi, inc;  // this lane's expert: its rows, and the tiles up to it

    LS_DEV void load(int e0) {
        const int e = e0 + lane_id();
        lo = e < E ? row_at(off, e, P) : 0;
        hi = e < E ? max(row_at(off, e + 1, P), lo) : 0;
        inc = (int)wave_inclusive_scan((uint32_t)((hi - lo + BM - 1) / BM));
    }
    LS_DEV RowTiles(const int32_t* __restrict__ off_, int E_, int P_) : off(off_), E(E_), P(P_) { load(0); }

    LS_DEV RowTile find(int tile) {
        int base = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            if (E > 64) load(e0);
            const unsigned long long hit = ballot(base + inc > tile);
            if (hit) {
                const int f = __builtin_ctzll(hit);
                RowTile t;
                t.e = e0 + f;
                t.elo = __builtin_amdgcn_readlane(lo, f);
                t.ehi = __builtin_amdgcn_readlane(hi, f);
                t.first = base + __builtin_amdgcn_readlane(inc, f) - (t.ehi - t.elo + BM - 1) / BM;
                t.lo = t.elo + (tile - t.first) * BM;
                t.hi = min(t.lo + BM, t.ehi);
                return t;
            }
            base += __builtin_amdgcn_readlane(inc, 63);
        }
        const int used = uniform(row_at(off, E, P));
        const int at = (int)min((long long)used + (long long)(tile - base) * BM, (long long)P);
        return {E, at, min(at + BM, P), base, used, P};
    }
    LS_DEV int count() {
        int n = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            if (E > 64) load(e0);
            n += __builtin_amdgcn_readlane(inc, 63);
        }
        return n + (P - uniform(row_at(off, E, P)) + BM - 1) / BM;
    }
};
template <int BM>
LS_DEV RowTile find_row_tile(const int32_t* __restrict__ off, int E, int P, int tile) {
    return RowTiles<BM>(off, E, P).find(tile);
}
// most tiles there can be (host)
template <int BM>
inline long long max_row_tiles(long long P, int E) {
    return P / BM + E + 1;
}

template <class T>
LS_DEV float to_f(T v) {
    return (float)v;
}
template <class T>
LS_DEV T from_f(float v) {
    return (T)v;
}

// 1 / (1 + e^-z): the hardware exponential and reciprocal, 1 ulp each; e^-z
// of very negative z is inf and its reciprocal 0, as it should be
LS_DEV float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}
// The normal distribution's tail Q(x) = erfc(x / sqrt 2) / 2 for x >= 0: a
// polynomial in t = 1 / (1 + c x) times e = e^(-x x / 2).  Its coefficients are
// a linear program's: least absolute error under a bound of 2e-4 on the
// relative one for x <= 13.2, past which bf16 has no normal Q.  As computed
// here, within 2e-7 of Q and 2.1e-4 Q of it.  (Five terms after Abramowitz and
// Stegun 7.1.26 are as near in absolute terms but 0.4 % off at 6 and 4 % at 13,
// more than bf16's rounding.)
LS_DEV float normal_tail(float x, float e) {
    const float t = __builtin_amdgcn_rcpf(fmaf(x, 0.287f, 1.0f));
    float s = fmaf(t, -0.09359798f, 0.31303203f);
    s = fmaf(t, s, -0.12899813f);
    s = fmaf(t, s, 0.19959147f);
    s = fmaf(t, s, 0.0937095f);
    s = fmaf(t, s, 0.11626307f);
    return s * t * e;
}

// Activations and their slopes, in fp32; T is the rows' type.  For 16-bit
// rows gelu takes the polynomial tail, whose relative error is below half of
// fp16's rounding and a sixteenth of bf16's, at the far end of z too.
template <int ACT, class T>
LS_DEV float act_of(float z) {
    if (ACT == kActRelu) return z > 0.0f ? z : (z != z ? z : 0.0f);
    if (ACT == kActSilu) return z * sigmoid(z);
    if (ACT == kActGelu) {
        if (sizeof(T) == 4) return 0.5f * z * (1.0f + erff(z * 0.70710678f));
        const float q = normal_tail(fabsf(z), __builtin_amdgcn_exp2f(z * z * (-0.5f * 1.4426950408889634f)));
        return z * (z > 0.0f ? 1.0f - q : q);
    }
    return z;
}
template <int ACT, class T>
LS_DEV float slope_of(float z) {
    if (ACT == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
    if (ACT == kActSilu) {
        const float q = sigmoid(z);
        return q * fmaf(z, 1.0f - q, 1.0f);
    }
    if (ACT == kActGelu) {
        const float e = __builtin_amdgcn_exp2f(z * z * (-0.5f * 1.4426950408889634f));
        if (sizeof(T) == 4) return fmaf(z * 0.39894228f, e, 0.5f * (1.0f + erff(z * 0.70710678f)));
        const float q = normal_tail(fabsf(z), e);
        return fmaf(z * 0.39894228f, e, z > 0.0f ? 1.0f - q : q);
    }
    return 1.0f;
}

// z as the VJP keeps it: fp32 for fp32 rows, else fp16, where a z beyond its
// range becomes infinite (the VJP takes it as the largest fp16: the slopes
// are 0 or 1 out there).  relu's slope depends on the sign alone, so a
// positive z that rounds to 0 is kept as the smallest positive value.
template <class T>
struct ZKeep {
    using type = _Float16;
    template <int ACT>
    static LS_DEV _Float16 make(float z) {
        const _Float16 h = (_Float16)z;
        if (ACT == kActRelu && z > 0.0f && h == (_Float16)0.0f) return (_Float16)5.9604645e-8f;
        return h;
    }
    static LS_DEV float value(_Float16 h) {
        const float z = (float)h;
        return fabsf(z) > 65504.0f ? copysignf(65504.0f, z) : z;
    }
};
template <>
struct ZKeep<float> {
    using type = float;
    template <int ACT>
    static LS_DEV float make(float z) {
        return z;
    }
    static LS_DEV float value(float z) { return z; }
};

#endif  // __HIPCC__

}  // namespace lapsum
