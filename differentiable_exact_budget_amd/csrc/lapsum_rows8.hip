// Rows to 8-bit floating point and back: blocks of 128 along a row, each e4m3
// values under a power of two.
//
// Mathematics: for a block with largest finite magnitude a, e is the least
// integer with a <= 448 2^e (held to -127 and more; 0 where a is 0), and q =
// e4m3(x 2^-e), to nearest, ties to even.  A power of two divides exactly, so
// the only rounding is e4m3's, and the scaled matrix instruction multiplies by
// it for nothing.  What is not finite becomes NaN and leaves its block's other
// values alone.  Rows are padded with zeros to whole blocks.
//
// 16 lanes take a block, 8 elements each; a wave takes 4 U neighbouring blocks
// of a row.  Memory bounds it: 65536 rows of 2048 in bf16 in 65 us, back in 72
// (6.2 and 5.6 TB/s; 403 MB either way); 64 rows in 3.8 and 3.2.
#include "lapsum_layer_ops.h"
#include "lapsum_rows.h"

namespace lapsum {

constexpr int kRows8Waves = 4;

// elements c .. c + 7 of a row, as floats; zeros past its end
template <class T>
LS_DEV void load8(float (&v)[8], const T* row, long long c, long long D) {
    constexpr int V = Pack<T>::V;
#pragma unroll
    for (int p = 0; p < 8 / V; ++p) {
        const Pack<T> x = ld<true>(row, c + p * V, D);
#pragma unroll
        for (int i = 0; i < V; ++i) v[p * V + i] = to_f(x.v[i]);
    }
}

template <class T, int U>
__global__ __launch_bounds__(kRows8Waves * 64) void k_quantize(const T* __restrict__ x, long long rows, long long D,
                                                               int blocks, int stretches, uint8_t* __restrict__ q,
                                                               uint8_t* __restrict__ scale) {
    const int l = lane_id();
    for (long long i = (long long)blockIdx.x * kRows8Waves + uniform(threadIdx.x >> 6); i < rows * stretches;
         i += (long long)gridDim.x * kRows8Waves) {
        const long long r = i / stretches;
        const int b0 = (int)(i - r * stretches) * (4 * U) + (l >> 4);
        float v[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) load8(v[u], x + r * D, (long long)(b0 + 4 * u) * kBlock8 + (l & 15) * 8, D);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t a = __float_as_uint(v[u][k]) & 0x7FFFFFFFu;
                top = max(top, a < 0x7F800000u ? a : 0u);
            }
            top = max(top, xor_lane<8>(top));
            top = max(top, xor_lane<4>(top));
            top = max(top, xor_lane<2>(top));
            top = max(top, xor_lane<1>(top));
            // 448 = 1.75 * 2^8
            int e = max((int)(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u), -127);
            if (top == 0) e = 0;
            const float by = __uint_as_float((uint32_t)(127 - e) << 23);
            uint32_t w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float f[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float y = v[u][h * 4 + k] * by;
                    f[k] = fabsf(y) <= 448.0f ? y : __builtin_nanf("");
                }
                int o = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
                w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], o, true);
            }
            const int b = b0 + 4 * u;
            if (b >= blocks) continue;
            *(uint2*)(q + ((r * blocks + b) * kBlock8 + (l & 15) * 8)) = make_uint2(w[0], w[1]);
            if ((l & 15) == 0) scale[r * blocks + b] = (uint8_t)(e + 127);
        }
    }
}

// what the values stand for, rounded to the rows' type
template <class T, int U>
__global__ __launch_bounds__(kRows8Waves * 64) void k_dequantize(const uint8_t* __restrict__ q,
                                                                 const uint8_t* __restrict__ scale, long long rows,
                                                                 long long D, int blocks, int stretches,
                                                                 T* __restrict__ x) {
    const int l = lane_id();
    for (long long i = (long long)blockIdx.x * kRows8Waves + uniform(threadIdx.x >> 6); i < rows * stretches;
         i += (long long)gridDim.x * kRows8Waves) {
        const long long r = i / stretches;
        const int b0 = (int)(i - r * stretches) * (4 * U) + (l >> 4);
        uint2 w[U];
        int e[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long b = r * blocks + min(b0 + 4 * u, blocks - 1);
            w[u] = *(const uint2*)(q + b * kBlock8 + (l & 15) * 8);
            e[u] = scale[b];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long c = (long long)(b0 + 4 * u) * kBlock8 + (l & 15) * 8;
            if (b0 + 4 * u >= blocks) continue;
            constexpr int V = Pack<T>::V;
            float v[8];
            for (int h = 0; h < 2; ++h) {
                const int word = h ? (int)w[u].y : (int)w[u].x;
                const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(word, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(word, true);
                v[h * 4] = lo[0], v[h * 4 + 1] = lo[1], v[h * 4 + 2] = hi[0], v[h * 4 + 3] = hi[1];
            }
#pragma unroll
            for (int p = 0; p < 8 / V; ++p) {
                Pack<T> o;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    // the scale 255 is NaN
                    const float y = __builtin_amdgcn_ldexpf(v[p * V + k], e[u] - 127);
                    o.v[k] = from_f<T>(e[u] == 255 ? __builtin_nanf("") : y);
                }
                st<T>(x + r * D, c + p * V, D, o);
            }
        }
    }
}

// blocks a lane has in flight: four where a row has so many
template <class F>
static void with_blocks(long long blocks, F&& f) {
    if (blocks >= 16) f(std::integral_constant<int, 4>{});
    else f(std::integral_constant<int, 1>{});
}

void launch_quantize(const void* x, int dtype, long long rows, long long D, uint8_t* q, uint8_t* scale, hipStream_t st) {
    const long long blocks = ceil_div(D, kBlock8);
    if (rows < 1 || blocks < 1) return;
    with_dtype(dtype, [&](auto tv) {
        using T = decltype(tv);
        with_blocks(blocks, [&](auto u) {
            const long long n = ceil_div(blocks, 4 * u.value);
            hipLaunchKernelGGL((k_quantize<T, u.value>), dim3(grid_of(ceil_div(rows * n, kRows8Waves))),
                               dim3(kRows8Waves * 64), 0, st, (const T*)x, rows, D, (int)blocks, (int)n, q, scale);
        });
    });
}
void launch_dequantize(const uint8_t* q, const uint8_t* scale, int dtype, long long rows, long long D, void* x,
                       hipStream_t st) {
    const long long blocks = ceil_div(D, kBlock8);
    if (rows < 1 || blocks < 1) return;
    with_dtype(dtype, [&](auto tv) {
        using T = decltype(tv);
        with_blocks(blocks, [&](auto u) {
            const long long n = ceil_div(blocks, 4 * u.value);
            hipLaunchKernelGGL((k_dequantize<T, u.value>), dim3(grid_of(ceil_div(rows * n, kRows8Waves))),
                               dim3(kRows8Waves * 64), 0, st, q, scale, rows, D, (int)blocks, (int)n, (T*)x);
        });
    });
}

}  // namespace lapsum
