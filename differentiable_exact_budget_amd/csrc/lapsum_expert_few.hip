// The forward product where every expert has few rows, as in decoding: bound
// by reading the weights, once each.
//
// A workgroup takes 16 rows of an expert and 16 of its outputs.  Its four
// waves split the sum over k; each multiplies its quarter straight from memory
// (a weight is used once, so LDS would only add a stop on its way): a fragment
// is one 16-byte load a lane, and with the few registers this takes (24) eight
// waves of a SIMD have theirs in flight.  The waves' sums meet in LDS and are
// added in wave order, with bias and activation behind.
//
// 64 rows at 41 of 64 experts 2048 -> 1024 in bf16, 172 MB of weights: 33 us
// from memory, 5.2 TB/s (a large copy moves 4.9), and 29 us from the memory-side
// cache; with loads that pass the caches by, 36 us from either.
#include "lapsum_expert_tile.h"

namespace lapsum {

constexpr int kFewWaves = 4;

template <class T, int ACT>
__global__ __launch_bounds__(kFewWaves * 64) void k_product_few(LinearArgs g, int cols) {
    constexpr int U = 8;  // steps of 32 k without a masked end at a time
    using Z = typename ZKeep<T>::type;
    __shared__ float part[kFewWaves][16][20];
    const int l = lane_id(), w = uniform(threadIdx.x >> 6), i16 = l & 15, k8 = (l >> 4) * 8;
    const RowTile t = find_row_tile<16>(g.off, g.E, g.P, blockIdx.x / cols);
    if (t.lo >= t.hi) return;
    const int j0 = blockIdx.x % cols * 16, rows = t.hi - t.lo, N = g.out, K = g.in;
    const bool used = t.e < g.E;
    f32x4 acc = {};
    if (used) {
        // this lane's row of xs and of the weights: those past the end read
        // the last one again, and their results are not stored
        const T* x = (const T*)g.a + (long long)(t.lo + min(i16, rows - 1)) * K + k8;
        const T* b = (const T*)g.b + ((long long)t.e * N + min(j0 + i16, N - 1)) * K + k8;
        const int steps = (K + 31) / 32, whole = K / 32;  // whole: without a masked end
        const int s1 = (w + 1) * steps / kFewWaves;
        int s = w * steps / kFewWaves;
        for (; s + U <= min(s1, whole); s += U) {
            s16x8 fx[U], fb[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                fb[u] = *(const s16x8*)(b + (s + u) * 32);
                fx[u] = *(const s16x8*)(x + (s + u) * 32);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) acc = mfma16<T>(fb[u], fx[u], acc);
        }
        for (; s < s1; ++s) {
            const bool on = s * 32 + k8 < K;
            const s16x8 fb = on ? *(const s16x8*)(b + s * 32) : s16x8{};
            const s16x8 fx = on ? *(const s16x8*)(x + s * 32) : s16x8{};
            acc = mfma16<T>(fb, fx, acc);
        }
    }
    // lane l holds row l % 16, columns 4 (l / 16) .. + 3
    *(f32x4*)&part[w][i16][(l >> 4) * 4] = acc;
    __syncthreads();
    const int r = threadIdx.x >> 4, c = threadIdx.x & 15;
    if (r >= rows || j0 + c >= N) return;
    float v = part[0][r][c];
#pragma unroll
    for (int p = 1; p < kFewWaves; ++p) v += part[p][r][c];
    if (g.bias && used) v += to_f(((const T*)g.bias)[(long long)t.e * N + j0 + c]);
    const long long to = (long long)(t.lo + r) * N + j0 + c;
    ((T*)g.c)[to] = from_f<T>(act_of<ACT, T>(v));
    if (ACT != kActNone && g.z && used) ((Z*)g.z)[to] = ZKeep<T>::template make<ACT>(v);
}

static long long few_tiles(const LinearArgs& g) { return max_row_tiles<16>(g.P, g.E) * ceil_div(g.out, 16); }

// one tile a workgroup, whose threads a launch counts in 32 bits
bool expert_few_takes(const LinearArgs& g) { return few_tiles(g) < (1ll << 32) / (kFewWaves * 64); }

void launch_expert_few(int dtype, const LinearArgs& g, hipStream_t st) {
    const long long cols = ceil_div(g.out, 16), tiles = few_tiles(g);
    with_dtype(dtype, [&](auto tv) {
        using T = decltype(tv);
        if constexpr (sizeof(T) == 2)
            with_act(g.act, [&](auto av) {
                hipLaunchKernelGGL((k_product_few<T, decltype(av)::value>), dim3((unsigned)tiles),
                                   dim3(kFewWaves * 64), 0, st, g, (int)cols);
            });
    });
}

}  // namespace lapsum
