// Softmax cross entropy of 16-bit rows whose width is a multiple of 8: tiles in
// LDS and 16-bit matrix instructions (lapsum_tile_mfma.h), fp32 sums.
//
// Forward, a tile of logits stays in registers: a wave reduces its half of the
// tile's columns to a row's maximum and sum of exponentials, 8 bytes a row for
// BN / 2 columns, and the target's logit is written by the lane that holds it.
// Backward, the same tile becomes d, rounded to 16 bits, in scratch: a piece of
// the vocabulary at a time, small enough that the products that follow, dx +=
// d W and dW = d^T x, find it in the memory-side cache.  db's sums are taken of d in
// fp32, before that rounding: a wave's rows in registers, one partial row each.
//
// The products' feed bounds all of it (lapsum_tile_mfma.h), and beside a tile's
// first loads and its exponentials no products run.  8192 rows of 2048 over 65536
// in bf16: forward 1.69 to 1.76 ms (1.25 to 1.30 PFLOP/s; a library's product 1.2 to
// 1.44), gradients 5.05 to 5.35 ms, in pieces of 16384 columns d 0.47, dx and dW 0.40
// each (1.37 PFLOP/s).  4096 rows of 1024 over 50001 in fp16 with a bias: the forward
// call 411 to 437 us, its gradients 1500.
#include "lapsum_layer_ops.h"
#include "lapsum_tile_mfma.h"

namespace lapsum {

constexpr float kLog2e = 1.4426950408889634f;
// d of a piece: what the memory-side cache holds, and more, up to four times as
// much, where dW of so few columns would not fill the CUs with its widest tiles
// (us with 128 MiB / 256 MiB / 512 MiB / 1 GiB: 8192 rows, 65536 of 2048 5630 /
// 5430 / 5430 / 5470; 16384, 128256 of 4096 44400 / 42200 / 41200 / 41500; 32768,
// 32768 of 1024 11200 / 7900 / 7000 / 6030)
constexpr long long kPieceBytes = 256ll << 20, kMostBytes = 1ll << 30, kPieceWeights = 1 << 24;

static size_t take(size_t& at, size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~(size_t)255;
    return here;
}

bool loss_tile_takes(int dtype, const LossArgs& g) {
    if (dtype == kF32 || g.D % 8 || g.D < 8 || g.D > (1 << 20) || g.T < 1 || !aligned16(g.x) || !aligned16(g.w))
        return false;
    return ceil_div(g.T, 64) * ceil_div(g.V, 64) < 16 * kGridMax;  // one tile a workgroup
}

// The side of a product's tiles: wide ones where they fill the CUs.
static int side_of(long long M, long long N) {
    if (ceil_div(M, 256) * ceil_div(N, 256) >= 192) return 256;
    return ceil_div(M, 128) * ceil_div(N, 128) >= 128 ? 128 : 64;
}
template <class F>
static void with_side(int side, F&& f) {
    if (side == 256) f(std::integral_constant<int, 256>{});
    else if (side == 128) f(std::integral_constant<int, 128>{});
    else f(std::integral_constant<int, 64>{});
}

// Which tile of `rows` x `cols` a workgroup forms: four row tiles walk the
// columns together, XCD by XCD (take_turn).
struct TileAt {
    int i, j;  // -1: none
    int quarter;
};
LS_DEV TileAt tile_at(int rows, int cols, bool cut) {
    constexpr int kGroup = 4;
    const Turn t = take_turn(blockIdx.x, rows * cols, cut);
    if (t.tile < 0) return {-1, -1, -1};
    const int first = t.tile / (kGroup * cols) * kGroup, n = min(kGroup, rows - first);
    const int in = t.tile - first * cols;
    return {first + in % n, in / n, t.quarter};
}

// ---- forward ---------------------------------------------------------------------

// Up to kFewRows rows a tile would be mostly empty, and k_loss_few streams the
// weights instead (tiles / few, forward over 32768 of 2048 in bf16: 8 rows 43 / 35
// us, 32 rows 44 / 40, 64 rows 44 / 51).
constexpr int kFewRows = 32, kFewCols = 64, kFewWaves = 4;

LossParts loss_tile_parts(const LossArgs& g) {
    LossParts p{};
    const int side = side_of(g.T, g.V);
    p.parts = (int)(g.T <= kFewRows ? ceil_div(g.V, kFewCols) : 2 * ceil_div(g.V, side));
    size_t at = 0;
    p.pairs = take(at, (size_t)p.parts * g.T * sizeof(float2));
    p.zt = take(at, (size_t)g.T * 4);
    p.loss = take(at, (size_t)g.T * 4);
    p.bytes = at;
    return p;
}

// v += bias, eight columns from j of n
template <class T>
LS_DEV void add_bias(float (&v)[8], const T* bias, int j, int n) {
    if (!bias) return;
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] += j + r < n ? to_f(bias[j + r]) : 0.0f;
}
LS_DEV float across16(float v, bool max_) {  // over the four lanes that share a row
    float o = __uint_as_float(xor_lane<16>(__float_as_uint(v)));
    v = max_ ? fmaxf(v, o) : v + o;
    o = __uint_as_float(xor_lane<32>(__float_as_uint(v)));
    return max_ ? fmaxf(v, o) : v + o;
}

// A tile of B x B from row i0 and column j0: pairs of `part` and, of the tile's
// right half, part + 1; MERGE: one pair for both halves.
template <class T, int B, bool MERGE>
LS_DEV void loss_tile(const LossArgs& g, int i0, int j0, int part, char* lds, float2* __restrict__ pairs,
                      float* __restrict__ zt) {
    using Tile = TileSums<T, true, true, B, B>;
    const int M = g.T - i0, N = g.V - j0;
    Tile tile;
    tile.run((const T*)g.x + (long long)i0 * g.D, M, g.D, (const T*)g.w + (long long)j0 * g.D, N, g.D, g.D, lds);
    const int l = lane_id(), w = uniform(threadIdx.x >> 6);
    const int r0 = (w >> 1) * (B / 2), c0 = (w & 1) * (B / 2);
    const T* bias = g.bias ? (const T*)g.bias + j0 : nullptr;
    int64_t target[Tile::FM];
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i) target[i] = g.target[i0 + min(r0 + i * 16 + (l & 15), M - 1)];
    // a lane's columns: 8 (l / 16) .. + 7 of each 32; what is added to their
    // logits, -inf past the vocabulary's end
    const bool edge = bias || N < B;
    float add[Tile::FN][4] = {};
    if (edge) {
#pragma unroll
        for (int j = 0; j < Tile::FN; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int col = c0 + (j >> 1) * 32 + (l >> 4) * 8 + (j & 1) * 4 + r;
                add[j][r] = col >= N ? -__builtin_inff() : bias ? to_f(bias[col]) : 0.0f;
            }
    }
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i) {
        const int row = r0 + i * 16 + (l & 15);
        f32x4 v[Tile::FN];
        float m = -__builtin_inff();
#pragma unroll
        for (int j = 0; j < Tile::FN; ++j) {
            v[j] = tile.acc[i][j];
            if (edge) {
#pragma unroll
                for (int r = 0; r < 4; ++r) v[j][r] += add[j][r];
            }
            m = fmaxf(m, fmaxf(fmaxf(v[j][0], v[j][1]), fmaxf(v[j][2], v[j][3])));
        }
        m = across16(m, true);
        // m log2 e as it is rounded here cancels in the row's logarithm to within
        // its own rounding
        const float from = m == -__builtin_inff() ? 0.0f : m * -kLog2e;
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < Tile::FN; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) s += __builtin_amdgcn_exp2f(fmaf(v[j][r], kLog2e, from));
        s = across16(s, false);
        if (MERGE) {
            float2* half = (float2*)lds + row;  // (the sums' buffers are free)
            if (w & 1) *half = make_float2(m, s);
            __syncthreads();
            if (!(w & 1)) {
                const float2 o = *half;
                const float top = fmaxf(m, o.x), at = top == -__builtin_inff() ? 0.0f : top;
                s = s * __builtin_amdgcn_exp2f((m - at) * kLog2e) + o.y * __builtin_amdgcn_exp2f((o.x - at) * kLog2e);
                m = top;
                if (l < 16 && row < M) pairs[(long long)part * g.T + i0 + row] = make_float2(m, s);
            }
        } else if (l < 16 && row < M) {
            pairs[(long long)(part + (w & 1)) * g.T + i0 + row] = make_float2(m, s);
        }
        if (row >= M) continue;
        // the target, if this lane holds it
        const int64_t c = target[i] - j0 - c0;
        if (target[i] < 0 || target[i] >= g.V || c < 0 || c >= B / 2 || (c & 31) >> 3 != l >> 4) continue;
        float z = 0.0f;
#pragma unroll
        for (int j = 0; j < Tile::FN; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (c == (j >> 1) * 32 + (l >> 4) * 8 + (j & 1) * 4 + r) z = v[j][r];
        zt[i0 + row] = z;
    }
}

template <class T, int B>
__global__ __launch_bounds__(kProductThreads) void k_loss_tile(LossArgs g, int rows, int cols, float2* __restrict__ pairs,
                                                               float* __restrict__ zt) {
    __shared__ __align__(1024) char lds[TileSums<T, true, true, B, B>::kLds];
    const TileAt at = tile_at(rows, cols, B == 256);
    if (at.i < 0) return;
    if constexpr (B == 256) {
        if (at.quarter >= 0) {
            const int i0 = at.i * B + (at.quarter >> 1) * (B / 2), j0 = at.j * B + (at.quarter & 1) * (B / 2);
            const int part = at.j * 2 + (at.quarter & 1);
            if (i0 < g.T && j0 < g.V) {
                loss_tile<T, B / 2, true>(g, i0, j0, part, lds, pairs, zt);
            } else if (threadIdx.x < B / 2 && i0 + (int)threadIdx.x < g.T) {  // no columns
                pairs[(long long)part * g.T + i0 + threadIdx.x] = make_float2(-__builtin_inff(), 0.0f);
            }
            return;
        }
    }
    loss_tile<T, B, false>(g, at.i * B, at.j * B, at.j * 2, lds, pairs, zt);
}

// 16 FM rows and kFewCols columns of the piece v0 .. v0 + n - 1, to pairs or (GRAD)
// to d, as k_loss_dtile: bound by reading the weights, once.  The
// waves split the sum; each multiplies its share straight from memory (a weight
// is used once, so LDS would only add a stop on its way), and their sums meet in
// LDS, added in wave order.
template <class T, int FM, bool GRAD>
__global__ __launch_bounds__(kFewWaves * 64) void k_loss_few(LossArgs g, int v0, int n, float2* __restrict__ pairs,
                                                              float* __restrict__ zt, int ld,
                                                              const float* __restrict__ lse,
                                                              const float* __restrict__ grad, T* __restrict__ d,
                                                              float* __restrict__ db) {
    constexpr int FN = kFewCols / 16, U = FM == 1 ? 4 : 2;  // steps of 32 k in flight
    constexpr int kPad = kFewCols + 4;
    __shared__ float part[kFewWaves][16][kPad];
    const int l = lane_id(), w = uniform(threadIdx.x >> 6), i16 = l & 15, k8 = (l >> 4) * 8;
    const int j0 = blockIdx.x * kFewCols, D = g.D;
    // this lane's rows: those past the end read the last one again, and their
    // results are not stored
    const T *x[FM], *b[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) x[i] = (const T*)g.x + (long long)min(i * 16 + i16, g.T - 1) * D + k8;
#pragma unroll
    for (int j = 0; j < FN; ++j) b[j] = (const T*)g.w + (long long)(v0 + min(j0 + j * 16 + i16, n - 1)) * D + k8;
    f32x4 acc[FM][FN] = {};
    const int steps = (D + 31) / 32, whole = D / 32, s1 = (w + 1) * steps / kFewWaves;
    int s = w * steps / kFewWaves;
    for (; s + U <= min(s1, whole); s += U) {
        s16x8 fx[U][FM], fb[U][FN];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < FN; ++j) fb[u][j] = *(const s16x8*)(b[j] + (s + u) * 32);
#pragma unroll
            for (int i = 0; i < FM; ++i) fx[u][i] = *(const s16x8*)(x[i] + (s + u) * 32);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mfma16<T>(fb[u][j], fx[u][i], acc[i][j]);
    }
    for (; s < s1; ++s) {
        const bool on = s * 32 + k8 < D;
        s16x8 fx[FM], fb[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[j] = on ? *(const s16x8*)(b[j] + s * 32) : s16x8{};
#pragma unroll
        for (int i = 0; i < FM; ++i) fx[i] = on ? *(const s16x8*)(x[i] + s * 32) : s16x8{};
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = mfma16<T>(fb[j], fx[i], acc[i][j]);
    }
    // lane l holds row l % 16 of a fragment, columns 4 (l / 16) .. + 3
    const int row = threadIdx.x >> 4, c = (threadIdx.x & 15) * 4;
    float add[4], sums[4] = {};  // sums: of d over this thread's rows
#pragma unroll
    for (int r = 0; r < 4; ++r)
        add[r] = j0 + c + r >= n ? -__builtin_inff() : g.bias ? to_f(((const T*)g.bias)[v0 + j0 + c + r]) : 0.0f;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        if (i) __syncthreads();
#pragma unroll
        for (int j = 0; j < FN; ++j) *(f32x4*)&part[w][i16][j * 16 + (l >> 4) * 4] = acc[i][j];
        __syncthreads();
        const int t = i * 16 + row;
        if (t >= g.T) continue;  // (all 16 lanes of a row)
        f32x4 v = *(const f32x4*)&part[0][row][c];
#pragma unroll
        for (int p = 1; p < kFewWaves; ++p) v += *(const f32x4*)&part[p][row][c];
        const int64_t at = g.target[t] - v0 - j0 - c;
        if constexpr (GRAD) {
            const float gt = grad[t], lo = lse[t] * -kLog2e;
            struct __attribute__((aligned(8))) T4 { T v[4]; } o;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float p = __builtin_amdgcn_exp2f(fmaf(v[r] + add[r], kLog2e, lo));
                const bool on = gt != 0.0f && j0 + c + r < n;
                const float e = on ? (p - (at == r ? 1.0f : 0.0f)) * gt : 0.0f;
                sums[r] += e;
                o.v[r] = from_f<T>(e);
            }
            if (j0 + c < ld) *(T4*)(d + (long long)t * ld + j0 + c) = o;  // ld is a multiple of 8
            continue;
        }
        float m = -__builtin_inff();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            v[r] += add[r];
            m = fmaxf(m, v[r]);
        }
        m = fmaxf(m, __uint_as_float(xor_lane<8>(__float_as_uint(m))));
        m = fmaxf(m, __uint_as_float(xor_lane<4>(__float_as_uint(m))));
        m = fmaxf(m, __uint_as_float(xor_lane<2>(__float_as_uint(m))));
        m = fmaxf(m, __uint_as_float(xor_lane<1>(__float_as_uint(m))));
        const float from = m == -__builtin_inff() ? 0.0f : m * -kLog2e;
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) sum += __builtin_amdgcn_exp2f(fmaf(v[r], kLog2e, from));
        sum += __uint_as_float(xor_lane<8>(__float_as_uint(sum)));
        sum += __uint_as_float(xor_lane<4>(__float_as_uint(sum)));
        sum += __uint_as_float(xor_lane<2>(__float_as_uint(sum)));
        sum += __uint_as_float(xor_lane<1>(__float_as_uint(sum)));
        if (c == 0) pairs[(long long)blockIdx.x * g.T + t] = make_float2(m, sum);
        if (at < 0 || at >= 4 || g.target[t] >= g.V) continue;
        zt[t] = at == 0 ? v[0] : at == 1 ? v[1] : at == 2 ? v[2] : v[3];
    }
    if (!GRAD || !db) return;
    // the wave's four rows of each sixteen: a partial row a wave
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        sums[r] += __uint_as_float(xor_lane<16>(__float_as_uint(sums[r])));
        sums[r] += __uint_as_float(xor_lane<32>(__float_as_uint(sums[r])));
    }
    if (l < 16 && j0 + c < ld) *(f32x4*)(db + (long long)w * ld + j0 + c) = f32x4{sums[0], sums[1], sums[2], sums[3]};
}

template <bool GRAD>
static void launch_few(int dtype, const LossArgs& g, int v0, int n, float2* pairs, float* zt, int ld, const float* lse,
                       const float* grad, void* d, float* db, hipStream_t st) {
    with_dtype(dtype, [&](auto tv) {
        using T = decltype(tv);
        if constexpr (sizeof(T) == 2) {
            auto launch = [&](auto fm) {
                hipLaunchKernelGGL((k_loss_few<T, fm.value, GRAD>), dim3((unsigned)ceil_div(n, kFewCols)),
                                   dim3(kFewWaves * 64), 0, st, g, v0, n, pairs, zt, ld, lse, grad, (T*)d, db);
            };
            if (g.T <= 16) launch(std::integral_constant<int, 1>{});
            else launch(std::integral_constant<int, 2>{});
        }
    });
}

void launch_loss_tile(int dtype, const LossArgs& g, const LossParts& p, char* scratch, hipStream_t st) {
    if (g.T <= kFewRows) {
        launch_few<false>(dtype, g, 0, g.V, (float2*)(scratch + p.pairs), (float*)(scratch + p.zt), 0, nullptr, nullptr,
                          nullptr, nullptr, st);
        return;
    }
    with_side(side_of(g.T, g.V), [&](auto bv) {
        constexpr int B = bv.value;
        const long long rows = ceil_div(g.T, B), cols = ceil_div(g.V, B);
        with_dtype(dtype, [&](auto tv) {
            using T = decltype(tv);
            if constexpr (sizeof(T) == 2)
                hipLaunchKernelGGL((k_loss_tile<T, B>), dim3((unsigned)turns(rows * cols, B == 256)), dim3(kProductThreads), 0,
                                   st, g, (int)rows, (int)cols, (float2*)(scratch + p.pairs), (float*)(scratch + p.zt));
        });
    });
}

// ---- backward --------------------------------------------------------------------

LossVjpPlan loss_tile_plan(const LossArgs& g) {
    LossVjpPlan p{};
    const auto columns = [&](long long bytes) { return bytes / 2 / g.T / 256 * 256; };
    const long long fill = ceil_div(kPieceWeights, 256ll * g.D) * 256;
    const long long most = std::max({columns(kPieceBytes), std::min(fill, columns(kMostBytes)), 256ll});
    p.width = (int)std::min<long long>(std::min(most, 1ll << 18), g.V);
    p.ld = (p.width + 7) & ~7;
    p.pieces = (int)ceil_div(g.V, p.width);
    // dx's sum over a piece is shared out where its tiles are few
    const long long tiles = ceil_div(g.T, 64) * ceil_div(g.D, 64);
    p.shares = (int)std::max(1ll, std::min<long long>(512 / tiles, p.width / 512));
    size_t at = 0;
    p.g = take(at, ((size_t)g.T + 1) * 4);
    p.x = take(at, (size_t)g.T * g.D * 2);
    p.d = take(at, (size_t)g.T * p.ld * 2);
    p.db = take(at, (size_t)std::max<long long>(2 * ceil_div(g.T, 64), kFewWaves) * p.ld * 4);
    if (p.pieces * p.shares > 1) p.dx = take(at, (size_t)p.shares * g.T * g.D * 4);
    p.bytes = at;
    return p;
}

// d of the columns v0 .. v0 + n - 1, zeros up to a multiple of 8, and with
// DB: its column sums, unrounded, of each wave's rows: row 2 i + (0, 1) of db for row
// tile i.  (As a choice at run time it cost those without a bias 1 %.)
template <class T, int B, bool DB>
__global__ __launch_bounds__(kProductThreads) void k_loss_dtile(LossArgs g, int v0, int n, int ld, int rows, int cols,
                                                                const float* __restrict__ lse,
                                                                const float* __restrict__ grad, T* __restrict__ d,
                                                                float* __restrict__ db) {
    using Tile = TileSums<T, true, true, B, B>;
    __shared__ __align__(1024) char lds[Tile::kLds];
    const TileAt at = tile_at(rows, cols, false);
    if (at.i < 0) return;
    const int i0 = at.i * B, j0 = at.j * B, M = g.T - i0, N = n - j0;
    Tile tile;
    tile.run((const T*)g.x + (long long)i0 * g.D, M, g.D, (const T*)g.w + (long long)(v0 + j0) * g.D, N, g.D, g.D, lds);
    const T* bias = g.bias ? (const T*)g.bias + v0 + j0 : nullptr;
    struct __attribute__((aligned(16))) T8 { T v[8]; };
    const int l = lane_id(), w = uniform(threadIdx.x >> 6);
    const int r0 = (w >> 1) * (B / 2), c0 = (w & 1) * (B / 2);
    // this lane's rows, all asked for at once
    float gt[Tile::FM], lo[Tile::FM];
    int hit[Tile::FM];
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i) {
        const int t = i0 + min(r0 + i * 16 + (l & 15), M - 1);
        gt[i] = grad[t];
        lo[i] = lse[t] * -kLog2e;
        const int64_t at = g.target[t] - v0 - j0 - c0;
        hit[i] = at >= 0 && at < B / 2 ? (int)at : -1;
    }
#pragma unroll
    for (int j = 0; j < Tile::FN; j += 2) {
        const int in = j * 16 + (l >> 4) * 8, col = c0 + in;
        if (col >= ((N + 7) & ~7)) continue;
        float b[8] = {};
        add_bias(b, bias, col, N);
        float sums[8] = {};
#pragma unroll
        for (int i = 0; i < Tile::FM; ++i) {
            const int row = r0 + i * 16 + (l & 15);
            T8 o;
            float p[8], e[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                float v = tile.acc[i][j + (r >> 2)][r & 3];
                if (bias) v += b[r];
                p[r] = __builtin_amdgcn_exp2f(fmaf(v, kLog2e, lo[i]));
                // an ignored row has no gradient, whatever its logits are
                e[r] = gt[i] == 0.0f ? 0.0f : p[r] * gt[i];
            }
            if ((hit[i] & ~7) == in && gt[i] != 0.0f) {  // the target is here
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (hit[i] == in + r) e[r] = (p[r] - 1.0f) * gt[i];
            }
            if (DB && row < M) {
#pragma unroll
                for (int r = 0; r < 8; ++r) sums[r] += e[r];
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) o.v[r] = from_f<T>(e[r]);
            if (col + 8 > N) {
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (col + r >= N) o.v[r] = from_f<T>(0.0f);
            }
            if (row < M) *(T8*)(d + (long long)(i0 + row) * ld + j0 + col) = o;
        }
        if (!DB) continue;
#pragma unroll
        for (int r = 0; r < 8; ++r) {  // over the 16 lanes of these columns
            sums[r] += __uint_as_float(xor_lane<8>(__float_as_uint(sums[r])));
            sums[r] += __uint_as_float(xor_lane<4>(__float_as_uint(sums[r])));
            sums[r] += __uint_as_float(xor_lane<2>(__float_as_uint(sums[r])));
            sums[r] += __uint_as_float(xor_lane<1>(__float_as_uint(sums[r])));
        }
        if ((l & 15) == 0) {
            f32x4* to = (f32x4*)(db + (long long)(at.i * 2 + (w >> 1)) * ld + j0 + col);
            to[0] = f32x4{sums[0], sums[1], sums[2], sums[3]};
            to[1] = f32x4{sums[4], sums[5], sums[6], sums[7]};
        }
    }
}

struct LossProduct {
    const void *a, *b;
    int M, N, K, lda, ldb;
    int own_a;            // a's rows that can be read
    void* c;
    const float* g;       // of dx's rows: those of a 0 are 0, whatever the weights are (of dW: null)
    const float* unscale;
    int shares;           // of K: partial sums, M * N elements apart
    int share;            // k of a share, a multiple of 64
    bool add;
};
template <class T, bool kA, bool PART, int BM, int BN>
LS_DEV void product_tile(const LossProduct& g, int i0, int j0, int z, char* lds) {
    const int k0 = z * g.share, K = min(g.share, g.K - k0);
    const T* a = (const T*)g.a + (kA ? (long long)i0 * g.lda + k0 : (long long)k0 * g.lda + i0);
    const T* b = (const T*)g.b + (long long)k0 * g.ldb + j0;
    const int M = g.M - i0, N = g.N - j0;
    TileSums<T, kA, false, BM, BN> tile;
    tile.run(a, g.own_a - i0, g.lda, b, N, g.ldb, K, lds);
    struct __attribute__((aligned(16))) T8 { T v[8]; };
    const float unscale = PART ? 1.0f : *g.unscale;
    // kA: dx
    constexpr int FM = BM / 32;
    uint32_t none = 0;  // a bit a fragment
    if constexpr (kA) {
        const int r0 = (uniform(threadIdx.x >> 6) >> 1) * (BM / 2) + (lane_id() & 15);
#pragma unroll
        for (int i = 0; i < FM; ++i) none |= (g.g[i0 + min(r0 + i * 16, M - 1)] == 0.0f ? 1u : 0u) << i;
    }
    tile.each8([&](int row, int col, float (&v)[8]) {
        if (row >= M || col >= N) return;
        if constexpr (kA) {
            if (none >> (row >> 4 & (FM - 1)) & 1) {
#pragma unroll
                for (int r = 0; r < 8; ++r) v[r] = 0.0f;
            }
        }
        const long long to = (long long)(i0 + row) * g.N + j0 + col;
        if constexpr (PART) {
            f32x4* p = (f32x4*)((float*)g.c + (long long)z * g.M * g.N + to);
            f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
            if (g.add) lo += p[0], hi += p[1];
            p[0] = lo;
            p[1] = hi;
        } else {
            T8 o;
#pragma unroll
            for (int r = 0; r < 8; ++r) o.v[r] = from_f<T>(v[r] * unscale);
            *(T8*)((T*)g.c + to) = o;
        }
    });
}
template <class T, bool kA, bool PART, int B>
__global__ __launch_bounds__(kProductThreads) void k_loss_product(LossProduct g, int rows, int cols) {
    __shared__ __align__(1024) char lds[TileSums<T, kA, false, B, B>::kLds];
    const TileAt at = tile_at(rows, cols, B == 256);
    if (at.i < 0) return;
    int i0 = at.i * B, j0 = at.j * B;
    if constexpr (B == 256) {
        if (at.quarter >= 0) {
            i0 += (at.quarter >> 1) * (B / 2);
            j0 += (at.quarter & 1) * (B / 2);
            if (i0 < g.M && j0 < g.N) product_tile<T, kA, PART, B / 2, B / 2>(g, i0, j0, blockIdx.y, lds);
            return;
        }
    }
    product_tile<T, kA, PART, B, B>(g, i0, j0, blockIdx.y, lds);
}

template <bool kA, bool PART>
static void launch_product(int dtype, LossProduct& g, hipStream_t st) {
    g.share = (int)(ceil_div(ceil_div(g.K, g.shares), 64) * 64);
    with_side(side_of(g.M, g.N), [&](auto bv) {
        constexpr int B = bv.value;
        const long long rows = ceil_div(g.M, B), cols = ceil_div(g.N, B);
        with_dtype(dtype, [&](auto tv) {
            using T = decltype(tv);
            if constexpr (sizeof(T) == 2)
                hipLaunchKernelGGL((k_loss_product<T, kA, PART, B>),
                                   dim3((unsigned)turns(rows * cols, B == 256), (unsigned)g.shares), dim3(kProductThreads),
                                   0, st, g, (int)rows, (int)cols);
        });
    });
}

void launch_loss_tile_vjp(int dtype, const LossArgs& g, const LossVjpPlan& p, const float* lse, char* scratch,
                          void* dx, void* dw, void* db, hipStream_t st) {
    float* rows = (float*)(scratch + p.g);
    const float* unscale = rows + g.T;
    const bool part = p.pieces * p.shares > 1;
    for (int i = 0; i < p.pieces; ++i) {
        const int v0 = i * p.width, n = std::min(p.width, g.V - v0);
        float* part_db = db ? (float*)(scratch + p.db) : nullptr;
        long long db_rows = kFewWaves;
        if (g.T <= kFewRows)
            launch_few<true>(dtype, g, v0, n, nullptr, nullptr, p.ld, lse, rows, scratch + p.d, part_db, st);
        else with_side(side_of(g.T, n), [&](auto bv) {
            constexpr int B = bv.value;
            const long long r = ceil_div(g.T, B), c = ceil_div(n, B);
            db_rows = 2 * r;
            with_dtype(dtype, [&](auto tv) {
                using T = decltype(tv);
                auto launch = [&](auto sums) {
                    hipLaunchKernelGGL((k_loss_dtile<T, B, sums.value>), dim3((unsigned)turns(r * c, false)),
                                       dim3(kProductThreads), 0, st, g, v0, n, p.ld, (int)r, (int)c, lse, rows,
                                       (T*)(scratch + p.d), part_db);
                };
                if constexpr (sizeof(T) == 2) {
                    if (db) launch(std::true_type{});
                    else launch(std::false_type{});
                }
            });
        });
        if (db) launch_loss_db(dtype, part_db, p.ld, (int)db_rows, n, unscale, (char*)db + (size_t)v0 * 2, st);
        LossProduct q{};
        q.a = scratch + p.d;
        q.lda = p.ld;
        q.g = rows;
        q.unscale = unscale;
        if (dx) {
            q.b = (const char*)g.w + (size_t)v0 * g.D * 2;
            q.M = q.own_a = g.T, q.N = g.D, q.K = n, q.ldb = g.D;
            q.c = part ? scratch + p.dx : dx;
            q.shares = p.shares;
            q.add = i > 0;
            if (part) launch_product<true, true>(dtype, q, st);
            else launch_product<true, false>(dtype, q, st);
        }
        if (dw) {
            q.b = scratch + p.x;
            q.M = n, q.own_a = (n + 7) & ~7, q.N = g.D, q.K = g.T, q.ldb = g.D;
            q.c = (char*)dw + (size_t)v0 * g.D * 2;
            q.shares = 1;
            q.add = false;
            launch_product<false, false>(dtype, q, st);
        }
    }
    if (dx && part) launch_loss_dx(dtype, (const float*)(scratch + p.dx), p.shares, (long long)g.T * g.D, unscale, dx, st);
}

}  // namespace lapsum
