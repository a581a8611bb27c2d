// Softmax cross entropy of a product with a vocabulary's weights: the steps
// around the products, and the products of every type, size and alignment.
//
// Mathematics: z = x W^T + b, lse = log sum over v of e^z_v, loss = lse -
// z_target; with g the loss' gradient, d = (e^(z - lse) - onehot) g and
//   dx = d W,  dW = d^T x,  db = sum of d over the rows.
//
// z is never kept whole.  Forward, columns are taken in parts: each leaves a
// row's maximum and its sum of exponentials about it, which launch_loss_rows
// merges.  Backward, z is formed again, a piece of the vocabulary at a time,
// and turned into d by the lse of the forward pass.
//
// Here the products are those for any alignment (lapsum_tile_any.h).  Tiles of
// 32 columns reduce them as they are; wide tiles' logits go through scratch in
// fp32, a piece of the vocabulary at a time.  For dx and dW d is rounded to the
// rows' type once, because the matrix instructions take it so; its rows are taken
// over the largest gradient of a row's loss (k_loss_grad_rows), and the products
// are multiplied by that again in fp32.  db is summed before the rounding, by the
// tiles that form d.
//
// fp32's matrix rate bounds the large ones: 4096 rows of 1024 over 8192, forward
// 576 us (119 TFLOP/s of 154).  513 rows of 257 over 1001 in fp32: kernels of 9 to
// 12 us, the latencies of sums this short.
#include "lapsum_layer_ops.h"
#include "lapsum_rows.h"
#include "lapsum_tile_any.h"

namespace lapsum {

constexpr float kLog2e = 1.4426950408889634f;
constexpr long long kPieceBytes = 128ll << 20;  // of fp32 logits, or of d as it were fp32
static_assert(sizeof(float2) == 8);

static size_t take(size_t& at, size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~(size_t)255;
    return here;
}

// The side of a product's tiles, which 32-wide ones share among a workgroup's
// waves: for 16-bit rows as for the experts' products; for fp32, whose wide tiles
// take long, 128 from three rounds of them on, and 64 before (forward, us, 128 /
// 64 / 32: 4096 rows over 8192 of 1024 576 / 620 / -; 2000 over 3000 of 512 85 / 79
// / -; 156 over 43301 of 3624 984 / 594 / -; 300 over 5000 of 333 44 / 30 / 35; 513
// over 1001 of 257 37 / 21 / 17).
static int any_side(int dtype, long long M, long long N, int shares) {
    const auto tiles = [&](int side) { return ceil_div(M, side) * ceil_div(N, side) * shares; };
    const long long least = std::min(M, N);
    if (dtype != kF32) return least > 64 && tiles(128) >= 128 ? 128 : 32;
    if (least > 64 && tiles(128) >= 1536) return 128;
    return least > 32 && tiles(64) >= 320 ? 64 : 32;
}

static int any_width(const LossArgs& g) {
    const long long w = std::max(kPieceBytes / 4 / std::max(g.T, 1) / 128 * 128, 128ll);
    return (int)std::min<long long>(w, std::max(g.V, 1));
}

LossParts loss_any_parts(int dtype, const LossArgs& g) {
    LossParts p{};
    p.width = any_width(g);
    // narrow tiles reduce their columns themselves
    const bool logits = any_side(dtype, g.T, std::min(p.width, g.V), 1) > 32;
    p.parts = (int)(logits ? ceil_div(g.V, p.width) : ceil_div(g.V, 32));
    size_t at = 0;
    p.pairs = take(at, (size_t)p.parts * g.T * sizeof(float2));
    p.zt = take(at, (size_t)g.T * 4);
    p.loss = take(at, (size_t)g.T * 4);
    if (logits) p.logits = take(at, (size_t)g.T * p.width * 4);
    p.bytes = at;
    return p;
}

// The shares of dx's sum over a piece: as many as make enough wide tiles (156 rows
// of 3624 over 43301 in fp32: 3900 us unshared, 550 in seven), or enough narrow
// ones where there are few rows.
static int any_shares(int dtype, const LossArgs& g, int width) {
    const auto shares = [&](long long need, int side, int least) {
        const long long tiles = std::max(ceil_div(g.T, side) * ceil_div(g.D, side), 1ll);
        return (int)std::max(1ll, std::min<long long>(ceil_div(need, tiles), width / least));
    };
    const int wide = dtype == kF32 ? shares(1024, 64, 1024) : shares(128, 128, 1024);
    if (any_side(dtype, g.T, g.D, wide) > 32) return wide;
    return shares(512, 32, 512);
}

LossVjpPlan loss_any_plan(int dtype, const LossArgs& g) {
    LossVjpPlan p{};
    p.width = any_width(g);
    p.ld = p.width;
    p.pieces = (int)ceil_div(g.V, p.width);
    p.shares = any_shares(dtype, g, p.width);
    size_t at = 0;
    p.g = take(at, ((size_t)g.T + 1) * 4);
    p.x = take(at, (size_t)g.T * g.D * dtype_size(dtype));
    p.d = take(at, (size_t)g.T * p.width * dtype_size(dtype));
    p.db = dtype == kF32 ? p.d : take(at, (size_t)ceil_div(g.T, 32) * 4 * p.width * 4);
    if (p.pieces * p.shares > 1) p.dx = take(at, (size_t)p.shares * g.T * g.D * 4);
    p.bytes = at;
    return p;
}

// ---- the products ---------------------------------------------------------------

template <class T>
struct PutLogits {
    float* c;
    const T* bias;
    long long ldc;
    LS_DEV void one(int i, int j, float v) const { c[i * ldc + j] = bias ? v + to_f(bias[j]) : v; }
};
// a row's pair of the tile's columns, and the target's logit
template <class T>
struct PutPairs {
    const T* bias;
    const int64_t* target;  // of the tile's first row
    long long j0;           // of its first column in the vocabulary
    int V;
    float2* pairs;          // of the tile's first row
    float* zt;
    LS_DEV void cell(int i, int j, float v, bool on) const {
        const float z = !on ? -__builtin_inff() : bias ? v + to_f(bias[j]) : v;
        float m = z;
        m = fmaxf(m, __uint_as_float(xor_lane<16>(__float_as_uint(m))));
        m = fmaxf(m, __uint_as_float(xor_lane<8>(__float_as_uint(m))));
        m = fmaxf(m, __uint_as_float(xor_lane<4>(__float_as_uint(m))));
        m = fmaxf(m, __uint_as_float(xor_lane<2>(__float_as_uint(m))));
        m = fmaxf(m, __uint_as_float(xor_lane<1>(__float_as_uint(m))));
        const float from = m == -__builtin_inff() ? 0.0f : m;
        float s = __builtin_amdgcn_exp2f((z - from) * kLog2e);
        s += __uint_as_float(xor_lane<16>(__float_as_uint(s)));
        s += __uint_as_float(xor_lane<8>(__float_as_uint(s)));
        s += __uint_as_float(xor_lane<4>(__float_as_uint(s)));
        s += __uint_as_float(xor_lane<2>(__float_as_uint(s)));
        s += __uint_as_float(xor_lane<1>(__float_as_uint(s)));
        if (!on) return;
        if (j == 0) pairs[i] = make_float2(m, s);
        if (target[i] == j0 + j) zt[i] = z;
    }
    LS_DEV void one(int, int, float) const {}
};
// d of a piece
template <class T>
struct PutD {
    T* d;
    const T* bias;
    const int64_t* target;  // of the tile's first row
    const float *lse, *g;
    long long ld, j0;
    LS_DEV float value(int i, int j, float v) const {
        const float z = bias ? v + to_f(bias[j]) : v, gt = g[i];
        const float p = __builtin_amdgcn_exp2f((z - lse[i]) * kLog2e);
        // an ignored row has no gradient, whatever its logits are
        const float e = gt == 0.0f ? 0.0f : (p - (target[i] == j0 + j ? 1.0f : 0.0f)) * gt;
        d[i * ld + j] = from_f<T>(e);
        return e;
    }
    LS_DEV void one(int i, int j, float v) const { value(i, j, v); }
};
// and its column sums, unrounded
template <class T>
struct PutDColumns : PutD<T> {
    float* db;  // the tile's partial rows
    LS_DEV void columns(int part, int j, float s) const { db[part * this->ld + j] = s; }
};
// (a row of dx whose g is 0 is 0, whatever the weights are)
struct PutPart {
    float* c;
    const float* g;
    long long ldc;
    bool add;
    LS_DEV void one(int i, int j, float v) const {
        if (g[i] == 0.0f) v = 0.0f;
        c[i * ldc + j] = add ? c[i * ldc + j] + v : v;
    }
};
template <class T>
struct PutOut {
    T* c;
    const float* g;  // of dW: null
    long long ldc;
    float unscale;
    LS_DEV void one(int i, int j, float v) const { c[i * ldc + j] = from_f<T>(g && g[i] == 0.0f ? 0.0f : v * unscale); }
};
// (eight at a time, one by one)
template <class P>
struct Each : P {
    int N;
    LS_DEV void eight(int i, int j, const float (&v)[8]) const {
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (j + r < N) P::one(i, j + r, v[r]);
    }
};

struct AnyProduct {
    const void *a, *b;
    int M, N, K, lda, ldb;
    void* c;
    long long ldc;
    const float* unscale;  // of rows
    int shares;            // of K: partial sums, M * N elements apart
    bool add;
    const float* g;        // of the rows, where c has a row for each
    // of logits
    const void* bias;
    const int64_t* target;
    const float* lse;
    float* db;             // partial rows of d's column sums: 2 of a tile of rows, or 4 of a shared one; may be null
    int v0, V;             // the piece's first column; the vocabulary
    float2* pairs;
    float* zt;
};
// What becomes of a product's sums: fp32 logits, pairs of the tile's columns, d;
// partial sums (of dx) or rows (of dx, of dW).
enum Use : int { kLogits, kPairs, kD, kPartDx, kDx, kDw };

template <class T, int USE, int B, bool SPLIT>
__global__ __launch_bounds__(kAnyThreads) void k_loss_any(AnyProduct g, long long tiles, int cols) {
    constexpr bool kA = USE != kDw, kB = USE <= kD;
    __shared__ __align__(128) char lds[2 * any_steps(SPLIT) * 2 * B * 64 * (SPLIT ? 4 : 1)];
    for (long long t = blockIdx.x; t < tiles * g.shares; t += gridDim.x) {
        const int share = (int)(t / tiles);
        const long long q = t % tiles;
        const int i0 = (int)(q / cols) * B, tj = (int)(q % cols), j0 = tj * B;
        const int k0 = (int)((long long)g.K * share / g.shares), k1 = (int)((long long)g.K * (share + 1) / g.shares);
        const T* a = (const T*)g.a + (kA ? (long long)i0 * g.lda + k0 : (long long)k0 * g.lda + i0);
        const T* b = (const T*)g.b + (kB ? (long long)j0 * g.ldb + k0 : (long long)k0 * g.ldb + j0);
        const T* bias = g.bias ? (const T*)g.bias + j0 : nullptr;
        const int64_t* target = g.target + i0;
        const long long to = (long long)i0 * g.ldc + j0, v0 = (long long)g.v0 + j0;
        auto sums = [&](const auto& put) {
            any_sums<T, kA, kB, B, SPLIT>(a, g.M - i0, g.lda, b, g.N - j0, g.ldb, k1 - k0, lds, put);
        };
        const int N = g.N - j0;
        if constexpr (USE == kLogits) {
            sums(Each<PutLogits<T>>{{(float*)g.c + to, bias, g.ldc}, N});
        } else if constexpr (USE == kPairs) {
            static_assert(SPLIT && B == 32);
            sums(Each<PutPairs<T>>{{bias, target, v0, g.V, g.pairs + (long long)tj * g.M + i0, g.zt + i0}, N});
        } else if constexpr (USE == kD) {
            const PutD<T> put{(T*)g.c + to, bias, target, g.lse + i0, g.g + i0, g.ldc, v0};
            if constexpr (sizeof(T) == 2) {
                if (g.db) sums(PutDColumns<T>{put, g.db + (long long)(i0 / B) * (SPLIT ? 4 : 2) * g.ldc + j0});
                else sums(Each<PutD<T>>{put, N});
            } else {
                sums(Each<PutD<T>>{put, N});
            }
        } else if constexpr (USE == kPartDx) {
            sums(Each<PutPart>{{(float*)g.c + (long long)share * g.M * g.ldc + to, g.g + i0, g.ldc, g.add}, N});
        } else {
            sums(Each<PutOut<T>>{{(T*)g.c + to, USE == kDx ? g.g + i0 : nullptr, g.ldc, *g.unscale}, N});
        }
        __syncthreads();
    }
}

template <int USE>
static void launch_any_product(int dtype, const AnyProduct& g, hipStream_t st) {
    if (g.M < 1 || g.N < 1) return;
    with_dtype(dtype, [&](auto tv) {
        using T = decltype(tv);
        auto launch = [&](auto bv, auto sv) {
            constexpr int B = bv.value;
            const long long cols = ceil_div(g.N, B), tiles = cols * ceil_div(g.M, B);
            hipLaunchKernelGGL((k_loss_any<T, USE, B, sv.value>), dim3(grid_of(tiles * g.shares)), dim3(kAnyThreads), 0,
                               st, g, tiles, (int)cols);
        };
        if constexpr (USE == kPairs) {
            launch(std::integral_constant<int, 32>{}, std::true_type{});
        } else {
            const int side = any_side(dtype, g.M, g.N, g.shares);
            constexpr bool k32 = sizeof(T) == 4;
            if (side == 128) launch(std::integral_constant<int, 128>{}, std::false_type{});
            // (the last piece of logits may have fewer tiles than the others)
            else if (side == 64 || USE == kLogits) launch(std::integral_constant<int, k32 ? 64 : 128>{}, std::false_type{});
            else if constexpr (USE != kLogits) launch(std::integral_constant<int, 32>{}, std::true_type{});
        }
    });
}

// the product of rows and a piece of the vocabulary
static AnyProduct any_piece(int dtype, const LossArgs& g, int v0, int n, void* c, long long ldc) {
    const size_t es = dtype_size(dtype);
    AnyProduct p{};
    p.a = g.x;
    p.b = (const char*)g.w + (size_t)v0 * g.D * es;
    p.bias = g.bias ? (const char*)g.bias + (size_t)v0 * es : nullptr;
    p.M = g.T, p.N = n, p.K = g.D, p.lda = g.D, p.ldb = g.D;
    p.c = c, p.ldc = ldc;
    p.shares = 1;
    p.target = g.target;
    p.v0 = v0, p.V = g.V;
    return p;
}

// ---- rows of logits ---------------------------------------------------------------

// Adds b's maximum and sum of exponentials about it to a's.
struct MaxSum {
    float m, s;
};
LS_DEV MaxSum merge(MaxSum a, MaxSum b) {
    const float m = fmaxf(a.m, b.m);
    // nothing but -inf so far (or a sum that is NaN: it stays)
    const float ea = a.m == m ? a.s : a.s * __builtin_amdgcn_exp2f((a.m - m) * kLog2e);
    const float eb = b.m == m ? b.s : b.s * __builtin_amdgcn_exp2f((b.m - m) * kLog2e);
    return {m, ea + eb};
}
template <int D>
LS_DEV MaxSum merge_lanes(MaxSum a) {
    return merge(a, {__uint_as_float(xor_lane<D>(__float_as_uint(a.m))), __uint_as_float(xor_lane<D>(__float_as_uint(a.s)))});
}

// A row of a piece, one workgroup: its pair, and the target's logit.  The row is
// read twice, the second time from the caches.
__global__ __launch_bounds__(256) void k_loss_part(const float* __restrict__ z, const int64_t* __restrict__ target,
                                                   int T, int V, int v0, int n, int ld, float2* __restrict__ pairs,
                                                   float* __restrict__ zt) {
    __shared__ MaxSum s[4];
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        const float* row = z + (long long)t * ld;
        MaxSum a{-__builtin_inff(), 0.0f};
#pragma unroll 4
        for (int c = threadIdx.x; c < n; c += 256) a.m = fmaxf(a.m, row[c]);
        const float from = a.m == -__builtin_inff() ? 0.0f : a.m;
#pragma unroll 4
        for (int c = threadIdx.x; c < n; c += 256) a.s += __builtin_amdgcn_exp2f((row[c] - from) * kLog2e);
        a = merge_lanes<32>(a);
        a = merge_lanes<16>(a);
        a = merge_lanes<8>(a);
        a = merge_lanes<4>(a);
        a = merge_lanes<2>(a);
        a = merge_lanes<1>(a);
        if (lane_id() == 0) s[threadIdx.x >> 6] = a;
        __syncthreads();
        if (threadIdx.x == 0) {
            a = merge(merge(s[0], s[1]), merge(s[2], s[3]));
            pairs[t] = make_float2(a.m, a.s);
            const int64_t at = target[t] - v0;
            if (target[t] >= 0 && target[t] < V && at >= 0 && at < n) zt[t] = row[at];
        }
        __syncthreads();
    }
}

// ---- rows and sums -------------------------------------------------------------------

// A row's pairs merged, 16 rows a workgroup and 16 lanes a row.
__global__ __launch_bounds__(256) void k_loss_rows(const float2* __restrict__ pairs, int parts,
                                                   const int64_t* __restrict__ target, const float* __restrict__ zt,
                                                   int T, int V, float* __restrict__ loss, float* __restrict__ lse) {
    __shared__ MaxSum s[16][17];
    const int r = threadIdx.x & 15, q = threadIdx.x >> 4;
    for (long long t0 = (long long)blockIdx.x * 16; t0 < T; t0 += (long long)gridDim.x * 16) {
        const long long t = t0 + r;
        MaxSum a{-__builtin_inff(), 0.0f};
        if (t < T) {
            int p = q;
            for (; p + 7 * 16 < parts; p += 8 * 16) {
                float2 v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) v[u] = pairs[(long long)(p + u * 16) * T + t];
#pragma unroll
                for (int u = 0; u < 8; ++u) a = merge(a, {v[u].x, v[u].y});
            }
            for (; p < parts; p += 16) {
                const float2 v = pairs[(long long)p * T + t];
                a = merge(a, {v.x, v.y});
            }
        }
        s[q][r] = a;
        __syncthreads();
        if (q == 0 && t < T) {
#pragma unroll
            for (int i = 1; i < 16; ++i) a = merge(a, s[i][r]);
            const float l = a.m + logf(a.s);
            if (lse) lse[t] = l;
            if (loss) loss[t] = target[t] >= 0 && target[t] < V ? l - zt[t] : 0.0f;
        }
        __syncthreads();
    }
}

void launch_loss_rows(const LossArgs& g, const LossParts& p, char* scratch, float* loss, float* lse, hipStream_t st) {
    if (g.T < 1) return;
    hipLaunchKernelGGL(k_loss_rows, dim3(grid_of(ceil_div(g.T, 16))), dim3(256), 0, st,
                       (const float2*)(scratch + p.pairs), p.parts, g.target, (const float*)(scratch + p.zt), g.T, g.V,
                       loss, lse);
}

// Sum or mean of the rows' losses, one workgroup: fp64 lanes' sums, in the
// order of the lanes.
__global__ __launch_bounds__(1024) void k_loss_reduce(const float* __restrict__ loss, const int64_t* __restrict__ target,
                                                      int T, int V, int mean, float* __restrict__ out) {
    __shared__ double s[16], c[16];
    double sum = 0.0, count = 0.0;
    for (int t = threadIdx.x; t < T; t += 1024) {
        sum += (double)loss[t];
        count += target[t] >= 0 && target[t] < V ? 1.0 : 0.0;
    }
    sum = wave_sum(sum);
    count = wave_sum(count);
    if (lane_id() == 0) s[threadIdx.x >> 6] = sum, c[threadIdx.x >> 6] = count;
    __syncthreads();
    if (threadIdx.x) return;
    for (int i = 1; i < 16; ++i) sum += s[i], count += c[i];
    *out = (float)(mean ? sum / (count > 0.0 ? count : 1.0) : sum);
}
void launch_loss_reduce(const LossArgs& g, const float* loss, int reduction, float* out, hipStream_t st) {
    hipLaunchKernelGGL(k_loss_reduce, dim3(1), dim3(1024), 0, st, loss, g.target, g.T, g.V, reduction == kReduceMean,
                       out);
}

// The gradient of every row's loss over the largest one's magnitude, 0 for an
// ignored row; behind them what the products are multiplied by again.  One
// workgroup.  So d is p - onehot itself where all rows have one gradient, and is
// rounded row by row (times a common factor, the factor's rounding was in all
// rows alike: up to 2^-9 of dx and dW in bf16).  In fp16 times 2^13, which keeps
// small shares of the softmax above the type's least numbers.
//
// The other workgroups copy x to `live` for dW's sums, with zeros in the rows
// whose loss has no gradient: their d is 0, but 0 times what they hold is NaN
// where that is not finite.  (A launch of their own took 3 us.)
template <class T>
__global__ __launch_bounds__(1024) void k_loss_grad_rows(LossArgs a, const float* __restrict__ dloss, int reduction,
                                                         float* __restrict__ g, int packs, T* __restrict__ live) {
    const auto on = [&](long long t) { return a.target[t] >= 0 && a.target[t] < a.V; };
    const auto at = [&](long long t) { return dloss[reduction == kReduceNone ? t : 0]; };
    if (blockIdx.x > 0) {
        const long long n = (long long)packs * a.T;
        for (long long i = (long long)(blockIdx.x - 1) * 1024 + threadIdx.x; i < n; i += (long long)(gridDim.x - 1) * 1024) {
            const long long t = i / packs;
            const int c = (int)(i - t * packs) * Pack<T>::V;
            Pack<T> v{};
            if (on(t) && at(t) != 0.0f) v = ld<false>((const T*)a.x + t * a.D, c, a.D);
            st<T>(live + t * a.D, c, a.D, v);
        }
        return;
    }
    __shared__ uint32_t s[16], c[16];
    uint32_t top = 0, count = 0;
    for (int t = threadIdx.x; t < a.T; t += 1024) {
        count += on(t);
        // finite magnitudes, ordered as their bits
        const uint32_t u = __float_as_uint(at(t)) & 0x7FFFFFFFu;
        if (on(t) && u < 0x7F800000u) top = max(top, u);
    }
    count = (uint32_t)wave_sum_u64(count);
    top = wave_max_u32(top);
    if (lane_id() == 0) s[threadIdx.x >> 6] = top, c[threadIdx.x >> 6] = count;
    __syncthreads();
    for (int i = 0; i < 16; ++i) top = max(top, s[i]);
    count = 0;
    for (int i = 0; i < 16; ++i) count += c[i];
    const float div = reduction == kReduceMean ? (float)max(count, 1u) : 1.0f;
    const float most = top ? __uint_as_float(top) : 1.0f, scale = std::is_same_v<T, _Float16> ? 8192.0f : 1.0f;
    for (int t = threadIdx.x; t < a.T; t += 1024) g[t] = on(t) ? at(t) / most * scale : 0.0f;
    if (threadIdx.x == 0) g[a.T] = most / div / scale;
}
void launch_loss_grad_rows(int dtype, const LossArgs& g, const float* dloss, int reduction, float* rows, void* live,
                           hipStream_t st) {
    with_dtype(dtype, [&](auto tv) {
        using X = decltype(tv);
        const long long packs = ceil_div(g.D, Pack<X>::V), n = live ? packs * g.T : 0;
        hipLaunchKernelGGL(k_loss_grad_rows<X>, dim3((unsigned)(1 + std::min(ceil_div(n, 1024), 1ll << 16))), dim3(1024),
                           0, st, g, dloss, reduction, rows, (int)packs, (X*)live);
    });
}

// Column sums of a piece's partial rows, 64 columns a workgroup: a wave adds every
// sixteenth row, and the waves' sums are added in wave order.
template <class T>
__global__ __launch_bounds__(1024) void k_loss_db(const float* __restrict__ part, int ld, int rows, int n,
                                                  const float* __restrict__ unscale, T* __restrict__ db) {
    __shared__ float s[16][64];
    const int l = lane_id(), w = uniform(threadIdx.x >> 6), c = blockIdx.x * 64 + l;
    float sum = 0.0f;
    if (c < n) {
#pragma unroll 8
        for (int t = w; t < rows; t += 16) sum += part[(long long)t * ld + c];
    }
    s[w][l] = sum;
    __syncthreads();
    if (w || c >= n) return;
    for (int i = 1; i < 16; ++i) sum += s[i][l];
    db[c] = from_f<T>(sum * *unscale);
}
void launch_loss_db(int dtype, const float* part, int ld, int rows, int n, const float* unscale, void* db,
                    hipStream_t st) {
    with_dtype(dtype, [&](auto tv) {
        using X = decltype(tv);
        hipLaunchKernelGGL(k_loss_db<X>, dim3((unsigned)ceil_div(n, 64)), dim3(1024), 0, st, part, ld, rows, n,
                           unscale, (X*)db);
    });
}

// dx from its shares' partial sums, in their order
template <class T>
__global__ __launch_bounds__(256) void k_loss_dx(const float* __restrict__ part, int shares, long long n,
                                                 const float* __restrict__ unscale, T* __restrict__ dx) {
    const float u = *unscale;
    for (long long i = ((long long)blockIdx.x * 256 + threadIdx.x); i < n; i += (long long)gridDim.x * 256) {
        float sum = part[i];
        for (int s = 1; s < shares; ++s) sum += part[(long long)s * n + i];
        dx[i] = from_f<T>(sum * u);
    }
}
void launch_loss_dx(int dtype, const float* part, int shares, long long n, const float* unscale, void* dx,
                    hipStream_t st) {
    if (n < 1) return;
    with_dtype(dtype, [&](auto tv) {
        using X = decltype(tv);
        hipLaunchKernelGGL(k_loss_dx<X>, dim3((unsigned)std::min(ceil_div(n, 256), 1ll << 16)), dim3(256), 0, st, part,
                           shares, n, unscale, (X*)dx);
    });
}

// ---- the passes --------------------------------------------------------------------

void launch_loss_any(int dtype, const LossArgs& g, const LossParts& p, char* scratch, hipStream_t st) {
    float2* pairs = (float2*)(scratch + p.pairs);
    float* zt = (float*)(scratch + p.zt);
    if (g.T < 1) return;
    if (!p.logits) {
        AnyProduct q = any_piece(dtype, g, 0, g.V, nullptr, 0);
        q.pairs = pairs;
        q.zt = zt;
        launch_any_product<kPairs>(dtype, q, st);
        return;
    }
    float* logits = (float*)(scratch + p.logits);
    for (int i = 0; i < p.parts; ++i) {
        const int v0 = i * p.width, n = std::min(p.width, g.V - v0);
        launch_any_product<kLogits>(dtype, any_piece(dtype, g, v0, n, logits, p.width), st);
        hipLaunchKernelGGL(k_loss_part, dim3(grid_of(g.T)), dim3(256), 0, st, logits, g.target, g.T, g.V, v0, n, p.width,
                           pairs + (long long)i * g.T, zt);
    }
}

void launch_loss_any_vjp(int dtype, const LossArgs& g, const LossVjpPlan& p, const float* lse, char* scratch, void* dx,
                         void* dw, void* db, hipStream_t st) {
    const size_t es = dtype_size(dtype);
    float* rows = (float*)(scratch + p.g);
    const float* unscale = rows + g.T;
    const bool part = p.pieces * p.shares > 1;
    for (int i = 0; i < p.pieces; ++i) {
        const int v0 = i * p.width, n = std::min(p.width, g.V - v0);
        AnyProduct z = any_piece(dtype, g, v0, n, scratch + p.d, p.ld);
        z.lse = lse;
        z.g = rows;
        // (fp32's d is not rounded: its own rows)
        z.db = db && dtype != kF32 ? (float*)(scratch + p.db) : nullptr;
        launch_any_product<kD>(dtype, z, st);
        const int side = any_side(dtype, g.T, n, 1);
        const long long parts = dtype == kF32 ? g.T : ceil_div(g.T, side) * (side > 32 ? 2 : 4);
        if (db) launch_loss_db(dtype, (const float*)(scratch + p.db), p.ld, (int)parts, n, unscale, (char*)db + (size_t)v0 * es, st);
        AnyProduct q{};
        q.a = scratch + p.d;
        q.lda = p.ld;
        q.g = rows;
        q.unscale = unscale;
        if (dx) {
            q.b = (const char*)g.w + (size_t)v0 * g.D * es;
            q.M = g.T, q.N = g.D, q.K = n, q.ldb = g.D, q.ldc = g.D;
            q.c = part ? scratch + p.dx : dx;
            q.shares = p.shares;
            q.add = i > 0;
            if (part) launch_any_product<kPartDx>(dtype, q, st);
            else launch_any_product<kDx>(dtype, q, st);
        }
        if (dw) {
            q.b = scratch + p.x;
            q.M = n, q.N = g.D, q.K = g.T, q.ldb = g.D, q.ldc = g.D;
            q.c = (char*)dw + (size_t)v0 * g.D * es;
            q.shares = 1;
            launch_any_product<kDw>(dtype, q, st);
        }
    }
    if (dx && part) launch_loss_dx(dtype, (const float*)(scratch + p.dx), p.shares, (long long)g.T * g.D, unscale, dx, st);
}

}  // namespace lapsum
