// Layer norm of rows and its gradients.
//
// Mathematics: mu = mean of a row's x, s = 1 / sqrt(mean of (x - mu)^2 + eps),
// xh = (x - mu) s, y = xh w + b.  With g = dy w:
//   dx = s (g - mean(g) - xh mean(g xh)),  dw = sum of dy xh over the rows,
//   db = sum of dy over them.
//
// A row belongs to one wave (narrow rows) or one workgroup, whose threads hold
// it in registers, U packs of 16 bytes each: it is read once, and its mean and
// centred squares come from registers.  A wave takes the squares about its own
// mean, and with them the sum of the differences, which is what the mean's
// rounding left (so a row of one value has that mean, and its y is the bias); the
// waves' counts, means and squares are merged afterwards, in one exchange
// through LDS, and no squares of uncentred values are subtracted.  Values are
// summed under a power of two, so the mean of finite values is finite; where the
// sum of the squares passes float32's range, they are summed again under another,
// so a variance is infinite only where it is past that range itself.  rstd and xh
// are 0 then, and y is the bias.
//
// Workgroups walk the rows with the next row's loads in flight;
// weight and bias stay in registers meanwhile, and so do the sums for their
// gradients, which leave as one row of partial sums a workgroup.  k_norm_sum
// adds those in their order: no atomics.
//
// Statistics, sums and partial sums are fp32.  The row's own rounding to 16
// bits happens once, at the store.
//
// Memory bounds it: 16384 rows of 4096 in bf16 with fp32 weights, 268 MB, 49 to 55
// us back to back (4.9 to 5.5 TB/s); its gradients, 403 MB, 70 to 77 us (5.2 to 5.8
// TB/s) of which k_norm_sum is 5 to 7.  1000 rows of 1001 in fp32: 4.8 and 10 us,
// latencies of a row's loads and of the sums after each other.  2000 rows of 32768 in
// bf16, past registers: 151 us (131 MB read three times and written) and 254.
#include "lapsum_layer_ops.h"
#include "lapsum_rows.h"

namespace lapsum {

constexpr int kNormWide = 1024;  // threads of a row that registers do not hold

// (a launch counts its threads in 32 bits)
static unsigned wide_grid(long long n) { return (unsigned)std::min(n, kGridMax / 4); }

// What values are summed times: those of a row in registers (2^14 at most), and of
// any row (2^31); and those whose squares are summed again.
constexpr float kDown = 0x1p-16f, kUp = 0x1p16f;
constexpr float kDownWide = 0x1p-32f, kUpWide = 0x1p32f;
constexpr float kDownSquares = 0x1p-84f, kUpSquares = 0x1p84f;

// Whether sums over a row in registers can pass float32's range.
template <class T>
constexpr bool kFar = !std::is_same_v<T, _Float16>;

// What a row's values are taken about once its variance is known: its mean, or 0
// where rstd is 0 (differences from such a row's mean may be infinite).
LS_DEV float about(float mean, float rstd) { return rstd == 0.0f ? 0.0f : mean; }

// The squares about a mean that was off by left / n, about the right one: in
// their rounding where they cancel, infinite where they pass float32's range.
LS_DEV float centred(float sq, float left, float inv) {
    return sq < __builtin_inff() ? fmaxf(sq - left * (left * inv), 0.0f) : sq;
}

// Adds `a` and `b` over the NT threads that share a row.  s: LDS of the two
// sums of every wave, taken in turn by `flip`, so that one barrier is enough.
template <int NT>
LS_DEV void row_sums(float& a, float& b, float (*s)[2][16], int& flip) {
    a = wave_sum_f32(a);
    b = wave_sum_f32(b);
    if constexpr (NT > 64) {
        const int w = threadIdx.x >> 6;
        if (lane_id() == 0) {
            s[flip][0][w] = a;
            s[flip][1][w] = b;
        }
        __syncthreads();
        a = s[flip][0][0];
        b = s[flip][1][0];
#pragma unroll
        for (int i = 1; i < NT / 64; ++i) {
            a += s[flip][0][i];
            b += s[flip][1][i];
        }
        flip ^= 1;
    }
}

// Mean and sum of squares about it over the NT threads that share a row: each
// wave has those of its n elements.
template <int NT>
LS_DEV void row_moments(float& mean, float& sq, float n, float D, float (*s)[2][16], float* count, int& flip) {
    if constexpr (NT > 64) {
        const int w = threadIdx.x >> 6;
        if (lane_id() == 0) {
            s[flip][0][w] = mean;
            s[flip][1][w] = sq;
            count[w] = n;  // the same for every row
        }
        __syncthreads();
        // about the first wave's, so that equal means stay as they are
        const float first = s[flip][0][0];
        float sum = 0.0f;
#pragma unroll
        for (int i = 1; i < NT / 64; ++i)
            sum = fmaf(s[flip][0][i] * 0.5f - first * 0.5f, count[i] * (2.0f * kDown), sum);
        mean = fmaf(sum / D, kUp, first);
        sq = 0.0f;
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) {
            const float d = s[flip][0][i] - mean;
            // a wave past the row's end has no elements
            sq += count[i] > 0.0f ? fmaf(d * d, count[i], s[flip][1][i]) : 0.0f;
        }
        flip ^= 1;
    }
}

// V elements from column c of a row of D weights, as floats; `none` where
// there are none.  (One load an element instead of 16 bytes: 16384 rows of 4096
// with fp32 weights 69 us in place of 59, its gradients 84 in place of 77.)
template <class W, int V>
LS_DEV void weights(float (&v)[V], const W* __restrict__ w, long long c, long long D, float none) {
    constexpr int P = V < Pack<W>::V ? V : Pack<W>::V;
    struct __attribute__((packed, aligned(sizeof(W)))) Few {
        W v[P];
    };
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = none;
    if (!w) return;
#pragma unroll
    for (int p = 0; p < V; p += P) {
        if (c + p + P <= D) {
            const Few x = *reinterpret_cast<const Few*>(w + c + p);
#pragma unroll
            for (int i = 0; i < P; ++i) v[p + i] = to_f(x.v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (c + p + i < D) v[p + i] = to_f(w[c + p + i]);
        }
    }
}

template <class T, class W, int NT, int U>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_norm(const T* __restrict__ x, const W* __restrict__ weight,
                                                              const W* __restrict__ bias, long long rows, long long D,
                                                              float eps, T* __restrict__ y, float* __restrict__ mean_out,
                                                              float* __restrict__ rstd_out) {
    constexpr int V = Pack<T>::V, kRows = NT < 256 ? 256 / NT : 1;
    __shared__ float s[2][2][16], count[16];
    const int tid = threadIdx.x % NT, sub = threadIdx.x / NT;
    float w[U][V], b[U][V];
    int mine = 0;  // elements of a row that this thread holds
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long c = (long long)(u * NT + tid) * V;
        weights<W, V>(w[u], weight, c, D, 1.0f);
        weights<W, V>(b[u], bias, c, D, 0.0f);
        mine += (int)min(max(D - c, 0ll), (long long)V);
    }
    const int held = mine;
    const float n = wave_sum_f32((float)mine), inv = 1.0f / fmaxf(n, 1.0f);
    int flip = 0;
    Pack<T> next[U];
    const long long stride = (long long)gridDim.x * kRows;
    long long r = (long long)blockIdx.x * kRows + sub;
    auto load = [&](long long row) {
#pragma unroll
        for (int u = 0; u < U; ++u) next[u] = take<false>(x + row * D, (long long)(u * NT + tid) * V, D);
    };
    if (r < rows) load(r);
    for (; r < rows; r += stride) {
        float v[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Pack<T> p = settle(next[u], (long long)(u * NT + tid) * V, D);
#pragma unroll
            for (int i = 0; i < V; ++i) v[u][i] = to_f(p.v[i]);
        }
        if (r + stride < rows) load(r + stride);
        float sum = 0.0f;  // (past the row's end the packs hold zeros)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i) sum = fmaf(v[u][i], kDown, sum);
        float mean = wave_sum_f32(sum) * (inv * kUp), sq = 0.0f, left = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int n_u = min(max(held - u * V, 0), V);
            if (n_u == V) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = v[u][i] - mean;
                    sq = fmaf(d, d, sq);
                    left += d;
                }
            } else {  // the row's end
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = i < n_u ? v[u][i] - mean : 0.0f;
                    sq = fmaf(d, d, sq);
                    left += d;
                }
            }
        }
        left = wave_sum_f32(left);
        // (differences that overflow leave the mean as it is)
        mean = !kFar<T> || fabsf(left) < __builtin_inff() ? fmaf(left, inv, mean) : mean;
        sq = centred(wave_sum_f32(sq), left, inv);
        row_moments<NT>(mean, sq, n, (float)D, s, count, flip);
        float var = sq / (float)D;
        // (the same for the row's threads)
        if (kFar<T> && uniform(!(sq < __builtin_inff()))) {
            float again = 0.0f, none = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = u * V + i < held ? fmaf(v[u][i], kDownSquares, -mean * kDownSquares) : 0.0f;
                    again = fmaf(d, d, again);
                }
            row_sums<NT>(again, none, s, flip);
            var = again / (float)D * kUpSquares * kUpSquares;
        }
        const float rstd = 1.0f / sqrtf(var + eps);
        if (tid == 0) {
            if (mean_out) mean_out[r] = mean;
            if (rstd_out) rstd_out[r] = rstd;
        }
        if (kFar<T>) mean = about(mean, rstd);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Pack<T> o;
#pragma unroll
            for (int i = 0; i < V; ++i) o.v[i] = from_f<T>(fmaf((v[u][i] - mean) * rstd, w[u][i], b[u][i]));
            st<T>(y + r * D, (long long)(u * NT + tid) * V, D, o);
        }
    }
}

// Rows wider than registers hold: read three times, twice of them from caches.
template <class T, class W>
__global__ __launch_bounds__(kNormWide) void k_norm_wide(const T* __restrict__ x, const W* __restrict__ weight,
                                                         const W* __restrict__ bias, long long rows, long long D,
                                                         float eps, T* __restrict__ y, float* __restrict__ mean_out,
                                                         float* __restrict__ rstd_out) {
    constexpr int V = Pack<T>::V, kStep = kNormWide * V;
    __shared__ float s[2][2][16];
    int flip = 0;
    for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* row = x + r * D;
        float sum = 0.0f, none = 0.0f;
        for (long long c = (long long)threadIdx.x * V; c < D; c += kStep) {
            const Pack<T> p = ld<false>(row, c, D);
#pragma unroll
            for (int i = 0; i < V; ++i) sum = fmaf(to_f(p.v[i]), kDownWide, sum);
        }
        row_sums<kNormWide>(sum, none, s, flip);
        float mean = sum / (float)D * kUpWide, sq = 0.0f, left = 0.0f;
        for (long long c = (long long)threadIdx.x * V; c < D; c += kStep) {
            const Pack<T> p = ld<false>(row, c, D);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = c + i < D ? to_f(p.v[i]) - mean : 0.0f;
                sq = fmaf(d, d, sq);
                left += d;
            }
        }
        row_sums<kNormWide>(sq, left, s, flip);
        if (fabsf(left) < __builtin_inff()) mean += left / (float)D;
        sq = centred(sq, left, 1.0f / (float)D);
        float var = sq / (float)D;
        if (!(sq < __builtin_inff())) {
            float again = 0.0f;
            for (long long c = (long long)threadIdx.x * V; c < D; c += kStep) {
                const Pack<T> p = ld<false>(row, c, D);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = c + i < D ? fmaf(to_f(p.v[i]), kDownSquares, -mean * kDownSquares) : 0.0f;
                    again = fmaf(d, d, again);
                }
            }
            row_sums<kNormWide>(again, none, s, flip);
            var = again / (float)D * kUpSquares * kUpSquares;
        }
        const float rstd = 1.0f / sqrtf(var + eps);
        if (threadIdx.x == 0) {
            if (mean_out) mean_out[r] = mean;
            if (rstd_out) rstd_out[r] = rstd;
        }
        mean = about(mean, rstd);
        for (long long c = (long long)threadIdx.x * V; c < D; c += kStep) {
            const Pack<T> p = ld<false>(row, c, D);
            float w[V], b[V];
            weights<W, V>(w, weight, c, D, 1.0f);
            weights<W, V>(b, bias, c, D, 0.0f);
            Pack<T> o;
#pragma unroll
            for (int i = 0; i < V; ++i) o.v[i] = from_f<T>(fmaf((to_f(p.v[i]) - mean) * rstd, w[i], b[i]));
            st<T>(y + r * D, c, D, o);
        }
    }
}

// dx (may be null), and the partial sums of dw and db (may be null): row
// blockIdx.x of gridDim.x of each, db's behind dw's.
template <class T, class W, int NT, int U>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_norm_vjp(const T* __restrict__ x, const W* __restrict__ weight,
                                                                  const float* __restrict__ mean_in,
                                                                  const float* __restrict__ rstd_in,
                                                                  const T* __restrict__ dy, long long rows, long long D,
                                                                  T* __restrict__ dx, float* __restrict__ part) {
    constexpr int V = Pack<T>::V, kRows = NT < 256 ? 256 / NT : 1;
    __shared__ float s[2][2][16];
    __shared__ float meet[kRows > 1 ? kRows : 1][kRows > 1 ? NT * V : 1];
    const int tid = threadIdx.x % NT, sub = threadIdx.x / NT;
    float w[U][V], dw[U][V] = {}, db[U][V] = {};
    auto load_weights = [&] {
#pragma unroll
        for (int u = 0; u < U; ++u) weights<W, V>(w[u], weight, (long long)(u * NT + tid) * V, D, 1.0f);
    };
    const float inv = 1.0f / (float)D;
    int flip = 0;
    Pack<T> nx[U], ng[U];
    float nm = 0.0f, ns = 0.0f;
    const long long stride = (long long)gridDim.x * kRows;
    long long r = (long long)blockIdx.x * kRows + sub;
    auto load = [&](long long row) {
        nm = mean_in[row];
        ns = rstd_in[row];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            nx[u] = take<true>(x + row * D, (long long)(u * NT + tid) * V, D);
            ng[u] = take<true>(dy + row * D, (long long)(u * NT + tid) * V, D);
        }
    };
    // the widest rows leave no registers for the next one's and for weights
    // (4096 rows of 16384 in bf16: 150 us with both, 119 with neither)
    constexpr bool kAhead = U < 4;
    if (kAhead) load_weights();
    if (kAhead && r < rows) load(r);
    for (; r < rows; r += stride) {
        if (!kAhead) load(r), load_weights();
        float xh[U][V], g[U][V];
        const float rstd = ns, mean = about(nm, rstd);
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long c = (long long)(u * NT + tid) * V;
            const Pack<T> px = settle(nx[u], c, D), pg = settle(ng[u], c, D);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                // (past the row's end dy is 0)
                xh[u][i] = (to_f(px.v[i]) - mean) * rstd;
                const float d = to_f(pg.v[i]);
                dw[u][i] = fmaf(d, xh[u][i], dw[u][i]);
                db[u][i] += d;
                g[u][i] = d * w[u][i];
                s1 += g[u][i];
                s2 = fmaf(g[u][i], xh[u][i], s2);
            }
        }
        if (kAhead && r + stride < rows) load(r + stride);
        if (!dx) continue;
        row_sums<NT>(s1, s2, s, flip);
        s1 *= inv;
        s2 *= inv;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Pack<T> o;
#pragma unroll
            for (int i = 0; i < V; ++i) o.v[i] = from_f<T>(rstd * (g[u][i] - fmaf(xh[u][i], s2, s1)));
            st<T>(dx + r * D, (long long)(u * NT + tid) * V, D, o);
        }
    }
    if (!part) return;
    // the workgroup's sums: of one row of threads, or added over them in order
    for (int which = 0; which < 2; ++which) {
        float* to = part + ((long long)which * gridDim.x + blockIdx.x) * D;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float(&a)[V] = which ? db[u] : dw[u];
            if constexpr (kRows > 1) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < V; ++i) meet[sub][i * NT + tid] = a[i];
                __syncthreads();
                if (sub) continue;
#pragma unroll
                for (int q = 1; q < kRows; ++q)
#pragma unroll
                    for (int i = 0; i < V; ++i) a[i] += meet[q][i * NT + tid];
            }
            const long long c = (long long)(u * NT + tid) * V;
#pragma unroll
            for (int p = 0; p < V; p += 4) {
                const Pack<float> o{{a[p], a[p + 1], a[p + 2], a[p + 3]}};
                st<float>(to, c + p, D, o);
            }
        }
    }
}

// dx of rows wider than registers hold: x and dy are read twice
template <class T, class W>
__global__ __launch_bounds__(kNormWide) void k_norm_vjp_wide(const T* __restrict__ x, const W* __restrict__ weight,
                                                             const float* __restrict__ mean_in,
                                                             const float* __restrict__ rstd_in,
                                                             const T* __restrict__ dy, long long rows, long long D,
                                                             T* __restrict__ dx) {
    constexpr int V = Pack<T>::V, kStep = kNormWide * V;
    __shared__ float s[2][2][16];
    int flip = 0;
    for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
        const float rstd = rstd_in[r], mean = about(mean_in[r], rstd);
        float s1 = 0.0f, s2 = 0.0f;
        auto pass = [&](auto&& f) {
            for (long long c = (long long)threadIdx.x * V; c < D; c += kStep) {
                const Pack<T> px = ld<false>(x + r * D, c, D), pg = ld<false>(dy + r * D, c, D);
                float w[V], xh[V], g[V];
                weights<W, V>(w, weight, c, D, 1.0f);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    xh[i] = (to_f(px.v[i]) - mean) * rstd;
                    g[i] = to_f(pg.v[i]) * w[i];
                }
                f(c, xh, g);
            }
        };
        pass([&](long long, const float (&xh)[V], const float (&g)[V]) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s1 += g[i];
                s2 = fmaf(g[i], xh[i], s2);
            }
        });
        row_sums<kNormWide>(s1, s2, s, flip);
        s1 /= (float)D;
        s2 /= (float)D;
        pass([&](long long c, const float (&xh)[V], const float (&g)[V]) {
            Pack<T> o;
#pragma unroll
            for (int i = 0; i < V; ++i) o.v[i] = from_f<T>(rstd * (g[i] - fmaf(xh[i], s2, s1)));
            st<T>(dx + r * D, c, D, o);
        });
    }
}
// their partial sums of dw and db: a thread a column, gridDim.y shares of the rows
template <class T>
__global__ __launch_bounds__(256) void k_norm_dw_wide(const T* __restrict__ x, const float* __restrict__ mean_in,
                                                      const float* __restrict__ rstd_in, const T* __restrict__ dy,
                                                      long long rows, long long D, float* __restrict__ part) {
    for (long long c = (long long)blockIdx.x * 256 + threadIdx.x; c < D; c += (long long)gridDim.x * 256) {
        float dw = 0.0f, db = 0.0f;
#pragma unroll 4
        for (long long r = blockIdx.y; r < rows; r += gridDim.y) {
            const float d = to_f(dy[r * D + c]);
            dw = fmaf(d, (to_f(x[r * D + c]) - about(mean_in[r], rstd_in[r])) * rstd_in[r], dw);
            db += d;
        }
        part[(long long)blockIdx.y * D + c] = dw;
        part[((long long)gridDim.y + blockIdx.y) * D + c] = db;
    }
}

// dw (blockIdx.y = 0) and db from their n partial rows, 64 columns a
// workgroup: a wave adds every sixteenth row, and the waves' sums are added in
// wave order
template <class W>
__global__ __launch_bounds__(1024) void k_norm_sum(const float* __restrict__ part, int n, long long D,
                                                   W* __restrict__ dw, W* __restrict__ db) {
    __shared__ float s[16][64];
    W* to = blockIdx.y ? db : dw;
    if (!to) return;
    const float* p = part + (long long)blockIdx.y * n * D;
    const int l = lane_id(), w = uniform(threadIdx.x >> 6);
    for (long long c0 = (long long)blockIdx.x * 64; c0 < D; c0 += (long long)gridDim.x * 64) {
        const long long c = c0 + l;
        float sum = 0.0f;
        if (c < D) {
#pragma unroll 8
            for (int i = w; i < n; i += 16) sum += p[(long long)i * D + c];
        }
        s[w][l] = sum;
        __syncthreads();
        if (w == 0 && c < D) {
#pragma unroll
            for (int i = 1; i < 16; ++i) sum += s[i][l];
            to[c] = from_f<W>(sum);
        }
        __syncthreads();
    }
}

// calls f with the threads that share a row and the packs each holds, or
// (0, 0) where registers do not hold it
template <class T, class F>
static void with_shape(long long D, F&& f) {
    constexpr int V = Pack<T>::V;
    const long long packs = ceil_div(D, V);
    auto is = [&](auto nt, auto u) {
        if (packs > nt.value * u.value) return false;
        f(nt, u);
        return true;
    };
    using std::integral_constant;
    is(integral_constant<int, 64>{}, integral_constant<int, 1>{}) ||
        is(integral_constant<int, 64>{}, integral_constant<int, 2>{}) ||
        is(integral_constant<int, 256>{}, integral_constant<int, 1>{}) ||
        is(integral_constant<int, 256>{}, integral_constant<int, 2>{}) ||
        is(integral_constant<int, 512>{}, integral_constant<int, 2>{}) ||
        is(integral_constant<int, 512>{}, integral_constant<int, 4>{}) ||
        (f(integral_constant<int, 0>{}, integral_constant<int, 0>{}), true);
}

// weights have the rows' type or fp32
template <class F>
static void with_types(int dtype, int wtype, F&& f) {
    with_dtype(dtype, [&](auto tv) {
        if (wtype == kF32) f(tv, float{});
        else f(tv, tv);
    });
}

void launch_norm(const void* x, const void* weight, const void* bias, int dtype, int wtype, long long rows, long long D,
                 float eps, void* y, float* mean, float* rstd, hipStream_t st) {
    with_types(dtype, wtype, [&](auto tv, auto wv) {
        using T = decltype(tv);
        using W = decltype(wv);
        with_shape<T>(D, [&](auto nt, auto u) {
            constexpr int NT = nt.value, U = u.value;
            if constexpr (NT == 0) {
                hipLaunchKernelGGL((k_norm_wide<T, W>), dim3(wide_grid(rows)), dim3(kNormWide), 0, st, (const T*)x,
                                   (const W*)weight, (const W*)bias, rows, D, eps, (T*)y, mean, rstd);
            } else {
                constexpr int kRows = NT < 256 ? 256 / NT : 1;
                // the workgroups that are resident at once, or nearly (16384 rows
                // of 4096 in bf16, two / four / five / eight on a CU: 60 / 55 / 66
                // / 62 us; 8192 of 8192, one / two of 512 threads: 63 / 52)
                constexpr long long kMost = NT <= 256 ? 1024 : U < 4 ? 512 : 256;
                const long long groups = std::min<long long>(ceil_div(rows, kRows), kMost);
                hipLaunchKernelGGL((k_norm<T, W, NT, U>), dim3((unsigned)groups), dim3(std::max(NT, 256)), 0, st,
                                   (const T*)x, (const W*)weight, (const W*)bias, rows, D, eps, (T*)y, mean, rstd);
            }
        });
    });
}

// partial rows of dw, and of db
static long long norm_parts(int dtype, long long rows, long long D) {
    long long n = 0;
    with_dtype(dtype, [&](auto tv) {
        using T = decltype(tv);
        with_shape<T>(D, [&](auto nt, auto) {
            constexpr int NT = nt.value;
            // a workgroup's partial row is written and read again: two of 256
            // threads on a CU (16384 rows of 4096 in bf16, one / two / four: 81 / 77
            // / 88 us; 65536 of 1024: 78 / 75 / 88), or one of 512
            if constexpr (NT == 0) n = std::min<long long>(rows, 64);
            else n = std::min<long long>(ceil_div(rows, NT < 256 ? 256 / NT : 1), 256 * 512 / std::max(NT, 256));
        });
    });
    return std::max(n, 1ll);
}
size_t norm_vjp_scratch(int dtype, long long rows, long long D) {
    return sizeof(float) * 2 * (size_t)norm_parts(dtype, rows, D) * (size_t)D;
}

void launch_norm_vjp(const void* x, const void* weight, const float* mean, const float* rstd, const void* dy, int dtype,
                     int wtype, long long rows, long long D, void* dx, void* dweight, void* dbias, float* part,
                     hipStream_t st) {
    const long long n = norm_parts(dtype, rows, D);
    if (!dweight && !dbias) part = nullptr;
    with_types(dtype, wtype, [&](auto tv, auto wv) {
        using T = decltype(tv);
        using W = decltype(wv);
        with_shape<T>(D, [&](auto nt, auto u) {
            constexpr int NT = nt.value, U = u.value;
            if constexpr (NT == 0) {
                if (dx && rows > 0)
                    hipLaunchKernelGGL((k_norm_vjp_wide<T, W>), dim3(wide_grid(rows)), dim3(kNormWide), 0, st,
                                       (const T*)x, (const W*)weight, mean, rstd, (const T*)dy, rows, D, (T*)dx);
                if (part)
                    hipLaunchKernelGGL((k_norm_dw_wide<T>), dim3((unsigned)std::min(ceil_div(D, 256), 65535ll), (unsigned)n),
                                       dim3(256), 0, st, (const T*)x, mean, rstd, (const T*)dy, rows, D, part);
            } else {
                hipLaunchKernelGGL((k_norm_vjp<T, W, NT, U>), dim3((unsigned)n), dim3(std::max(NT, 256)), 0, st,
                                   (const T*)x, (const W*)weight, mean, rstd, (const T*)dy, rows, D, (T*)dx, part);
            }
        });
        if (part)
            hipLaunchKernelGGL((k_norm_sum<W>), dim3(wide_grid(ceil_div(D, 64)), 2), dim3(1024), 0, st, part, (int)n, D,
                               (W*)dweight, (W*)dbias);
    });
}

}  // namespace lapsum
