// From gates to a plan: the m largest gates of every row, their gradient, and
// the (token, slot) pairs in expert order.
//
//  k_expert_topk      16 lanes hold a row and take its largest key m times
//  k_expert_topk_vjp  a few rows of dgates at a time, scattered in LDS
//  k_sort_one         the whole counting sort in one workgroup
//  k_sort_count, k_sort_scan, k_sort_place   the same over many workgroups
#include <algorithm>

#include "lapsum_expert_ops.h"

namespace lapsum {

// ---------------------------------------------------------------------------
// the m largest gates of every row
// ---------------------------------------------------------------------------
// A row lies in 16 lanes, V gates each (expert lane + 16 i), four rows to a
// wave.  A gate's key is 64 bits: its order-preserving 32-bit key above
// 1023 - expert, so keys differ and the larger of two equal gates is the one
// of the lower expert.  Keys are below 2^62 and positive, so they order alike
// as doubles, and the double maximum and compare take one instruction each
// where integers take several.  Each of m rounds takes the row's largest key
// (over a lane's keys, then over the 16 lanes) and blanks it; a key without
// its upper half is below every gate's.  V is E / 16 rounded up to few sizes.
// Vector instructions bound it: about 3 V + 20 a round for four rows
// (65536 rows of 257 gates, m = 8: 17 us; with 32-bit keys, a second search
// for the expert and a compare to blank it, 40 us).
constexpr int kTopkLanes = 16;
constexpr int kTopkThreads = 256;
static_assert(kExpertsMax <= 1024, "an expert has 10 bits of a key");

// max of two non-negative doubles that are not NaN
LS_DEV double max_f64(double a, double b) {
    double d;
    asm("v_max_f64 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
    return d;
}
LS_DEV double max16(double v) {
    v = max_f64(v, xor_lane_f64<8>(v));
    v = max_f64(v, xor_lane_f64<4>(v));
    v = max_f64(v, xor_lane_f64<2>(v));
    return max_f64(v, xor_lane_f64<1>(v));
}

template <int V>
LS_DEV void topk_row(const float* __restrict__ gates, long long row, long long T, int E, int m, float floor,
                     int32_t* __restrict__ ids, float* __restrict__ w, float* __restrict__ sums) {
    const int l = threadIdx.x & (kTopkLanes - 1);
    const bool live = row < T;
    const float* g = gates + (live ? row : T - 1) * E;
    double key[V];
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = l + kTopkLanes * i < E ? g[l + kTopkLanes * i] : -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t k = f2key(v[i]);
        const unsigned long long q = ((unsigned long long)k << 30) | (uint32_t)(1023 - (l + kTopkLanes * i));
        key[i] = v[i] > floor ? __longlong_as_double((long long)q) : 0.0;
    }
    constexpr int kBlocks = kSlotsMax / kTopkLanes;
    int id[kBlocks];
    float wt[kBlocks];
    float sum = 0.0f;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        id[b] = -1;
        wt[b] = 0.0f;
        for (int j = 0; j < kTopkLanes && b * kTopkLanes + j < m; ++j) {
            double best = key[0];
#pragma unroll
            for (int i = 1; i < V; ++i) best = max_f64(best, key[i]);
            best = max16(best);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int hi = key[i] == best ? 0 : __double2hiint(key[i]);
                key[i] = __hiloint2double(hi, __double2loint(key[i]));
            }
            const unsigned long long q = (unsigned long long)__double_as_longlong(best);
            const bool some = (q >> 32) != 0;  // a gate above the floor has a key of at least 2^53
            const float gate = some ? key2f((uint32_t)(q >> 30)) : 0.0f;
            sum += gate;
            if (j == l) {
                id[b] = some ? 1023 - (int)(q & 1023) : -1;
                wt[b] = gate;
            }
        }
    }
    if (!live) return;
    if (sums) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) wt[b] = sum > 0.0f ? wt[b] / sum : 0.0f;
        if (l == 0) sums[row] = sum;
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        const int j = b * kTopkLanes + l;
        if (j < m) {
            ids[row * m + j] = id[b];
            w[row * m + j] = wt[b];
        }
    }
}
template <int V>
__global__ __launch_bounds__(kTopkThreads) void k_expert_topk(const float* __restrict__ gates, long long T, int E,
                                                               int m, float floor, int32_t* __restrict__ ids,
                                                               float* __restrict__ w, float* __restrict__ sums) {
    constexpr int kRows = kTopkThreads / kTopkLanes;
    for (long long row0 = (long long)blockIdx.x * kRows; row0 < T; row0 += (long long)gridDim.x * kRows)
        topk_row<V>(gates, row0 + threadIdx.x / kTopkLanes, T, E, m, floor, ids, w, sums);
}

void launch_expert_topk(const float* gates, long long T, int E, int m, float floor, int32_t* ids, float* w,
                        float* sums, hipStream_t st) {
    if (T < 1) return;
    const dim3 grid(grid_of(ceil_div(T, kTopkThreads / kTopkLanes))), block(kTopkThreads);
    const int v = (E + kTopkLanes - 1) / kTopkLanes;
#define LS_TOPK(V)                                                                                          \
    if (v <= V) {                                                                                           \
        hipLaunchKernelGGL((k_expert_topk<V>), grid, block, 0, st, gates, T, E, m, floor, ids, w, sums);    \
        return;                                                                                             \
    }
    LS_TOPK(1) LS_TOPK(2) LS_TOPK(3) LS_TOPK(4) LS_TOPK(6) LS_TOPK(8) LS_TOPK(10) LS_TOPK(12) LS_TOPK(14) LS_TOPK(16)
    LS_TOPK(18) LS_TOPK(20) LS_TOPK(24) LS_TOPK(28) LS_TOPK(32) LS_TOPK(40) LS_TOPK(48) LS_TOPK(64)
#undef LS_TOPK
}

// ---------------------------------------------------------------------------
// gradient of the gates
// ---------------------------------------------------------------------------
// A workgroup writes whole rows: `rows` rows of dgates are cleared in LDS,
// every slot's value is put at its expert (the experts of a row differ), and
// the rows go out as one contiguous run.  The row's sum of dw w is taken over
// mp = the power of two >= m lanes.
constexpr int kTopkVjpThreads = 256;
constexpr int kTopkVjpFloats = 4096;

__global__ __launch_bounds__(kTopkVjpThreads) void k_expert_topk_vjp(const int32_t* __restrict__ ids,
                                                                      const float* __restrict__ w,
                                                                      const float* __restrict__ dw,
                                                                      const float* __restrict__ sums, long long T,
                                                                      int E, int m, int mp, int rows,
                                                                      float* __restrict__ dgates) {
    __shared__ float s[kTopkVjpFloats];
    for (long long row0 = (long long)blockIdx.x * rows; row0 < T; row0 += (long long)gridDim.x * rows) {
        const int nr = (int)min((long long)rows, T - row0);
        const int n = nr * E;
        for (int i = threadIdx.x; i < n; i += kTopkVjpThreads) s[i] = 0.0f;
        __syncthreads();
        const int per = kTopkVjpThreads / mp;  // rows a step
        for (int r0 = 0; r0 < nr; r0 += per) {
            const int r = r0 + threadIdx.x / mp, j = threadIdx.x & (mp - 1);
            const bool on = r < nr && j < m;
            const long long at = (row0 + r) * m + j;
            const int id = on ? ids[at] : -1;
            const bool put = id >= 0 && id < E;
            float g = put ? dw[at] : 0.0f;
            if (sums) {
                float dot = put ? g * w[at] : 0.0f;
                for (int d = 1; d < mp; d <<= 1) dot += __uint_as_float(xor_lane_rt(__float_as_uint(dot), d));
                const float sum = on ? sums[row0 + r] : 1.0f;
                g = sum > 0.0f ? (g - dot) / sum : 0.0f;
            }
            if (put) s[r * E + id] = g;
        }
        __syncthreads();
        float* out = dgates + row0 * E;
        for (int i = threadIdx.x; i < n; i += kTopkVjpThreads) out[i] = s[i];
        __syncthreads();
    }
}

void launch_expert_topk_vjp(const int32_t* ids, const float* w, const float* dw, const float* sums, long long T,
                            int E, int m, float* dgates, hipStream_t st) {
    if (T < 1) return;
    int mp = 1;
    while (mp < m) mp <<= 1;
    const int rows = std::max(1, kTopkVjpFloats / E);
    hipLaunchKernelGGL(k_expert_topk_vjp, dim3(grid_of(ceil_div(T, rows))), dim3(kTopkVjpThreads), 0, st, ids, w, dw,
                       sums, T, E, m, mp, rows, dgates);
}

// ---------------------------------------------------------------------------
// pairs in expert order: a stable counting sort by expert
// ---------------------------------------------------------------------------
// A workgroup of W waves ranks W * 256 pairs at a time: each wave takes four
// runs of 64 consecutive pairs, finds the lanes of a run that share an expert
// by ballots over the id's bits, and counts per wave and expert in LDS; the
// waves' counts are then summed in wave order.  A pair's place is the
// expert's base + the pairs of earlier waves + those of its own wave's
// earlier runs + those of lower lanes.
//
// Up to kSortOneMax pairs one workgroup does it all, in one launch.  More are
// dealt out in contiguous shares to many: counts per share and expert, their
// prefix sums over the shares (a wave per expert), and the places.  Launches
// and LDS latencies bound it, not the 12 bytes a pair (65536 x 8 pairs, 257
// experts: count 3, scan 3, place 6 us, at 6 TB/s the bytes would take 1).
constexpr int kPairRuns = 4;
constexpr int kOneWaves = 16;                       // the single workgroup
constexpr int kManyWaves = 8;                       // one of many
constexpr int kPairTile = kManyWaves * 64 * kPairRuns;  // 2048 pairs
constexpr int kPairBlocksMax = 1024;
constexpr int kSortOneMax = 4 * kOneWaves * 64 * kPairRuns;  // 16384

// ids outside [0, E) have no expert: -1
LS_DEV int pair_expert(const int32_t* __restrict__ ids, long long i, long long hi, int E) {
    const int e = i < hi ? ids[i] : -1;
    return (unsigned)e < (unsigned)E ? e : -1;
}

struct PairRuns {
    int e[kPairRuns];     // expert or -1
    int rank[kPairRuns];  // pairs of the same expert before it in this wave's runs
};

// Counts this wave's runs into cnt[E] (LDS, zero before) and ranks its pairs.
LS_DEV void rank_runs(const int32_t* __restrict__ ids, long long lo, long long hi, int E, int bits, uint32_t* cnt,
                      PairRuns& r) {
    const int l = lane_id();
#pragma unroll
    for (int q = 0; q < kPairRuns; ++q) r.e[q] = pair_expert(ids, lo + q * 64 + l, hi, E);
#pragma unroll
    for (int q = 0; q < kPairRuns; ++q) {
        const int e = r.e[q];
        unsigned long long same = ballot(e >= 0);
        for (int b = 0; b < bits; ++b) {
            const bool bit = (e >> b) & 1;
            const unsigned long long bal = ballot(bit);
            same &= bit ? bal : ~bal;
        }
        const int below = mbcnt(same);
        int before = 0;
        if (e >= 0 && below == 0) before = (int)atomicAdd(&cnt[e], (uint32_t)popc64(same));
        const int leader = same ? __builtin_ctzll(same) : 0;
        r.rank[q] = __shfl(before, leader) + below;
    }
}

// bits that tell the experts 0 .. E-1 apart
inline int id_bits(int E) {
    int b = 0;
    while ((1 << b) < E) ++b;
    return b;
}

// cnt[wave][E] -> base[e] + the counts of earlier waves; base[e] (LDS) moves
// past this tile's pairs
template <int W>
LS_DEV void spread_counts(uint32_t* cnt, uint32_t* base, int E) {
    for (int e = threadIdx.x; e < E; e += W * 64) {
        uint32_t c[W];
#pragma unroll
        for (int w = 0; w < W; ++w) c[w] = cnt[w * E + e];
        uint32_t run = base[e];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            cnt[w * E + e] = run;
            run += c[w];
        }
        base[e] = run;
    }
}

LS_DEV void place_runs(const PairRuns& r, long long lo, long long hi, const uint32_t* cnt, int32_t* __restrict__ order,
                       int32_t* __restrict__ place) {
    const int l = lane_id();
#pragma unroll
    for (int q = 0; q < kPairRuns; ++q) {
        const long long i = lo + q * 64 + l;
        if (i >= hi) continue;
        int pos = -1;
        if (r.e[q] >= 0) {
            pos = (int)cnt[r.e[q]] + r.rank[q];
            order[pos] = (int32_t)i;
        }
        place[i] = pos;
    }
}

// counts of the pairs [lo, hi) per expert into tot (LDS, E words)
template <int W>
LS_DEV void count_pairs(const int32_t* __restrict__ ids, long long lo, long long hi, int E, uint32_t* tot) {
    for (int e = threadIdx.x; e < E; e += W * 64) tot[e] = 0u;
    __syncthreads();
#pragma unroll 4
    for (long long i = lo + threadIdx.x; i < hi; i += W * 64) {
        const int e = pair_expert(ids, i, hi, E);
        if (e >= 0) atomicAdd(&tot[e], 1u);
    }
    __syncthreads();
}

// tot[E] -> exclusive prefix in base[E] (LDS); returns the sum.  A thread
// takes the experts K t .. K t + K - 1.
template <int W>
LS_DEV uint32_t prefix_experts(const uint32_t* tot, uint32_t* base, int E, uint32_t* scr) {
    constexpr int K = (kExpertsMax + W * 64 - 1) / (W * 64);
    const int e0 = threadIdx.x * K;
    uint32_t v[K], mine = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < K; ++i) mine += v[i] = e0 + i < E ? tot[e0 + i] : 0u;
    uint32_t ex = block_exclusive_scan<W * 64>(mine, &sum, scr);
#pragma unroll
    for (int i = 0; i < K; ++i) {
        if (e0 + i < E) base[e0 + i] = ex;
        ex += v[i];
    }
    __syncthreads();
    return sum;
}

// ranks and places the pairs [lo, hi), base[e] (LDS) = the next place of e
template <int W>
LS_DEV void place_pairs(const int32_t* __restrict__ ids, long long lo, long long hi, int E, int bits, uint32_t* cnt,
                        uint32_t* base, int32_t* __restrict__ order, int32_t* __restrict__ place) {
    const int w = threadIdx.x >> 6;
    for (long long t = lo; t < hi; t += W * 64 * kPairRuns) {
        for (int i = threadIdx.x; i < W * E; i += W * 64) cnt[i] = 0u;
        __syncthreads();
        const long long at = t + (long long)w * (64 * kPairRuns);
        PairRuns r;
        rank_runs(ids, at, hi, E, bits, cnt + w * E, r);
        __syncthreads();
        spread_counts<W>(cnt, base, E);
        __syncthreads();
        place_runs(r, at, hi, cnt + w * E, order, place);
        __syncthreads();
    }
}

LS_DEV void write_offsets(const uint32_t* base, uint32_t used, int E, int32_t* __restrict__ offsets) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) offsets[e] = (int32_t)base[e];
    if (threadIdx.x == 0) offsets[E] = (int32_t)used;
}

__global__ __launch_bounds__(kOneWaves * 64) void k_sort_one(const int32_t* __restrict__ ids, int P, int E, int bits,
                                                              int32_t* __restrict__ offsets,
                                                              int32_t* __restrict__ order,
                                                              int32_t* __restrict__ place) {
    __shared__ uint32_t cnt[kOneWaves * kExpertsMax], tot[kExpertsMax], base[kExpertsMax], scr[kOneWaves + 2];
    count_pairs<kOneWaves>(ids, 0, P, E, tot);
    const uint32_t used = prefix_experts<kOneWaves>(tot, base, E, scr);
    write_offsets(base, used, E, offsets);
    for (int i = (int)used + threadIdx.x; i < P; i += kOneWaves * 64) order[i] = -1;
    __syncthreads();
    place_pairs<kOneWaves>(ids, 0, P, E, bits, cnt, base, order, place);
}

// counts[e][b]: workgroup b's pairs of expert e
__global__ __launch_bounds__(kManyWaves * 64) void k_sort_count(const int32_t* __restrict__ ids, long long P, int E,
                                                                 long long per, uint32_t* __restrict__ counts) {
    __shared__ uint32_t tot[kExpertsMax];
    const long long lo = (long long)blockIdx.x * per, hi = min(lo + per, P);
    count_pairs<kManyWaves>(ids, lo, hi, E, tot);
    for (int e = threadIdx.x; e < E; e += kManyWaves * 64) counts[(size_t)e * gridDim.x + blockIdx.x] = tot[e];
}

// counts[e][b] -> the pairs of e before workgroup b (in place); totals[E]
__global__ __launch_bounds__(256) void k_sort_scan(uint32_t* __restrict__ counts, int nb, int E,
                                                    uint32_t* __restrict__ totals) {
    const int e = blockIdx.x * 4 + uniform(threadIdx.x >> 6), l = lane_id();
    if (e >= E) return;
    uint32_t* c = counts + (size_t)e * nb;
    uint32_t run = 0;
    for (int b0 = 0; b0 < nb; b0 += 64) {
        const uint32_t v = b0 + l < nb ? c[b0 + l] : 0u;
        const uint32_t inc = wave_inclusive_scan(v);
        if (b0 + l < nb) c[b0 + l] = run + inc - v;
        run += (uint32_t)__builtin_amdgcn_readlane((int)inc, 63);
    }
    if (l == 0) totals[e] = run;
}

__global__ __launch_bounds__(kManyWaves * 64) void k_sort_place(const int32_t* __restrict__ ids, long long P, int E,
                                                                 int bits, long long per,
                                                                 const uint32_t* __restrict__ counts,
                                                                 const uint32_t* __restrict__ totals,
                                                                 int32_t* __restrict__ offsets,
                                                                 int32_t* __restrict__ order,
                                                                 int32_t* __restrict__ place) {
    __shared__ uint32_t cnt[kManyWaves * kExpertsMax], base[kExpertsMax], scr[kManyWaves + 2];
    const uint32_t used = prefix_experts<kManyWaves>(totals, base, E, scr);
    if (blockIdx.x == 0) write_offsets(base, used, E, offsets);
    const long long lo = (long long)blockIdx.x * per, hi = min(lo + per, P);
    for (long long i = max(lo, (long long)used) + threadIdx.x; i < hi; i += kManyWaves * 64) order[i] = -1;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kManyWaves * 64) base[e] += counts[(size_t)e * gridDim.x + blockIdx.x];
    __syncthreads();
    place_pairs<kManyWaves>(ids, lo, hi, E, bits, cnt, base, order, place);
}

static long long sort_blocks(long long P) {
    return std::min<long long>(kPairBlocksMax, ceil_div(P, kPairTile));
}
size_t expert_sort_scratch(long long P, int E) {
    return P <= kSortOneMax ? 0 : sizeof(uint32_t) * (size_t)(sort_blocks(P) + 1) * (size_t)E;
}

void launch_expert_sort(const int32_t* ids, long long P, int E, int32_t* offsets, int32_t* order, int32_t* place,
                        uint32_t* scratch, hipStream_t st) {
    const int bits = id_bits(E);
    if (P <= kSortOneMax) {
        hipLaunchKernelGGL(k_sort_one, dim3(1), dim3(kOneWaves * 64), 0, st, ids, (int)P, E, bits, offsets, order,
                           place);
        return;
    }
    const long long nb = sort_blocks(P), per = ceil_div(ceil_div(P, nb), kPairTile) * kPairTile;
    const dim3 grid((unsigned)nb), block(kManyWaves * 64);
    uint32_t* totals = scratch + (size_t)nb * (size_t)E;
    hipLaunchKernelGGL(k_sort_count, grid, block, 0, st, ids, P, E, per, scratch);
    hipLaunchKernelGGL(k_sort_scan, dim3((unsigned)ceil_div(E, 4)), dim3(256), 0, st, scratch, (int)nb, E, totals);
    hipLaunchKernelGGL(k_sort_place, grid, block, 0, st, ids, P, E, bits, per, scratch, totals, offsets, order,
                       place);
}

}  // namespace lapsum
