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
// A row lies in 16 lanes, V keys each (expert lane + 16 i), four rows to a
// wave.  Keys order like the gates; 0 marks a gate that cannot be chosen.
// Each round takes the row's largest key by lane exchanges over the 16 lanes,
// then the lowest expert that has it, and blanks that one.
constexpr int kTopkLanes = 16;
constexpr int kTopkThreads = 256;

LS_DEV uint32_t max16(uint32_t v) {
    v = max(v, xor_lane<8>(v));
    v = max(v, xor_lane<4>(v));
    v = max(v, xor_lane<2>(v));
    v = max(v, xor_lane<1>(v));
    return v;
}
LS_DEV uint32_t min16(uint32_t v) {
    v = min(v, xor_lane<8>(v));
    v = min(v, xor_lane<4>(v));
    v = min(v, xor_lane<2>(v));
    v = min(v, xor_lane<1>(v));
    return v;
}

template <int V>
LS_DEV void topk_row(const float* __restrict__ gates, long long row, long long T, int E, int m, float floor,
                     int32_t* __restrict__ ids, float* __restrict__ w, float* __restrict__ sums) {
    const int l = threadIdx.x & (kTopkLanes - 1);
    const bool live = row < T;
    const float* g = gates + (live ? row : T - 1) * E;
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = l + kTopkLanes * i;
        const float v = e < E ? g[e] : -INFINITY;
        key[i] = v > floor ? f2key(v) : 0u;
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
            uint32_t best = 0u;
#pragma unroll
            for (int i = 0; i < V; ++i) best = max(best, key[i]);
            best = max16(best);
            uint32_t at = 0xFFFFFFFFu;
#pragma unroll
            for (int i = V - 1; i >= 0; --i) at = key[i] == best ? (uint32_t)i : at;
            at = min16(at == 0xFFFFFFFFu ? at : at * kTopkLanes + l);
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = at == (uint32_t)(kTopkLanes * i + l) ? 0u : key[i];
            const bool some = best != 0u;
            const float v = some ? key2f(best) : 0.0f;
            sum += v;
            if (j == l) {
                id[b] = some ? (int)at : -1;
                wt[b] = v;
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
    LS_TOPK(1) LS_TOPK(2) LS_TOPK(4) LS_TOPK(8) LS_TOPK(16) LS_TOPK(24) LS_TOPK(32) LS_TOPK(48) LS_TOPK(64)
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
// A workgroup of kSortWaves waves ranks kSortWaves * R * 64 pairs at a time:
// each wave takes R runs of 64 consecutive pairs, finds the lanes of a run
// that share an expert by ballots over the id's bits, and counts per wave and
// expert in LDS; the waves' counts are then summed in wave order.  A pair's
// place is the expert's base + the pairs of earlier waves + those of its own
// wave's earlier runs + those of lower lanes.
constexpr int kSortWaves = 16;
constexpr int kPairThreads = kSortWaves * 64;
constexpr int kPairRuns = 4;
constexpr int kPairTile = kPairThreads * kPairRuns;  // 4096 pairs
constexpr int kPairBlocksMax = 1024;
constexpr int kSortOneMax = 4 * kPairTile;  // pairs that one workgroup sorts alone

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
LS_DEV void spread_counts(uint32_t* cnt, uint32_t* base, int E) {
    for (int e = threadIdx.x; e < E; e += kPairThreads) {
        uint32_t run = base[e];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t c = cnt[w * E + e];
            cnt[w * E + e] = run;
            run += c;
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

// Counts of the pairs [lo, hi) per expert into s_tot (LDS, E words).  Each
// wave counts on its own in cnt (LDS, waves x E) so that few lanes meet.
LS_DEV void count_pairs(const int32_t* __restrict__ ids, long long lo, long long hi, int E, uint32_t* tot) {
    for (int e = threadIdx.x; e < E; e += kPairThreads) tot[e] = 0u;
    __syncthreads();
    for (long long i = lo + threadIdx.x; i < hi; i += kPairThreads) {
        const int e = pair_expert(ids, i, hi, E);
        if (e >= 0) atomicAdd(&tot[e], 1u);
    }
    __syncthreads();
}

// tot[E] (LDS) -> exclusive prefix in base[E] (LDS); returns the sum
LS_DEV uint32_t prefix_experts(const uint32_t* tot, uint32_t* base, int E, uint32_t* scr) {
    static_assert(kExpertsMax <= kPairThreads, "one expert per thread");
    const int e = threadIdx.x;
    const uint32_t v = e < E ? tot[e] : 0u;
    uint32_t sum = 0;
    const uint32_t ex = block_exclusive_scan<kPairThreads>(v, &sum, scr);
    if (e < E) base[e] = ex;
    __syncthreads();
    return sum;
}

// ranks and places the pairs [lo, hi), base[e] (LDS) = the next place of e
LS_DEV void place_pairs(const int32_t* __restrict__ ids, long long lo, long long hi, int E, int bits, uint32_t* cnt,
                        uint32_t* base, int32_t* __restrict__ order, int32_t* __restrict__ place) {
    const int w = threadIdx.x >> 6;
    for (long long t = lo; t < hi; t += kPairTile) {
        for (int i = threadIdx.x; i < kSortWaves * E; i += kPairThreads) cnt[i] = 0u;
        __syncthreads();
        const long long at = t + (long long)w * (64 * kPairRuns);
        PairRuns r;
        rank_runs(ids, at, hi, E, bits, cnt + w * E, r);
        __syncthreads();
        spread_counts(cnt, base, E);
        __syncthreads();
        place_runs(r, at, hi, cnt + w * E, order, place);
        __syncthreads();
    }
}

__global__ __launch_bounds__(kPairThreads) void k_sort_one(const int32_t* __restrict__ ids, int P, int E, int bits,
                                                            int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                                                            int32_t* __restrict__ place) {
    extern __shared__ uint32_t dyn[];  // cnt[waves][E], tot[E], base[E]
    __shared__ uint32_t scr[kSortWaves + 2];
    uint32_t* cnt = dyn;
    uint32_t* tot = cnt + kSortWaves * E;
    uint32_t* base = tot + E;
    count_pairs(ids, 0, P, E, tot);
    const uint32_t used = prefix_experts(tot, base, E, scr);
    for (int e = threadIdx.x; e < E; e += kPairThreads) offsets[e] = (int32_t)base[e];
    if (threadIdx.x == 0) offsets[E] = (int32_t)used;
    for (int i = (int)used + threadIdx.x; i < P; i += kPairThreads) order[i] = -1;
    __syncthreads();
    place_pairs(ids, 0, P, E, bits, cnt, base, order, place);
}

// counts[b][E] of workgroup b's pairs
__global__ __launch_bounds__(kPairThreads) void k_sort_count(const int32_t* __restrict__ ids, long long P, int E,
                                                              long long per, uint32_t* __restrict__ counts) {
    extern __shared__ uint32_t dyn[];
    const long long lo = (long long)blockIdx.x * per, hi = min(lo + per, P);
    count_pairs(ids, lo, hi, E, dyn);
    for (int e = threadIdx.x; e < E; e += kPairThreads) counts[(size_t)blockIdx.x * E + e] = dyn[e];
}

// counts[b][e] -> the pairs of e before workgroup b (in place); totals[E]
__global__ __launch_bounds__(256) void k_sort_scan(uint32_t* __restrict__ counts, int nb, int E,
                                                    uint32_t* __restrict__ totals) {
    const int e = blockIdx.x * 64 + (threadIdx.x & 63), w = threadIdx.x >> 6;
    __shared__ uint32_t part[4][64];
    const int q = (nb + 3) / 4, b0 = w * q, b1 = min(b0 + q, nb);
    uint32_t sum = 0;
    if (e < E)
        for (int b = b0; b < b1; ++b) sum += counts[(size_t)b * E + e];
    part[w][threadIdx.x & 63] = sum;
    __syncthreads();
    if (e >= E) return;
    uint32_t run = 0;
    for (int v = 0; v < w; ++v) run += part[v][threadIdx.x & 63];
    for (int b = b0; b < b1; ++b) {
        const uint32_t c = counts[(size_t)b * E + e];
        counts[(size_t)b * E + e] = run;
        run += c;
    }
    if (w == 3) totals[e] = run;
}

__global__ __launch_bounds__(kPairThreads) void k_sort_place(const int32_t* __restrict__ ids, long long P, int E,
                                                              int bits, long long per,
                                                              const uint32_t* __restrict__ counts,
                                                              const uint32_t* __restrict__ totals,
                                                              int32_t* __restrict__ offsets,
                                                              int32_t* __restrict__ order,
                                                              int32_t* __restrict__ place) {
    extern __shared__ uint32_t dyn[];  // cnt[waves][E], base[E]
    __shared__ uint32_t scr[kSortWaves + 2];
    uint32_t* cnt = dyn;
    uint32_t* base = cnt + kSortWaves * E;
    const uint32_t used = prefix_experts(totals, base, E, scr);
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e < E; e += kPairThreads) offsets[e] = (int32_t)base[e];
        if (threadIdx.x == 0) offsets[E] = (int32_t)used;
    }
    const long long lo = (long long)blockIdx.x * per, hi = min(lo + per, P);
    for (long long i = max(lo, (long long)used) + threadIdx.x; i < hi; i += kPairThreads) order[i] = -1;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kPairThreads) base[e] += counts[(size_t)blockIdx.x * E + e];
    __syncthreads();
    place_pairs(ids, lo, hi, E, bits, cnt, base, order, place);
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
        const size_t lds = sizeof(uint32_t) * (size_t)E * (kSortWaves + 2);
        hipLaunchKernelGGL(k_sort_one, dim3(1), dim3(kPairThreads), lds, st, ids, (int)P, E, bits, offsets, order,
                           place);
        return;
    }
    const long long nb = sort_blocks(P), per = ceil_div(ceil_div(P, nb), kPairTile) * kPairTile;
    uint32_t* totals = scratch + (size_t)nb * (size_t)E;
    hipLaunchKernelGGL(k_sort_count, dim3((unsigned)nb), dim3(kPairThreads), sizeof(uint32_t) * (size_t)E, st, ids, P,
                       E, per, scratch);
    hipLaunchKernelGGL(k_sort_scan, dim3((unsigned)ceil_div(E, 64)), dim3(256), 0, st, scratch, (int)nb, E, totals);
    hipLaunchKernelGGL(k_sort_place, dim3((unsigned)nb), dim3(kPairThreads),
                       sizeof(uint32_t) * (size_t)E * (kSortWaves + 1), st, ids, P, E, bits, per, scratch, totals,
                       offsets, order, place);
}

}  // namespace lapsum
