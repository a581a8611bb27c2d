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
// A row lies in 16 lanes (expert e in lane e % 16), four rows to a wave.  A
// gate's key is 64 bits: its order-preserving 32-bit key above 1023 - expert,
// so keys differ and the larger of two equal gates is the one of the lower
// expert.  Keys are below 2^62 and positive, so they order alike as doubles,
// and the double maximum takes one instruction where integers take several.  A
// key without its upper half is below every gate's.
//
// Each of m rounds takes the largest of the 16 lanes' largest keys, blanks it,
// and finds its lane's next one.  Up to 192 experts a lane's keys are in
// registers and every lane searches its own again; with more, where only the
// one lane's keys have changed, they lie in LDS and the row's 16 lanes search
// them together.  Vector instructions bound both.  Measured, registers / LDS,
// us, 2^24 gates in rows of E, of which m are chosen:
//   E       128            192            257            512            1024
//   m = 2   16.1 / 16.7    15.6 / 16.9    16.4 / 17.4    16.7 / 14.8    32.6 / 22.6
//   m = 8   28.4 / 29.9    26.9 / 26.1    27.8 / 24.9    26.8 / 20.4    50.6 / 28.1
//   m = 32  82.6 / 99.2    73.9 / 72.8    74.9 / 59.1    67.6 / 42.2     122 / 49.5
// (the 67 MB of gates take 13 us).
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

// the key of expert e's gate from its 32-bit key; 0: not to be chosen
LS_DEV double wide_key(uint32_t k, int e) {
    const unsigned long long q = ((unsigned long long)k << 30) | (uint32_t)(1023 - e);
    return k ? __longlong_as_double((long long)q) : 0.0;
}
LS_DEV uint32_t gate_key(float v, float floor) { return v > floor ? f2key(v) : 0u; }

// What a row's 16 lanes collect: slot 16 b + l in lane l.
struct TopkRow {
    static constexpr int kBlocks = kSlotsMax / kTopkLanes;
    int id[kBlocks];
    float wt[kBlocks];
    float sum = 0.0f;

    // runs the m rounds; next(some, e) gives this lane's largest key once
    // expert e's is blanked
    template <class F>
    LS_DEV void collect(double mine, int m, F&& next) {
        const int l = threadIdx.x & (kTopkLanes - 1);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            id[b] = -1;
            wt[b] = 0.0f;
            for (int j = 0; j < kTopkLanes && b * kTopkLanes + j < m; ++j) {
                const double best = max16(mine);
                const unsigned long long q = (unsigned long long)__double_as_longlong(best);
                const bool some = (q >> 32) != 0;  // a gate above the floor has a key of at least 2^53
                const int e = 1023 - (int)(q & 1023);
                const float gate = some ? key2f((uint32_t)(q >> 30)) : 0.0f;
                sum += gate;
                if (j == l) {
                    id[b] = some ? e : -1;
                    wt[b] = gate;
                }
                mine = next(best, some, e);
            }
        }
    }
    LS_DEV void store(long long row, int m, int32_t* __restrict__ ids, float* __restrict__ w,
                      float* __restrict__ sums) {
        const int l = threadIdx.x & (kTopkLanes - 1);
        if (sums && l == 0) sums[row] = sum;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            const int j = b * kTopkLanes + l;
            if (j >= m) continue;
            ids[row * m + j] = id[b];
            w[row * m + j] = !sums ? wt[b] : sum > 0.0f ? wt[b] / sum : 0.0f;
        }
    }
};

// V keys a lane, in registers
template <int V>
__global__ __launch_bounds__(kTopkThreads) void k_expert_topk(const float* __restrict__ gates, long long T, int E,
                                                               int m, float floor, int32_t* __restrict__ ids,
                                                               float* __restrict__ w, float* __restrict__ sums) {
    constexpr int kRows = kTopkThreads / kTopkLanes;
    const int l = threadIdx.x & (kTopkLanes - 1);
    for (long long row0 = (long long)blockIdx.x * kRows; row0 < T; row0 += (long long)gridDim.x * kRows) {
        const long long row = row0 + threadIdx.x / kTopkLanes;
        const float* g = gates + min(row, T - 1) * E;
        double key[V];
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = l + kTopkLanes * i < E ? g[l + kTopkLanes * i] : -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = wide_key(gate_key(v[i], floor), l + kTopkLanes * i);
        auto largest = [&] {
            double k = key[0];
#pragma unroll
            for (int i = 1; i < V; ++i) k = max_f64(k, key[i]);
            return k;
        };
        TopkRow r;
        r.collect(largest(), m, [&](double best, bool, int) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                key[i] = __hiloint2double(key[i] == best ? 0 : __double2hiint(key[i]), __double2loint(key[i]));
            return largest();
        });
        if (row < T) r.store(row, m, ids, w, sums);
    }
}

// the 32-bit keys of a workgroup's rows in LDS (E words a row)
__global__ __launch_bounds__(kTopkThreads) void k_expert_topk_lds(const float* __restrict__ gates, long long T, int E,
                                                                   int m, float floor, int32_t* __restrict__ ids,
                                                                   float* __restrict__ w, float* __restrict__ sums) {
    extern __shared__ uint32_t lds_keys[];
    constexpr int kRows = kTopkThreads / kTopkLanes;
    const int l = threadIdx.x & (kTopkLanes - 1);
    uint32_t* keys = lds_keys + threadIdx.x / kTopkLanes * E;
    for (long long row0 = (long long)blockIdx.x * kRows; row0 < T; row0 += (long long)gridDim.x * kRows) {
        const long long row = row0 + threadIdx.x / kTopkLanes;
        const float* g = gates + min(row, T - 1) * E;
        double mine = 0.0;
        constexpr int U = 8;  // loads in flight a lane
        for (int e0 = l; e0 < E; e0 += U * kTopkLanes) {
            float v[U];
#pragma unroll
            for (int i = 0; i < U; ++i) v[i] = e0 + kTopkLanes * i < E ? g[e0 + kTopkLanes * i] : -INFINITY;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int e = e0 + kTopkLanes * i;
                const uint32_t k = gate_key(v[i], floor);
                if (e < E) keys[e] = k;
                mine = max_f64(mine, wide_key(k, e & 1023));
            }
        }
        TopkRow r;
        r.collect(mine, m, [&](double, bool some, int e) {
            // a row's keys are written and read by one wave, whose LDS
            // operations are served in order
            const int from = e & (kTopkLanes - 1);
            if (some && l == from) keys[e] = 0u;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            double k = 0.0;
            for (int o = from + kTopkLanes * l; o < E; o += kTopkLanes * kTopkLanes) k = max_f64(k, wide_key(keys[o], o));
            k = max16(k);
            if (l == from) mine = k;
            return mine;
        });
        if (row < T) r.store(row, m, ids, w, sums);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
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
    LS_TOPK(1) LS_TOPK(2) LS_TOPK(3) LS_TOPK(4) LS_TOPK(6) LS_TOPK(8) LS_TOPK(12)
#undef LS_TOPK
    hipLaunchKernelGGL(k_expert_topk_lds, grid, block, sizeof(uint32_t) * (size_t)E * (kTopkThreads / kTopkLanes), st,
                       gates, T, E, m, floor, ids, w, sums);
}

// ---------------------------------------------------------------------------
// gradient of the gates
// ---------------------------------------------------------------------------
// A workgroup writes whole rows: `rows` rows of dgates are cleared in LDS,
// every slot's value is put at its expert (the experts of a row differ), and
// the rows go out as one contiguous run.  The row's sum of dw w is taken over
// mp = the power of two >= m lanes.  The stores bound it: 65536 rows of 257
// gates, m = 8: 15.7 us for 74 MB, 4.7 TB/s (a large copy moves 4.9).
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
// Up to one such tile a workgroup of 16 waves does it all, in one launch (64
// pairs: 4.8 us, 4096 pairs: 6.3 us).  More are dealt out in contiguous shares
// to many: counts per share and expert, their prefix sums over the shares (a
// wave per expert), and the places (one workgroup, tile after tile / many, us:
// 4097 pairs of 64 experts 9.4 / 10.0, 8192 of 257 14.0 / 10.1, 16384 of 64
// 20.6 / 9.8).  Launches and LDS latencies bound it, not the 12 bytes a pair:
// 65536 x 8 pairs of 257 experts take 15 us back to back (count 3.5, scan 3.7,
// place 8.9), their bytes would take 1.
constexpr int kPairRuns = 4;
constexpr int kOneWaves = 16;                       // the single workgroup
constexpr int kManyWaves = 8;                       // one of many
constexpr int kPairTile = kManyWaves * 64 * kPairRuns;  // 2048 pairs
constexpr int kPairBlocksMax = 1024;
constexpr int kSortOneMax = kOneWaves * 64 * kPairRuns;  // its only tile: 4096 pairs

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

// The experts' pairs tot[E], of which a thread holds K t .. K t + K - 1.
template <int W>
struct ExpertCounts {
    static constexpr int K = (kExpertsMax + W * 64 - 1) / (W * 64);
    uint32_t v[K];

    LS_DEV void load(const uint32_t* tot, int E, size_t stride = 1) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int e = threadIdx.x * K + i;
            v[i] = e < E ? tot[e * stride] : 0u;
        }
    }
    // base[E] (LDS) = exclusive prefix + the thread's own more.v; returns the sum
    LS_DEV uint32_t prefix(const ExpertCounts& more, uint32_t* base, int E, uint32_t* scr) const {
        uint32_t mine = 0, sum = 0;
#pragma unroll
        for (int i = 0; i < K; ++i) mine += v[i];
        uint32_t ex = block_exclusive_scan<W * 64>(mine, &sum, scr);
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int e = threadIdx.x * K + i;
            if (e < E) base[e] = ex + more.v[i];
            ex += v[i];
        }
        __syncthreads();
        return sum;
    }
};

// One tile of pairs: rank() needs nothing but the ids, place() the experts'
// bases in LDS (the next place of each, moved past the tile).
template <int W>
struct PairTile {
    static constexpr int kPairs = W * 64 * kPairRuns;
    PairRuns r;
    long long at;

    LS_DEV void rank(const int32_t* __restrict__ ids, long long lo, long long hi, int E, int bits, uint32_t* cnt) {
        const int w = threadIdx.x >> 6;
        for (int i = threadIdx.x; i < W * E; i += W * 64) cnt[i] = 0u;
        __syncthreads();
        at = lo + (long long)w * (64 * kPairRuns);
        rank_runs(ids, at, hi, E, bits, cnt + w * E, r);
        __syncthreads();
    }
    LS_DEV void place(long long hi, int E, uint32_t* cnt, uint32_t* base, int32_t* __restrict__ order,
                      int32_t* __restrict__ to) {
        spread_counts<W>(cnt, base, E);
        __syncthreads();
        place_runs(r, at, hi, cnt + (threadIdx.x >> 6) * E, order, to);
        __syncthreads();
    }
};

LS_DEV void write_offsets(const uint32_t* base, uint32_t used, int E, int32_t* __restrict__ offsets) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) offsets[e] = (int32_t)base[e];
    if (threadIdx.x == 0) offsets[E] = (int32_t)used;
}

__global__ __launch_bounds__(kOneWaves * 64) void k_sort_one(const int32_t* __restrict__ ids, int P, int E, int bits,
                                                              int32_t* __restrict__ offsets,
                                                              int32_t* __restrict__ order,
                                                              int32_t* __restrict__ place) {
    __shared__ uint32_t cnt[kOneWaves * kExpertsMax], tot[kExpertsMax], base[kExpertsMax], scr[kOneWaves + 2];
    using Tile = PairTile<kOneWaves>;
    Tile t;
    t.rank(ids, 0, P, E, bits, cnt);
    for (int e = threadIdx.x; e < E; e += kOneWaves * 64) {
        uint32_t n = 0;
#pragma unroll
        for (int w = 0; w < kOneWaves; ++w) n += cnt[w * E + e];
        tot[e] = n;
    }
    __syncthreads();
    ExpertCounts<kOneWaves> all, none = {};
    all.load(tot, E);
    const uint32_t used = all.prefix(none, base, E, scr);
    write_offsets(base, used, E, offsets);
    for (int i = (int)used + threadIdx.x; i < P; i += kOneWaves * 64) order[i] = -1;
    __syncthreads();  // offsets are out before the bases move
    t.place(P, E, cnt, base, order, place);
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
    using Tile = PairTile<kManyWaves>;
    const long long lo = (long long)blockIdx.x * per, hi = min(lo + per, P);
    ExpertCounts<kManyWaves> all, before;  // their loads run beside the ids'
    all.load(totals, E);
    before.load(counts + blockIdx.x, E, gridDim.x);
    Tile t;
    t.rank(ids, lo, hi, E, bits, cnt);
    const uint32_t used = all.prefix(before, base, E, scr);
    if (blockIdx.x == 0) write_offsets(base, used, E, offsets);  // no pairs are before the first
    for (long long i = max(lo, (long long)used) + threadIdx.x; i < hi; i += kManyWaves * 64) order[i] = -1;
    __syncthreads();  // offsets are out before the bases move
    t.place(hi, E, cnt, base, order, place);
    for (long long q = lo + Tile::kPairs; q < hi; q += Tile::kPairs) {
        t.rank(ids, q, hi, E, bits, cnt);
        t.place(hi, E, cnt, base, order, place);
    }
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
