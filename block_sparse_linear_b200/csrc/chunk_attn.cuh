// Chunk attention: what its kernels share. Exact causal attention of a chunk of new tokens
// over the paged cache. With L_b tokens held by sequence b, the chunk's n_b among them,
// query t of the chunk stands at position L_b - n_b + t and sees the tokens up to its own:
//   o_t = sum_{s <= pos_t} p_ts v_s / sum p_ts,   p_ts = exp(scale q_t . k_s),
//   lse_t = log sum_{s <= pos_t} p_ts
// in one pass over the tokens with a running maximum (softmax attention as in the Baidu
// article's section 1; the paged pools are the decode path's own).
//
// Rows. The G query heads that share a KV head and consecutive new tokens are the rows of
// a tile (row = token * G + head), so a tile of K and V is read once for all of them. A
// unit is one (sequence, KV head, block of U query tokens).
//
// Split. Every unit takes T = ceil(visible tokens / KT) steps over KT-token tiles of K and
// V. All units' steps in a row, each with its cost (Cost: a step of a unit of two query
// tiles, of one, and what starting a unit takes), are cut into runs of equal cost, one per
// CTA (one CTA per SM), whatever the lengths: a single long sequence, a ragged batch and
// many short prompts all fill the GPU evenly.
// A unit that lies within one run is finished there; one that is cut leaves unnormalised
// partial sums (O, l, and the maximum m they are scaled by, in log2 units), which
// chunk_combine_kernel joins in run order, so results do not depend on timing.
#pragma once

#include "common.cuh"

// The split's arithmetic also compiles for the host, where it is tested.
#define SPLA_HD __host__ __device__ __forceinline__

namespace spla {

// What the split's run c left for the join, at its place in the workspace.
struct ChunkCut {
    int32_t parts;            // runs the unit that starts in run c and leaves it spans; 0: none
    int32_t rows;             // its rows that hold queries
    int32_t b, h, t0;         // sequence, KV head, first query token
    int32_t pad[3];
};

constexpr int kMaxRuns = kNumSms;
constexpr size_t kCutBytes = (sizeof(ChunkCut) * kMaxRuns + 255) / 256 * 256;
// One partial: O [rows][d], then m [rows], l [rows]; run c has two (0: of the unit it
// begins inside of, 1: of the unit it leaves unfinished).
__host__ __device__ constexpr int64_t part_floats(int d) { return 256 * (int64_t)(d + 2); }

// The chunk of sequence b; n = 0 where there is none or it is out of range, whose status
// bit is returned.
SPLA_HD int32_t chunk_of(const CacheView& c, const ChunkArgs& a, int b, int32_t* L, int32_t* n) {
    *L = c.lens[b];
    *n = a.n_new[b];
    int32_t bad = 0;
    if (*n < 0 || *n > a.max_new) bad = SPLA_DEV_BAD_COUNT;
    else if (*L < 0 || *L > (int64_t)c.mbp * c.bs) bad = SPLA_DEV_CAPACITY;
    else if (*n > *L) bad = SPLA_DEV_BAD_COUNT;
    if (bad) {
        *n = 0;
        *L = 0;
    }
    return bad;
}

// Steps of the units before query block qb of a sequence whose chunk starts at position
// base: sum over i < qb of ceil((base + (i+1) U) / KT). U and KT are powers of two.
template <int KT>
SPLA_HD int64_t steps_before(int32_t base, int32_t qb, int U) {
    if (U >= KT) {
        const int64_t k = U / KT;
        return (int64_t)qb * ((base + KT - 1) / KT) + k * ((int64_t)qb * (qb + 1) / 2);
    }
    // every r-th block of a class adds a step
    int lg = 1;
    while (U << lg < KT) ++lg;
    const int r = 1 << lg;
    int64_t sum = 0;
#pragma unroll 1
    for (int p = 0; p < r; ++p) {
        const int64_t k = (qb - p + r - 1) >> lg;
        sum += k * ((base + (p + 1) * U + KT - 1) / KT) + k * (k - 1) / 2;
    }
    return sum;
}

// Tokens of a step and what steps cost: bf16.
constexpr int kTcTile = 128;
// A step of a pair of tiles against one of a single tile, and a unit's start and end, as
// measured: with heads of 128 a pair's step takes its products' time (2.4 us), a single
// tile's its bytes' (1.5 us), and 7:4 beats 3:2 (12 chunks of 1 to 200 tokens over 500 to
// 30000: 210 us against 223; no difference where all units are alike); with heads of 64
// 3:2 beats 7:4 (12 chunks of 1 to 1000 over 100 to 8000: 114 us against 124). A unit's
// start and end take three to four steps of a single tile (24 prompts of 61 to 1500 tokens:
// 101 us with 7 for 3:2, 107 with 4, 99 with 10).
template <int D>
struct TcCost {
    static constexpr int kPair = D == 128 ? 7 : 3, kOne = D == 128 ? 4 : 2;
    static constexpr int kUnit = D == 128 ? 14 : 7;
};

// The same, fp32: units of one tile, whose start and end take a step's time.
constexpr int kFKT = 64;
struct FCost {
    static constexpr int kPair = 1, kOne = 1, kUnit = 1;
};

// A place in the row of all units' steps, and the walk over it that every role makes. A
// unit's step 0 stands at its place F in the row, step j at F + start + j w, and a run has
// the steps that stand in it. start is Cost::kUnit; with one unit per (sequence, KV head)
// and fewer of them than runs it is 0 where runs are shorter than three steps (those that start
// a unit would have no step besides), or where the longest unit fits into a run (all are about
// alike then, and each has a run for itself: nothing is cut). One token per sequence, bf16
// heads of 128, us with 0 / with kUnit:
//   runs of 2 steps: 8 units 14.8 / 15.9; 64 units of 0.2 to 1.8 times the mean 18.7 / 20.4;
//   144 units alike, runs of 4, 8, 32 steps: 18.2 / 25.3, 22.0 / 28.4, 55.3 / 57.8;
//   144 units of 0.2 to 1.8 times the mean, the same runs: 32.2 / 26.0, 38.1 / 29.4, 73.6 / 61.3;
//   8 units, runs of 4, 8, 20 steps: 18.2 / 16.2, 23.1 / 21.0, 41.5 / 41.6.
// Heads of 64 go the same way; in fp32, where a start costs a single step, units alike differ by
// up to 7 % either way (12 % in runs of 2 steps), ragged ones lose up to 18 % with 0.
// per_tile: query tokens of an MMA tile, U or U / 2. kSolo: no chunk of the call has more
// than one block of queries, of one tile (decode), which leaves little of the arithmetic.
template <int KT, class Cost, bool kSolo>
struct Walk {
    int b, h, qb;             // unit
    int32_t L, n;             // its sequence's length and chunk
    int j;                    // next step of the unit; -1: the unit is done
    int64_t F, end;           // the unit's place, this run's end
    int j0, j1, T, w;         // the current segment [j0, j1) of the unit's T steps of cost w
    int begin;                // what starting a unit costs

    SPLA_HD static int units(int32_t n, int U) {
        return kSolo ? 1 : (n + U - 1) / U;
    }
    // Whether the unit's queries reach past its first tile.
    SPLA_HD bool pair(int per_tile, int U) const {
        return !kSolo && (int64_t)qb * U + per_tile < n;
    }
    SPLA_HD int start() const { return kSolo ? begin : Cost::kUnit; }
    // Cost of a sequence's units before block qb, and of all of them, for one KV head (in
    // kSolo without the start).
    SPLA_HD static int64_t cost_before(int32_t base, int32_t qb, int U) {
        if (kSolo) return 0;
        return (int64_t)Cost::kUnit * qb + Cost::kPair * steps_before<KT>(base, qb, U);
    }
    SPLA_HD static int64_t cost_of(int32_t L, int32_t n, int per_tile, int U) {
        const int q = units(n, U) - 1;
        const int w = !kSolo && (int64_t)q * U + per_tile < n ? Cost::kPair : Cost::kOne;
        return cost_before(L - n, q, U) + (kSolo ? 0 : Cost::kUnit) + (int64_t)w * ((L + KT - 1) / KT);
    }
    // Next segment of this run; false at its end.
    SPLA_HD bool next(const CacheView& c, const ChunkArgs& a, int per_tile, int U) {
        if (j < 0) {                                  // the last unit is done: go to the next
            F += start() + (int64_t)T * w;
            j = 0;
            if (F < end && (kSolo || ++qb >= units(n, U))) {
                qb = 0;
                if (++h >= c.hkv) {
                    h = 0;
                    n = 0;
#pragma unroll 1
                    while (n == 0) {
                        if (++b >= c.batch) {
                            end = F;
                            return false;
                        }
                        chunk_of(c, a, b, &L, &n);
                    }
                }
            }
        }
        if (F >= end) return false;
        T = kSolo ? (L + KT - 1) / KT
                  : (int)((L - n + min((int64_t)(qb + 1) * U, (int64_t)n) + KT - 1) / KT);
        w = pair(per_tile, U) ? Cost::kPair : Cost::kOne;
        const int64_t room = end - F - start();
        j0 = j;
        j1 = room <= w ? 1 : room >= (int64_t)T * w ? T : (int)(((uint32_t)room + w - 1) / w);
        j1 = min(j1, T);
        if (j0 >= j1) return false;
        j = j1 < T ? j1 : -1;
        if (j > 0) end = F;                           // the run is over after this segment
        return true;
    }
    // Steps that query tile w of the unit takes part in end here.
    SPLA_HD int tile_end(int w, int per_tile, int U) const {
        const int64_t t0 = (int64_t)qb * U + (int64_t)w * per_tile;
        if (t0 >= n) return 0;
        const int64_t last = L - n + min(t0 + per_tile, (int64_t)n);
        return min(j1, (int)((last + KT - 1) / KT));
    }
    // For the join: what the current segment of run `run` leaves when its unit starts in it and
    // goes on past the run, of length C.
    SPLA_HD void note_cut(ChunkCut& cut, int run, int U, int G, int64_t C) const {
        if (j0 != 0 || j1 >= T) return;
        // from the next run's start to the unit's last step: less than the unit's cost
        const int64_t past = F + start() + (int64_t)(T - 1) * w - (int64_t)(run + 1) * C;
        cut.parts = 2 + (past < C ? 0 : (int)((uint32_t)past / (uint32_t)C));
        cut.rows = (int)min((int64_t)U, n - (int64_t)qb * U) * G;
        cut.b = b;
        cut.h = h;
        cut.t0 = qb * U;
    }

    // ---- finding a run's start. kSolo: the units, 2^22 at most, are counted in the same sum,
    // above the costs, which stay below 2^40: a bf16 sequence has 2^15 steps of kOne = 4 at
    // most, an fp32 one 2^16 of 1.
    static constexpr int64_t kSeq = kSolo ? 1ll << 40 : 0, kCosts = (1ll << 40) - 1;
    SPLA_HD static int64_t weigh(int32_t L, int32_t n, int hkv, int per_tile, int U) {
        return n ? hkv * (cost_of(L, n, per_tile, U) + kSeq) : 0;
    }
    // What starting a unit costs, by the sum over all sequences and the steps of the longest.
    SPLA_HD static int begin_of(int64_t W, int longest) {
        if (!kSolo || (W >> 40) >= kMaxRuns) return Cost::kUnit;
        const int64_t steps = W & kCosts;
        return steps < 3 * Cost::kOne * kMaxRuns ||
                       (int64_t)longest * Cost::kOne <= run_length(steps, 0) ? 0 : Cost::kUnit;
    }
    // A sum of weigh() as a cost, the starts included.
    SPLA_HD static int64_t total(int64_t sum, int begin) {
        return kSolo ? (sum & kCosts) + begin * (sum >> 40) : sum;
    }
    SPLA_HD static int64_t run_length(int64_t W, int begin) {
        // a run has the place of a step at least: steps stand no further apart
        int64_t C = max((W + kMaxRuns - 1) / kMaxRuns,
                        (int64_t)(begin + (kSolo ? Cost::kOne : max(Cost::kPair, Cost::kOne))));
        // whole steps: as many in the longest run, and the others' ends, with them, in fewer
        // units (one token over 4000: 17.5 us with runs of 7/4 steps, 15.8 with 8/4)
        if (kSolo) C = (C + Cost::kOne - 1) / Cost::kOne * Cost::kOne;
        return C;
    }
    // Goes to the run [f0, f0 + C) of all W, which starts `at` past the first unit of
    // sequence b0, within the units of the `per` sequences from there.
    SPLA_HD void seek(const CacheView& c, const ChunkArgs& a, int b0, int per, int64_t at,
                      int64_t f0, int64_t C, int64_t W, int start_cost, int per_tile, int U) {
#pragma unroll 1
        for (int i = 0; i < per; ++i) {
            b = b0 + i;
            chunk_of(c, a, b, &L, &n);
            if (!n) continue;
            const int32_t base = L - n;
            const int64_t one = cost_of(L, n, per_tile, U) + (kSolo ? start_cost : 0);
            if (at >= one * c.hkv) {
                at -= one * c.hkv;
                continue;
            }
#pragma unroll 1
            for (h = 0; at >= one; ++h) at -= one;
            int32_t lo = 0, hi = units(n, U) - 1;           // (kSolo: the block is 0)
#pragma unroll 1
            while (lo < hi) {
                const int32_t mid = (lo + hi + 1) / 2;
                if (cost_before(base, mid, U) <= at) lo = mid;
                else hi = mid - 1;
            }
            qb = lo;
            at -= cost_before(base, lo, U);                 // how far into the unit the run starts
            T = (int)((base + min((int64_t)(lo + 1) * U, (int64_t)n) + KT - 1) / KT);
            w = pair(per_tile, U) ? Cost::kPair : Cost::kOne;
            // the first step at or past that place, or the next unit
            const int64_t past = at - start_cost;
            j = at == 0 ? 0 : past <= w ? 1 : (int)(((uint32_t)past + w - 1) / w);
            if (j >= T) j = -1;
            break;
        }
        begin = start_cost;
        F = f0 - at;
        end = min(f0 + C, W);
    }
};

// This CTA's place, by all NT threads of it: contiguous sequences per thread, a scan over
// the CTA. *start (an empty run beforehand) and *run, its length, are for all after the
// call; scan and tops hold NT / 32 values each until then. Two barriers.
template <int NT, int KT, class Cost, bool kSolo>
__device__ __forceinline__ void find_run(const CacheView& c, const ChunkArgs& a, int per_tile,
                                         int U, int64_t* scan, int32_t* tops,
                                         Walk<KT, Cost, kSolo>* start, int64_t* run) {
    using W_ = Walk<KT, Cost, kSolo>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = ((unsigned)c.batch + NT - 1) / NT;
    int64_t mine = 0;
    int longest = 0;                                // (kSolo) steps of a unit
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b >= c.batch) break;
        int32_t L, n;
        const int32_t bad = chunk_of(c, a, b, &L, &n);
        if (bad && blockIdx.x == 0) set_status(a.status, bad);
        mine += W_::weigh(L, n, c.hkv, per_tile, U);
        if (kSolo && n) longest = max(longest, (L + KT - 1) / KT);
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    if (kSolo) longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 31) {
        scan[warp] = upto;
        if (kSolo) tops[warp] = longest;
    }
    __syncthreads();
    int64_t W = 0;
#pragma unroll 4
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) upto += scan[w];
        W += scan[w];
        if (kSolo) longest = max(longest, tops[w]);
    }
    const int begin = W_::begin_of(W, longest);
    W = W_::total(W, begin);
    mine = W_::total(mine, begin);
    upto = W_::total(upto, begin);
    const int64_t C = W_::run_length(W, begin);
    const int64_t f0 = (int64_t)blockIdx.x * C;
    if (mine && f0 < W && upto - mine <= f0 && f0 < upto) {
        W_ w;
        w.seek(c, a, tid * per, per, f0 - (upto - mine), f0, C, W, begin, per_tile, U);
        *start = w;
        *run = C;
    }
    __syncthreads();
}

// Whether sums scaled by the maximum m, with probabilities that add up to l, have a part in
// their row: not where no token was seen (m = -inf, l = 0); where all logits were NaN, l is.
__device__ __forceinline__ bool has_part(float m, float l) { return m != -SPLA_INF || l != l; }

// What infinities and NaN taken out of V (first[kind][dim]: the first token that holds
// +inf, -inf, NaN there) add to a row at position pos.
__device__ __forceinline__ float note_term(int32_t pinf, int32_t ninf, int32_t nan, int pos) {
    float add = 0.f;
    if (pinf <= pos) add += SPLA_INF;
    if (ninf <= pos) add -= SPLA_INF;
    if (nan <= pos) add = __int_as_float(0x7fffffff);
    return add;
}

// Join launch for units of `rows` rows at most.
cudaError_t launch_chunk_combine(const CacheView& c, int dtype, const ChunkArgs& a, int rows,
                                 cudaStream_t s);

}  // namespace spla
