// The split of chunk attention over the GPU, run on the host: every run's start as the CTA's
// threads find it and its walk, compared with the units' steps one after another.
#include <vector>

#include "chunk_attn.cuh"

using namespace spla;

#define CHECK(x) \
    do { if (!(x)) return __LINE__; } while (0)

template <int NT, int KT, class Cost, bool kSolo>
static int check(const CacheView& c, const ChunkArgs& a, int per_tile, int U, int64_t* longest) {
    using W_ = Walk<KT, Cost, kSolo>;
    // find_run's scan
    const int per = (c.batch + NT - 1) / NT;
    std::vector<int64_t> mine(NT), upto(NT);
    int64_t sum = 0;
    int longest_unit = 0;
    for (int t = 0; t < NT; ++t) {
        for (int i = 0; i < per && t * per + i < c.batch; ++i) {
            int32_t L, n;
            chunk_of(c, a, t * per + i, &L, &n);
            mine[t] += W_::weigh(L, n, c.hkv, per_tile, U);
            if (n && (L + KT - 1) / KT > longest_unit) longest_unit = (L + KT - 1) / KT;
        }
        upto[t] = sum += mine[t];
    }
    const int begin = W_::begin_of(sum, longest_unit);
    const int64_t W = W_::total(sum, begin), C = W_::run_length(W, begin);
    for (int t = 0; t < NT; ++t) {
        mine[t] = W_::total(mine[t], begin);
        upto[t] = W_::total(upto[t], begin);
    }
    CHECK((int64_t)kMaxRuns * C >= W);

    // where the units' steps have got to
    int b = -1, h = c.hkv - 1, qb = 0, units = 0, j = 0, T = 0;
    int32_t L = 0, n = 0;
    auto next_unit = [&]() {
        j = 0;
        if (++qb >= units) {
            qb = 0;
            if (++h >= c.hkv) {
                h = 0;
                do {
                    if (++b >= c.batch) return false;
                    chunk_of(c, a, b, &L, &n);
                } while (n == 0);
                units = (int)(((int64_t)n + U - 1) / U);
            }
        }
        const int64_t last = (int64_t)L - n + ((int64_t)(qb + 1) * U < n ? (int64_t)(qb + 1) * U : n);
        T = (int)((last + KT - 1) / KT);
        return true;
    };
    bool more = next_unit();
    if (kSolo) CHECK(!more || units == 1);
    // the cut unit whose join is awaited
    int cut_run = -1, cut_parts = 0, found = 0;
    for (int run = 0; run < kMaxRuns; ++run) {
        const int64_t f0 = run * C;
        W_ w;
        w.j = 0;
        w.F = w.end = 0;
        int finders = 0;
        for (int t = 0; t < NT; ++t)
            if (mine[t] && f0 < W && upto[t] - mine[t] <= f0 && f0 < upto[t]) {
                ++finders;
                w.seek(c, a, t * per, per, f0 - (upto[t] - mine[t]), f0, C, W, begin, per_tile, U);
            }
        CHECK(finders == (f0 < W));
        ChunkCut cut = {};
        int slots[2] = {}, segments = 0;
        int64_t cost = 0;
        while (w.next(c, a, per_tile, U)) {
            CHECK(more);
            CHECK(w.b == b && w.h == h && w.qb == qb && w.L == L && w.n == n && w.T == T);
            CHECK(w.j0 == j && w.j1 > w.j0 && w.j1 <= T);
            const bool pair = w.pair(per_tile, U);
            CHECK(pair == (!kSolo && (int64_t)qb * U + per_tile < n));
            for (int x = 0; x < U / per_tile; ++x) {        // steps a query tile takes part in
                const int64_t t0 = (int64_t)qb * U + (int64_t)x * per_tile;
                const int64_t hi = t0 + per_tile < n ? t0 + per_tile : n;
                const int64_t e = t0 < n ? (L - n + hi + KT - 1) / KT : 0;
                CHECK(w.tile_end(x, per_tile, U) == (e < w.j1 ? e : w.j1));
            }
            const bool whole = w.j0 == 0 && w.j1 == T;
            if (!whole) CHECK(slots[w.j0 == 0]++ == 0);     // a place of its own for each partial
            w.note_cut(cut, run, U, c.group, C);
            if (w.j0 > 0) {                                 // goes on with the unit that was cut
                CHECK(segments == 0 && cut_run >= 0 && run == cut_run + found);
                ++found;
            }
            if (w.j0 == 0 && w.j1 < T) {
                CHECK(cut.b == b && cut.h == h && cut.t0 == qb * U);
                const int64_t left = n - (int64_t)qb * U;
                CHECK(cut.rows == (left < U ? left : U) * c.group);
                CHECK(cut.parts >= 2 && run + cut.parts <= kMaxRuns);
                CHECK(cut_run < 0);
                cut_run = run;
                cut_parts = cut.parts;
                found = 1;
            }
            cost += (int64_t)(w.j1 - w.j0) * w.w + (w.j0 == 0 ? w.start() : 0);
            ++segments;
            if (w.j1 == T) {
                if (cut_run >= 0) CHECK(found == cut_parts);
                cut_run = -1;
                more = next_unit();
            } else {
                j = w.j1;
                CHECK(!w.next(c, a, per_tile, U));          // the run ends within a unit
                break;
            }
        }
        CHECK(cut.parts == 0 || cut_run == run);
        CHECK(cost <= C + Cost::kUnit + (Cost::kPair > Cost::kOne ? Cost::kPair : Cost::kOne));
        if (cost > *longest) *longest = cost;
    }
    CHECK(!more && cut_run < 0);
    return 0;
}

// 0, or the line of the check that failed. f32: the fp32 kernel's split, else bf16's.
extern "C" int chunk_split_check(int f32, int d, int batch, int hkv, int group, int bs, int mbp,
                                 int max_new, const int32_t* lens, const int32_t* n_new,
                                 int64_t* longest) {
    CacheView c = {};
    ChunkArgs a = {};
    c.lens = const_cast<int32_t*>(lens);
    c.batch = batch;
    c.hkv = hkv;
    c.group = group;
    c.hq = hkv * group;
    c.d = d;
    c.bs = bs;
    c.mbp = mbp;
    a.n_new = n_new;
    a.max_new = max_new;
    *longest = 0;
    const int64_t rows = (int64_t)max_new * group;
    if (f32) {
        const int U = (rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128) / group;
        return rows <= 64 ? check<256, kFKT, FCost, true>(c, a, U, U, longest)
                          : check<256, kFKT, FCost, false>(c, a, U, U, longest);
    }
    const int per_tile = 128 / group;
    if (rows > 128)
        return d == 128 ? check<384, kTcTile, TcCost<128>, false>(c, a, per_tile, 2 * per_tile, longest)
                        : check<384, kTcTile, TcCost<64>, false>(c, a, per_tile, 2 * per_tile, longest);
    return d == 128 ? check<384, kTcTile, TcCost<128>, true>(c, a, per_tile, per_tile, longest)
                    : check<384, kTcTile, TcCost<64>, true>(c, a, per_tile, per_tile, longest);
}
