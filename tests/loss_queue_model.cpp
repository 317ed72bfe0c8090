// The queue of the cross entropy's tiles, run on the host from the kernel's own
// functions: every tile comes once, lies within its tensors, and waits only for
// tiles before it.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <tuple>
#include <vector>

#include "loss_queue.cuh"

using namespace lhs;

#define CHECK(c)                                                                                               \
    do {                                                                                                       \
        if (!(c)) {                                                                                            \
            printf("line %d: %s (tokens %lld of %lld, vocab %lld, hidden %d, pieces %d, ahead %d, splits %d, item %u)\n", __LINE__, \
                   #c, static_cast<long long>(count), static_cast<long long>(q.Tpad), static_cast<long long>(q.V), q.H,     \
                   q.pieces, q.ahead, q.splits, at);                                                           \
            exit(1);                                                                                           \
        }                                                                                                      \
    } while (0)

static LossQueue queue_of(int64_t tokens, int64_t vocab, int32_t hidden) {
    LossQueue q = {};
    q.Tpad = round_up(tokens, kLossTile);
    q.V = vocab;
    q.vt = (vocab + kLossTile - 1) / kLossTile;
    q.H = hidden;
    choose_pieces(&q);
    return q;
}

// One tile by itself: what the kernel reads and writes for it.
static void within(const LossQueue &q, const LossShape &s, const Work &w, const Item &t, int64_t count, uint32_t at) {
    CHECK(t.kind == kLogits || t.kind == kDx || t.kind == kDtable);
    CHECK(t.piece >= 0 && t.piece < s.pieces && t.m >= 0 && t.n >= 0);
    CHECK(t.k0 >= 0 && t.k1 > t.k0);
    CHECK(t.width >= 32 && t.width <= kLossTile && t.width % 32 == 0);
    const int64_t row = t.piece * s.piece, rows = s.V - row < s.piece ? s.V - row : s.piece;
    const int slot = t.piece % s.slots;
    CHECK(row >= 0 && rows > 0 && slot >= 0 && slot < q.slots);
    if (t.kind == kLogits) {
        CHECK(t.m < static_cast<int>(w.blocks) && (t.m + 1) * kLossTile <= q.Tpad);
        CHECK(t.n < tiles_of(s, t.piece) && static_cast<int64_t>(t.n) * kLossTile < rows);
        CHECK((t.n + 1) * static_cast<int64_t>(kLossTile) <= s.piece);  // g's tile lies in the piece's columns
        CHECK(t.k0 == 0 && t.k1 == (q.H + kTileK - 1) / kTileK);
    } else {
        CHECK(t.n < s.ht && t.n * kLossTile + t.width >= (q.H < (t.n + 1) * kLossTile ? q.H : (t.n + 1) * kLossTile));
    }
    if (t.kind == kDx) {
        CHECK(s.want_dx && t.m < static_cast<int>(w.blocks) && t.split >= 0 && t.split < q.splits);
        CHECK(static_cast<int64_t>(t.k1 - 1) * kTileK < rows);  // no stage lies wholly behind the piece's rows
        CHECK((static_cast<int64_t>(t.m) * s.ht + t.n) * q.splits + t.split <
              q.Tpad / kLossTile * s.ht * q.splits);             // its counters
    }
    if (t.kind == kDtable) {
        CHECK(s.want_dtable && t.m < tiles_of(s, t.piece) && static_cast<int64_t>(t.m) * kLossTile < rows);
        for (int k = t.k0; k < t.k1; ++k) {
            const int64_t r = static_cast<int64_t>(k) * kTileK + (k >= w.turn ? w.gap : 0);
            CHECK(r >= 0 && r + kTileK <= q.Tpad);
            if (k > t.k0 + 8 && k < t.k1 - 8) k = t.k1 - 8;
        }
    }
    // a part of a sum for every chunk
    const int chunk = chunk_of<1>(t.kind);
    CHECK(chunk > 0 && chunk_of<0>(kLogits) == chunk_of<1>(kLogits));
}

static void whole(const LossQueue &q, const LossShape &s, int64_t count) {
    uint32_t at = 0;
    Work w = work_of<1>(s, static_cast<int>(count));
    set_divisors<1>(s, w);
    CHECK(w.total <= static_cast<uint64_t>(q.items));
    std::set<std::tuple<int, int, int, int, int>> seen;
    struct Span {
        uint32_t first = UINT32_MAX, last = 0;
        uint32_t n = 0;
        void add(uint32_t i) {
            if (i < first) first = i;
            if (i > last) last = i;
            ++n;
        }
    };
    std::vector<Span> g(s.pieces), products(s.pieces);
    std::map<std::tuple<int, int, int>, std::vector<std::pair<uint32_t, int>>> sums;  // dx: of (m, n, split), pieces in the queue's order
    std::map<std::tuple<int, int, int>, int> stages;                                  // dx: of (piece, m, n)
    for (at = 0; at < w.total; ++at) {
        const Item t = item_of<1>(s, w, at);
        within(q, s, w, t, count, at);
        CHECK(seen.insert({t.kind, t.piece, t.m, t.n, t.split}).second);
        if (t.kind == kLogits) g[t.piece].add(at);
        else products[t.piece].add(at);
        if (t.kind == kDx) {
            sums[{t.m, t.n, t.split}].push_back({at, t.piece});
            stages[{t.piece, t.m, t.n}] += t.k1 - t.k0;
        }
    }
    for (int k = 0; k < s.pieces; ++k) {
        CHECK(g[k].n == w.blocks * tiles_of(s, k));                        // what the products wait for
        CHECK(products[k].n == n_products_of(s, w, k));                    // what the slot's next g waits for
        CHECK(g[k].last < products[k].first);                              // g before its products
        if (k + s.slots < s.pieces) CHECK(products[k].last < g[k + s.slots].first);  // the slot's readers before its next g
        if (s.want_dx)
            for (int m = 0; m < static_cast<int>(w.blocks); ++m)
                for (int n = 0; n < s.ht; ++n) CHECK((stages[{k, m, n}]) == stages_of(s, k));
    }
    for (const auto &x : sums)  // a tile of dx's sums is added up piece by piece, each waiting for the one before
        for (size_t k = 0; k < x.second.size(); ++k) CHECK(x.second[k].second == static_cast<int>(k));
}

int main(int argc, char **argv) {
    const int rounds = argc > 1 ? atoi(argv[1]) : 1000;
    std::mt19937_64 rng(7);
    auto pick = [&](double lo, double hi) {
        return static_cast<int64_t>(lo * std::pow(hi / lo, std::uniform_real_distribution<double>(0, 1)(rng)));
    };
    LossQueue q = {};
    int64_t count = 0;
    uint32_t at = 0;
    for (int k = 0; k < 1000000; ++k) {  // quotients
        Divisor d;
        const uint32_t by = 1 + static_cast<uint32_t>(rng() >> (33 + rng() % 31));
        d.set(by > 0x7FFFFFFFu ? 0x7FFFFFFFu : by);
        uint32_t n = static_cast<uint32_t>(rng() & 0x7FFFFFFFu);
        if (k % 3 == 0) n = n / d.d * d.d - (n >= d.d);
        CHECK(d.of(n) == n / d.d);
    }
    for (int c = 0; c <= kLossTwin; ++c) {  // few positions: both terms' rows, each once
        q = queue_of(c > 0 ? c : 1, 300, 64);
        count = c;
        LossShape s = {};
        shape_of(q, true, true, true, &s);
        const Work w = work_of<1>(s, c);
        int rows[kLossTile] = {};
        for (int k = 0; k < w.token_stages; ++k) {
            const int r = k * kTileK + (k >= w.turn ? w.gap : 0);
            CHECK(r >= 0 && r + kTileK <= kLossTile);
            for (int i = 0; i < kTileK; ++i) ++rows[r + i];
        }
        for (int r = 0; r < kLossTile; ++r) CHECK(rows[r] <= 1);
        for (int r = 0; r < c; ++r) CHECK(rows[r] == 1 && rows[kLossTwin + r] == 1);
    }
    long tiles = 0;
    auto run = [&](int64_t tokens, int64_t vocab, int32_t hidden, int64_t positions, bool dx, bool dtable) {
        q = queue_of(tokens, vocab, hidden);
        count = positions;
        CHECK(q.pieces >= 1 && q.piece % kLossTile == 0 && q.piece * q.pieces >= q.V && q.piece * (q.pieces - 1) < q.V);
        CHECK(q.ahead >= 1 && q.ahead <= q.pieces && q.slots >= 1 && q.slots <= q.pieces && q.splits >= 1);
        LossShape s = {};
        shape_of(q, true, dx, dtable, &s);
        if (q.items < 200000) {
            whole(q, s, count);
            tiles += q.items;
        } else {  // too many to visit: some of them
            Work w = work_of<1>(s, static_cast<int>(count));
            set_divisors<1>(s, w);
            CHECK(w.total > 0);
            for (int k = 0; k < 2000; ++k) {
                at = k < 2 ? (k ? w.total - 1 : 0) : static_cast<uint32_t>(rng() % w.total);
                within(q, s, w, item_of<1>(s, w, at), count, at);
            }
        }
        // statistics: the same logits, in one piece
        shape_of(q, false, false, false, &s);
        Work w = work_of<0>(s, static_cast<int>(count));
        set_divisors<0>(s, w);
        CHECK(w.total == w.blocks * static_cast<uint64_t>(q.vt));
        for (int k = 0; k < 50; ++k) {
            at = k < 2 ? (k ? w.total - 1 : 0) : static_cast<uint32_t>(rng() % w.total);
            const Item t = item_of<0>(s, w, at);
            CHECK(t.piece == 0 && t.n >= 0 && t.n < q.vt && t.m >= 0 && t.m < static_cast<int>(w.blocks));
        }
    };
    for (int k = 0; k < rounds; ++k) {
        const int64_t tokens = pick(1, k % 4 ? 3000 : 20000), vocab = pick(1, k % 3 ? 20000 : 400000);
        const int32_t hidden = static_cast<int32_t>(pick(1, k % 5 ? 1500 : 20000));
        const int64_t positions = k % 7 == 0 ? 0 : k % 3 == 0 ? tokens : static_cast<int64_t>(rng() % (tokens + 1));
        const bool dx = k % 5 != 1;
        run(tokens, vocab, hidden, positions, dx, !dx || k % 5 != 2);
    }
    // the edges: one piece, as many pieces as are kept, short last pieces, many positions, large tables
    const int64_t edges[][3] = {{1, 1, 1},          {1, 256, 64},        {128, 257, 8},       {129, 513, 300},   {256, 77824, 64},
                                {256, 78080, 64},   {2048, 262144, 768}, {256, 262144, 5120}, {8192, 151936, 896}, {1, 151936, 896},
                                {1 << 24, 2, 40},   {1 << 24, 700, 64},  {70000, 300, 16},    {4, 400003, 8},    {30, 700, 65536},
                                {40, 3000000, 768}, {1, 0x7FFFFFFF, 1},  {65537, 513, 257},   {4096, 65793, 64}};
    for (const auto &e : edges)
        for (int64_t positions : {int64_t(0), int64_t(1), e[0] / 2, e[0]})
            for (int which = 1; which < 4; ++which)
                run(e[0], e[1], static_cast<int32_t>(e[2]), positions < e[0] ? positions : e[0], which & 1, which & 2);
    printf("ok: %ld tiles\n", tiles);
}
