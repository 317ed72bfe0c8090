// loss_queue.cuh — in what pieces the cross entropy's gradient goes through the
// vocabulary, and the queue of its tiles: which there are, in what order, what each reads
// and writes.  Nothing here needs a GPU (tests/loss_queue_model.cpp runs it).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define LHS_HD __host__ __device__ __forceinline__
#else
#define LHS_HD inline
#endif

namespace lhs {

constexpr int kLossTile = 256;      // tokens, and vocabulary rows, of a tile of logits
constexpr int kLossSyncWarps = 16;  // warps of a pair of CTAs that take a tile out
constexpr int kLossParts = 2;       // parts of a tile's columns with statistics of their own

inline int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// Up to this many positions, g is held in two 16-bit terms: a tile has as many rows again, which
// would be empty, and they hold what the first term's rounding left.
constexpr int kLossTwin = kLossTile / 2;
// Of more positions g is one term, and its entries at the targets are kept apart in f32: they carry nearly all
// of the gradient (the other entries of a position add up to as much, spread over the vocabulary), and a
// frequent target's row of the table's gradient is a sum of many of them, with different signs.  Their
// products with x and with the table are sums over the positions alone (dtable: T rows by target, dx:
// a row each).  256 x 262,144 x 5,120 bf16, targets as in natural text: largest error of dtable in units
// of max(|element|, rms) 1.05 -> 0.0078, error in norm 2.3e-3 -> 1.66e-3, one rounding of the result.  Its
// price: 1.47 -> 1.51 ms (8,192 x 151,936 x 896 3.83 -> 3.90, 628 positions 0.50 -> 0.53).
constexpr int kTileK = 64;          // of k of a stage
// The tensor cores cut their f32 sums instead of rounding them: each of a step's 17 addends at 2^-25 of
// the largest.  512 terms of one sign fall short by 2.6e-6 of their sum in f16, whose products have that
// many bits to lose, and by 2e-7 in bf16; a longer sum by as much for every 512 (hidden 5,376 in one sum: 5.7e-6
// of the loss; f32 on the CUDA cores 1e-6).  Logits are summed 512 of k at a time, and those sums added up, rounded,
// in registers: for g as for the statistics, whose lse they are compared with (one long sum for g left
// a row's probabilities short of 1, always to one side: 6e-5 in bf16 and 8e-4 in f16 for logits
// of 30, hidden 5,376 and terms of one sign).
constexpr int kChunk = 512 / kTileK;
// Sums over positions (dtable) or rows of a piece (dx) are as long as the call is (2^19 positions of one sign in
// one sum: 1.4e-3 short in bf16, 3.1e-3 in f16), and are cut into longer parts: 2,048 terms of one sign fall
// short by 1e-5 (f16).  (1,024: 1 x 151,936 x 896, whose dx has 1,216 in a sum, 224 -> 260 us.)
constexpr int kLongChunk = 2048 / kTileK;

// What a call's tiles are made of.
struct LossQueue {
    int64_t Tpad;           // positions rounded up to whole tiles (one at least)
    int64_t V, vt;          // vocabulary rows; tiles of them
    int32_t H;              // hidden
    int64_t piece;          // vocabulary rows of a piece, a multiple of kLossTile
    int pieces;
    int ahead, slots;       // pieces whose logits precede a piece's products; whose g is kept
    int splits;             // dx's sums are split along a piece's rows
    int64_t items;          // tiles of all products
    int64_t n_sync;         // words that CTAs tell one another by
};

// Pieces: small ones leave g and the table's rows in L2 between the logits and the
// products, but add dx up more often and make pairs wait for one another more.  At
// 8,192 x 151,936 x 896 under the power cap: 3 pieces 4.55 ms, 6 4.61, 10 4.54, 20
// 4.42, 40 4.60, 80 4.68.  Where logits are few, pieces are at least two waves of tiles
// (256 x 262,144 x 5,120: 4 pieces 1.45 ms, 10 1.48, 16 1.51; 1 x 151,936 x 896: 4
// pieces 204 us, 10 249).
constexpr int64_t kPieces = 18;
constexpr int64_t kPieceBytes = 512ll << 20;  // of g, at most, as several pieces' is kept
constexpr int kAhead = 3;
constexpr int kPairs = 76;                    // of CTAs that run at once

inline void choose_pieces(LossQueue *p) {
    const int64_t tiles = p->Tpad / kLossTile * p->vt;
    int64_t n = tiles / (2 * kPairs) < kPieces ? tiles / (2 * kPairs) : kPieces;
    const int64_t least = (2 * p->Tpad * p->V + kPieceBytes - 1) / kPieceBytes;
    if (n < least) n = least;
    if (n > (p->vt + 1) / 2) n = (p->vt + 1) / 2;  // two tiles' rows at least
    if (n < 1) n = 1;
    p->piece = round_up((p->V + n - 1) / n, kLossTile);
    p->pieces = static_cast<int>((p->V + p->piece - 1) / p->piece);
    const int64_t blocks = p->Tpad / kLossTile, gt = p->piece / kLossTile, ht = (p->H + kLossTile - 1) / kLossTile;
    const int64_t kh = (p->H + 63) / 64, kp = (p->V < p->piece ? p->V + 63 : p->piece) / 64;
    const int64_t share = (blocks * gt * kh + blocks * ht * kp + gt * ht * (p->Tpad / 64)) / kPairs + 1;
    // a tile of dx takes no longer than a share; the logits run ahead of the products by the pieces
    // that their tiles take
    const int64_t most = share > 16 ? share : 16;
    int64_t splits = (kp + most - 1) / most;
    if (splits > 32) splits = 32;
    if (splits > kp) splits = kp;
    p->splits = static_cast<int>(splits < 1 ? 1 : splits);
    const int64_t ahead = kAhead + kh / share;
    p->ahead = static_cast<int>(ahead < 6 ? ahead : 6);
    if (p->ahead > p->pieces) p->ahead = p->pieces;
    p->slots = p->ahead + 2 < p->pieces ? p->ahead + 2 : p->pieces;
    // the queue, two counters to a piece, a word to each warp's part of dx's sums
    p->n_sync = 1 + 2ll * p->pieces + blocks * ht * p->splits * kLossSyncWarps;
    p->items = blocks * p->vt + p->pieces * blocks * ht * p->splits + p->vt * ht;
}

// The same on the device.
struct LossShape {
    int64_t V, Tpad;
    int H, ht;               // hidden; tiles of it
    int64_t piece;           // rows of a piece, and tiles of them (statistics: one piece)
    int pieces, piece_tiles, last_tiles;
    bool want_dx, want_dtable;
    int ahead, slots, splits;
};
inline void shape_of(const LossQueue &q, bool grad, bool want_dx, bool want_dtable, LossShape *s) {
    s->V = q.V;
    s->Tpad = q.Tpad;
    s->H = q.H;
    s->ht = (q.H + kLossTile - 1) / kLossTile;
    s->piece = grad ? q.piece : q.V;
    s->pieces = grad ? q.pieces : 1;
    s->piece_tiles = static_cast<int>((s->piece + kLossTile - 1) / kLossTile);
    s->last_tiles = static_cast<int>((q.V - (s->pieces - 1) * s->piece + kLossTile - 1) / kLossTile);
    s->want_dx = want_dx;
    s->want_dtable = want_dtable;
    s->ahead = q.ahead;
    s->slots = q.slots;
    s->splits = q.splits;
}

enum { kLogits = 0, kDx = 1, kDtable = 2 };
// Stages of a tile whose products make one sum in the tensor cores.
template <int MODE>
LHS_HD int chunk_of(int kind) {
    return MODE == 0 || kind == kLogits ? kChunk : kLongChunk;
}

// A tile to work on, as the scheduler hands it out.
struct alignas(16) Item {
    int kind;     // -1: the end
    int piece;
    int m;        // tile of M: block of tokens, or of the piece's rows
    int n;        // tile of N: of the piece's rows (logits), or of hidden
    int split;    // dx; dtable: whether a row of the tile is a target
    int k0, k1;   // stages
    int width;    // N of the MMAs, a multiple of 32
};
static_assert(sizeof(Item) == 32, "two words of 16 bytes");

// ---------------------------------------------------------------------------
// items
// ---------------------------------------------------------------------------
// The queue: g of the first `ahead` pieces; then each piece's products, dx first,
// followed by g of the piece `ahead` of it.
// Quotients of numbers below 2^31: with 2^(l-1) < d <= 2^l and mul = ceil(2^(31+l) / d), which is
// below 2^32, n mul / 2^(31+l) exceeds n / d by less than n / 2^(31+l) < 1 / d.
struct Divisor {
    uint32_t d, mul, shift;
    LHS_HD void set(uint32_t d_) {
        d = d_;
        uint32_t l = 0;
        while (l < 31 && (1u << l) < d) ++l;
        shift = 31 + l;
        mul = static_cast<uint32_t>(((1ull << shift) + d - 1) / d);
    }
    LHS_HD uint32_t of(uint32_t n) const {
        return static_cast<uint32_t>((static_cast<uint64_t>(n) * mul) >> shift);
    }
};
struct Work {
    uint32_t blocks, total;
    int token_stages;     // k of dtable
    int turn, gap;        // from stage `turn` on, tokens lie `gap` rows further on (the second terms)
    uint32_t before;      // g of the first pieces
    Divisor block, head, period, ht, splits;  // what the scheduler divides by
};
LHS_HD int tiles_of(const LossShape &p, int piece) {
    return piece + 1 < p.pieces ? p.piece_tiles : p.last_tiles;
}
LHS_HD int stages_of(const LossShape &p, int piece) {
    const int64_t rows = piece + 1 < p.pieces ? p.piece : p.V - piece * p.piece;
    return static_cast<int>((rows + kTileK - 1) / kTileK);
}
LHS_HD int splits_of(const LossShape &p, int piece) {
    const int stages = stages_of(p, piece);
    return p.splits < stages ? p.splits : stages;
}
LHS_HD uint32_t n_dx_of(const LossShape &p, const Work &w, int piece) {
    return p.want_dx ? w.blocks * p.ht * splits_of(p, piece) : 0u;
}
LHS_HD uint32_t n_products_of(const LossShape &p, const Work &w, int piece) {
    return n_dx_of(p, w, piece) + (p.want_dtable ? static_cast<uint32_t>(tiles_of(p, piece)) * p.ht : 0u);
}
template <int MODE>
LHS_HD Work work_of(const LossShape &p, int count) {
    Work w = {};
    w.blocks = count > 0 ? (static_cast<uint32_t>(count) + kLossTile - 1) / kLossTile : 1u;
    w.token_stages = count > 0 ? (count + kTileK - 1) / kTileK : 1;  // (without any position one of zeros)
    w.turn = w.token_stages;
    if (MODE == 1 && count <= kLossTwin) {
        w.gap = kLossTwin - w.turn * kTileK;
        w.token_stages *= 2;
    }
    w.total = w.blocks * (static_cast<uint32_t>(p.pieces - 1) * p.piece_tiles + p.last_tiles);
    if (MODE == 1) {
        w.before = p.ahead < p.pieces ? w.blocks * p.ahead * p.piece_tiles : w.total;
        w.total += static_cast<uint32_t>(p.pieces - 1) * n_products_of(p, w, 0) + n_products_of(p, w, p.pieces - 1);
    }
    return w;
}
template <int MODE>
LHS_HD void set_divisors(const LossShape &p, Work &w) {
    w.block.set(w.blocks);
    if (MODE == 1) {
        w.head.set(w.blocks * p.piece_tiles);
        w.period.set(n_products_of(p, w, 0) + w.blocks * p.piece_tiles);
        w.ht.set(p.ht);
        w.splits.set(p.splits);
    }
}
LHS_HD int width_of(int H, int tile) {
    const int left = H - tile * kLossTile;
    return left >= kLossTile ? kLossTile : (left + 31) / 32 * 32;
}
template <int MODE>
LHS_HD Item item_of(const LossShape &p, const Work &w, uint32_t i) {
    Item t = {};
    bool logits = true;
    if (MODE == 1) {
        if (i < w.before) {
            t.piece = w.head.of(i);
            i -= t.piece * w.head.d;
        } else {
            i -= w.before;
            // pieces whose products, and the logits that follow them, are whole
            const int whole = p.pieces - p.ahead - 1;
            int q = 0;
            if (whole > 0) {
                q = static_cast<int>(w.period.of(i));
                q = q < whole ? q : whole;
                i -= q * w.period.d;
            }
            for (;; ++q) {  // a few steps at the end
                const uint32_t nq = n_products_of(p, w, q);
                if (i < nq) {
                    t.piece = q;
                    logits = false;
                    break;
                }
                i -= nq;
                const uint32_t g = q + p.ahead < p.pieces ? w.blocks * tiles_of(p, q + p.ahead) : 0u;
                if (i < g) {
                    t.piece = q + p.ahead;
                    break;
                }
                i -= g;
            }
        }
    }
    if (logits) {
        t.kind = kLogits;
        t.n = w.block.of(i);
        t.m = i - t.n * w.blocks;
        t.k1 = (p.H + kTileK - 1) / kTileK;
        t.width = kLossTile;
        return t;
    }
    const uint32_t n_dx = n_dx_of(p, w, t.piece);
    t.kind = i < n_dx ? kDx : kDtable;
    if (i >= n_dx) i -= n_dx;
    const uint32_t above = w.ht.of(i);
    t.n = i - above * p.ht;
    t.width = width_of(p.H, t.n);
    if (t.kind == kDx) {
        const int splits = splits_of(p, t.piece), stages = stages_of(p, t.piece);
        const bool same = splits == p.splits;  // but perhaps in the last piece
        t.m = same ? w.splits.of(above) : above / splits;
        t.split = above - t.m * splits;
        // (stages * splits stays far below 2^31: pieces are rows below 2^31 / 64 stages, splits at most 32)
        t.k0 = same ? w.splits.of(stages * t.split) : stages * t.split / splits;
        t.k1 = same ? w.splits.of(stages * (t.split + 1)) : stages * (t.split + 1) / splits;
    } else {
        t.m = above;
        t.k1 = w.token_stages;
    }
    return t;
}

}  // namespace lhs
