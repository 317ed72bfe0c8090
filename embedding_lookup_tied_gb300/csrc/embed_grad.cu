// embed_grad.cu — the gradient of the scaled embedding lookup: dtable[v] =
// scale * sum of dout over the positions that name row v.
//
// Counterpart of the lookup of ADR-0008 "Remote Embeddings and lm_head Service"
// (POST /v1/embed) with the scale of "embedding-inference — Port
// Specification" (Forward graph).
//
// Positions are ordered by (id, position); then every row of dout is read once,
// in runs of one id, summed in f32 registers and written once.  No sum depends on
// the order in which CTAs run: there are no floating-point atomics.
//  * Order.  Up to 8,192 ids a position's place is counted: the number of ids
//    below its own, and of equal ones before it (67 M comparisons at most, spread
//    over the chip, one launch).  More ids are sorted by two (18 bits of id) to
//    four passes over digits of up to 9 bits, stable, two launches a pass.
//  * Sums.  A group of threads walks a run of 16 to 128 sorted positions over the
//    columns that it holds.  An id that lies within the run is finished there.  One
//    that crosses its ends leaves an f32 sum for each run, which a last kernel joins
//    in a fixed order: a warp to an id, or a CTA where it has many runs (the hottest
//    id of natural text names a tenth of all positions).
//  * The table's gradient is zeroed first, by further CTAs of the launches that order
//    the ids, which use little of the chip (8,192 ids: 402 MB of zeros, 55 us, beside
//    13 us of comparisons).
//
// The same order and sums serve the loss's gradient: weighted rows of residuals by target.
//
// What bounds it.  262,144 positions of 151,936 x 896 bf16: 168 us for 110 of HBM; the
// sums read 470 MB in 95 us (5.6 TB/s with what they write), the sort takes 50 us
// beside the zeros' 40, the join 20.  8,192 positions into 262,144 x 768 bf16: 73 us
// for 63, nearly all of it zeros.
#include "train.cuh"

namespace lhs {
namespace {

constexpr int kRankMost = 8192;     // ids whose places are counted
constexpr int kRankThreads = 512;   // 32 ids to a CTA, its warps share the others
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9;
constexpr int kBins = 1 << kDigitBits;
constexpr int kSortSteps = 8;       // keys of a thread in a round
constexpr int kRound = kSortThreads * kSortSteps;
constexpr int kMostTiles = 128;     // each reads the counts of all
constexpr int kMostRun = 128;       // sorted positions that a group of threads sums
constexpr int kSumThreads = 128;
constexpr int kJoinWarps = 16;
constexpr int kJoinCols = 128;      // columns of a warp, four to a lane

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Zeros that CTAs `first` and up of a launch write, kZeroWords words of 16 bytes to a
// thread.  Many short CTAs walk through memory in order: 402 MB in 55 us; a CTA to an
// equal range each 69 us, one wave of CTAs striding through it 63 us.
constexpr int kZeroWords = 2;
struct Zero {
    uint4 *p;
    size_t n16;       // 16-byte words
    uint8_t *tail;    // what is left of the last one
    int ntail;
    int first;
};
__device__ __forceinline__ void write_zeros(const Zero &z) {
    const size_t c = blockIdx.x - z.first, i0 = c * (kZeroWords * blockDim.x) + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kZeroWords; ++k)
        if (i0 + k * blockDim.x < z.n16) z.p[i0 + k * blockDim.x] = make_uint4(0u, 0u, 0u, 0u);
    if (c == 0 && static_cast<int>(threadIdx.x) < z.ntail) z.tail[threadIdx.x] = 0;
}

__global__ void __launch_bounds__(512) zero_kernel(const Zero z) {
    pdl_wait();
    write_zeros(z);
}

// The id of a position that takes part, else vocab, which sorts last.
__device__ __forceinline__ uint32_t key_of(int32_t id, uint32_t vocab, int32_t ignore) {
    return static_cast<uint32_t>(id) < vocab && id != ignore ? static_cast<uint32_t>(id) : vocab;
}

// ---------------------------------------------------------------------------
// order of up to kRankMost ids
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kRankThreads)
    rank_ids_kernel(const int32_t *ids, int n, uint32_t vocab, int32_t ignore, uint32_t *keys, int32_t *order,
                    uint32_t *n_cross, const Zero z, int32_t *err) {
    extern __shared__ uint32_t all[];  // the keys, to a multiple of 32 with a larger value
    __shared__ uint32_t part[kRankThreads / 32][32];
    pdl_wait();
    pdl_trigger();
    if (static_cast<int>(blockIdx.x) >= z.first) return write_zeros(z);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kRankThreads / 32;
    const int padded = (n + 31) / 32 * 32;
    bool bad = false;
#pragma unroll 8
    for (int i = threadIdx.x; i < padded; i += kRankThreads) {
        const int32_t id = i < n ? ld_dep(ids + i) : ignore;
        const uint32_t k = key_of(id, vocab, ignore);
        if (k == vocab && id != ignore) bad = true;
        all[i] = i < n ? k : 0x7FFFFFFFu;
    }
    if (bad && blockIdx.x == 0) set_err(err, LHS_ERRBIT_BAD_TOKEN);
    if (blockIdx.x == 0 && threadIdx.x == 0) *n_cross = 0u;
    __syncthreads();
    const int i = blockIdx.x * 32 + lane;
    const uint32_t k = all[i];
    uint32_t rank = 0;
    // Words of four keys.  Those of other CTAs' positions lie wholly before this one's, where equal
    // keys count, or wholly behind.  Keys are below 2^31 (a pad equals vocab at most, which takes no
    // part in the order), so a < k is the sign of a - k: two instructions a key.
    const int own = static_cast<int>(blockIdx.x) * 8, words = padded / 4;
    const uint4 *word = reinterpret_cast<const uint4 *>(all);
    auto below = [](const uint4 &a, uint32_t b) {
        return ((a.x - b) >> 31) + ((a.y - b) >> 31) + ((a.z - b) >> 31) + ((a.w - b) >> 31);
    };
#pragma unroll 4
    for (int w = warp; w < own; w += warps) rank += below(word[w], k + 1u);
    if (warp < 8) {
        const uint4 a = word[own + warp];
        const int j = (own + warp) * 4;
        rank += (a.x < k || (a.x == k && j < i)) + (a.y < k || (a.y == k && j + 1 < i)) +
                (a.z < k || (a.z == k && j + 2 < i)) + (a.w < k || (a.w == k && j + 3 < i));
    }
#pragma unroll 4
    for (int w = own + 8 + warp; w < words; w += warps) rank += below(word[w], k);
    part[warp][lane] = rank;
    __syncthreads();
    if (warp == 0 && i < n) {
        for (int w = 1; w < warps; ++w) rank += part[w][lane];
        keys[rank] = k;
        order[rank] = i;
    }
}

// ---------------------------------------------------------------------------
// order of more ids: a stable pass over one digit
// ---------------------------------------------------------------------------
struct Pass {
    const int32_t *ids;        // the first pass reads them, later ones keys and order
    const uint32_t *keys_in;
    const int32_t *order_in;
    uint32_t *keys_out;
    int32_t *order_out;
    uint32_t *counts;          // [tiles][kBins]
    int64_t n, per;            // positions; of a tile, a multiple of kRound
    int tiles, shift, bits;
    uint32_t vocab;
    int32_t ignore;
    uint32_t *n_cross;
    int32_t *err;
};
__device__ __forceinline__ uint32_t pass_key(const Pass &p, int64_t i) {
    return p.ids ? key_of(ld_dep(p.ids + i), p.vocab, p.ignore) : ld_dep(p.keys_in + i);
}

__global__ void __launch_bounds__(kSortThreads) count_digits_kernel(const Pass p) {
    __shared__ uint32_t bins[kBins];
    pdl_wait();
    pdl_trigger();
    for (int b = threadIdx.x; b < kBins; b += kSortThreads) bins[b] = 0u;
    __syncthreads();
    const int64_t i0 = blockIdx.x * p.per, i1 = i0 + p.per < p.n ? i0 + p.per : p.n;
    const uint32_t mask = (1u << p.bits) - 1u;
    bool bad = false;
#pragma unroll 4
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads) {
        const uint32_t k = pass_key(p, i);
        if (p.ids && k == p.vocab && ld_dep(p.ids + i) != p.ignore) bad = true;
        atomicAdd(&bins[(k >> p.shift) & mask], 1u);
    }
    if (bad) set_err(p.err, LHS_ERRBIT_BAD_TOKEN);
    if (p.ids && blockIdx.x == 0 && threadIdx.x == 0) *p.n_cross = 0u;
    __syncthreads();
    for (int b = threadIdx.x; b < kBins; b += kSortThreads) p.counts[blockIdx.x * kBins + b] = bins[b];
}

// A tile's keys in rounds; warps hold consecutive keys, and a warp's steps follow
// each other, so equal digits keep their order.
__global__ void __launch_bounds__(kSortThreads) move_digits_kernel(const Pass p, const Zero z) {
    __shared__ uint32_t at[kSortWarps][kBins];  // keys of a digit that a warp has, then where its next one goes
    __shared__ uint32_t base[kBins];            // where the round's first key of a digit goes
    __shared__ uint32_t sums[kSortWarps];
    static_assert(kSortThreads == kBins, "a thread to a bin");
    pdl_wait();
    pdl_trigger();
    if (static_cast<int>(blockIdx.x) >= z.first) return write_zeros(z);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    {  // keys of smaller digits, and of this digit in tiles before
        uint32_t before = 0, total = 0;
#pragma unroll 8
        for (int t = 0; t < p.tiles; ++t) {
            const uint32_t c = ld_dep(p.counts + t * kBins + tid);
            total += c;
            before += t < static_cast<int>(blockIdx.x) ? c : 0u;
        }
        uint32_t incl = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        uint32_t smaller = incl - total;
        for (int w = 0; w < warp; ++w) smaller += sums[w];
        base[tid] = smaller + before;
    }
    const int64_t i0 = blockIdx.x * p.per, i1 = i0 + p.per < p.n ? i0 + p.per : p.n;
    const uint32_t mask = (1u << p.bits) - 1u;
    for (int64_t r = i0; r < i1; r += kRound) {
        for (int w = 0; w < kSortWarps; ++w) at[w][tid] = 0u;
        __syncthreads();
        uint32_t key[kSortSteps], place[kSortSteps];
        const int64_t first = r + warp * (32 * kSortSteps) + lane;
#pragma unroll
        for (int s = 0; s < kSortSteps; ++s) key[s] = first + s * 32 < i1 ? pass_key(p, first + s * 32) : 0u;
#pragma unroll
        for (int s = 0; s < kSortSteps; ++s) {
            const bool in = first + s * 32 < i1;
            const uint32_t d = in ? (key[s] >> p.shift) & mask : kBins;  // past the end: a digit of its own
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, d);
            const uint32_t had = in ? at[warp][d] : 0u;
            place[s] = had + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (in && lane == __ffs(same) - 1) at[warp][d] = had + __popc(same);
            __syncwarp();
        }
        __syncthreads();
        uint32_t next = base[tid];
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = at[w][tid];
            at[w][tid] = next;
            next += c;
        }
        base[tid] = next;
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kSortSteps; ++s) {
            const int64_t i = first + s * 32;
            if (i < i1) {
                const uint32_t o = at[warp][(key[s] >> p.shift) & mask] + place[s];
                p.keys_out[o] = key[s];
                p.order_out[o] = p.ids ? static_cast<int32_t>(i) : ld_dep(p.order_in + i);
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// sums
// ---------------------------------------------------------------------------
template <int BYTES>
struct Word;
template <>
struct Word<8> {
    using T = uint2;
};
template <>
struct Word<16> {
    using T = uint4;
};

// VEC consecutive values of a row, widened; added with a weight (1: a plain addition).
template <int DT, int VEC>
struct Pack;
template <int DT>
struct Pack<DT, 1> {
    typename Elem<DT>::T v;
    __device__ __forceinline__ void load(const typename Elem<DT>::T *p) { v = ld_dep(p); }
    __device__ __forceinline__ void add(float (&s)[1], float w) const { s[0] = fmaf(Elem<DT>::widen(v), w, s[0]); }
};
template <>
struct Pack<LHS_F32, 8> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = ld_dep(reinterpret_cast<const float4 *>(p));
        b = ld_dep(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void add(float (&s)[8], float w) const {
        s[0] = fmaf(a.x, w, s[0]), s[1] = fmaf(a.y, w, s[1]), s[2] = fmaf(a.z, w, s[2]), s[3] = fmaf(a.w, w, s[3]);
        s[4] = fmaf(b.x, w, s[4]), s[5] = fmaf(b.y, w, s[5]), s[6] = fmaf(b.z, w, s[6]), s[7] = fmaf(b.w, w, s[7]);
    }
};
template <int DT>
struct Pack<DT, 8> {
    uint4 w;
    __device__ __forceinline__ void load(const uint16_t *p) { w = ld_dep(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void add(float (&s)[8], float weight) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[2 * i] = fmaf(Elem<DT>::widen(static_cast<uint16_t>(u[i])), weight, s[2 * i]);
            s[2 * i + 1] = fmaf(Elem<DT>::widen(static_cast<uint16_t>(u[i] >> 16)), weight, s[2 * i + 1]);
        }
    }
};

// N values of the gradient.
template <int N, typename O>
struct Out {
    alignas(N == 8 ? 16 : sizeof(O)) O v[N];
    __device__ __forceinline__ void load(const O *o) {
        if (N == 8) {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(v) / 16); ++i)
                reinterpret_cast<uint4 *>(v)[i] = reinterpret_cast<const uint4 *>(o)[i];
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = o[i];
        }
    }
    // sums scaled, added to what was loaded if `add`, and stored
    __device__ __forceinline__ void store(O *o, const float (&s)[N], float scale, bool add) {
#pragma unroll
        for (int i = 0; i < N; ++i) put_rn(&v[i], fmaf(s[i], scale, add ? wide(v[i]) : 0.0f));
        if (N == 8) {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(v) / 16); ++i)
                reinterpret_cast<uint4 *>(o)[i] = reinterpret_cast<const uint4 *>(v)[i];
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] = v[i];
        }
    }
};

struct Sums {
    const uint32_t *keys;
    const int32_t *order;
    int64_t n;
    int run;                // sorted positions of a run, a multiple of 8
    int hidden, pitch;      // f32 sums of a run: rows of pitch, a multiple of 8
    int64_t vocab;
    float scale;
    int64_t dout_stride;
    bool accumulate;
    float *part;            // [2 x runs x pitch]: of a run's first id where it came from before, of its
                            // last where it goes on
    uint32_t *n_cross;      // runs whose last id starts there and goes on
    int32_t *cross;
    // sums of target rows: weighted, and not all rows of a table
    const int32_t *row_of;  // row of x of a position
    const float *weight;    // of a row of x
    int32_t *slot_of;       // [vocab] row of the sum of an id, told here; [tiles of them] 0 where one is
    int64_t out_pitch;
    bool by_id;             // sums lie by id, else by the sorted place of an id's last position in its first run
};
// Where the sum of an id goes.
template <bool TARGETS, typename O>
__device__ __forceinline__ O *sum_row(const Sums &p, O *out, uint32_t id, int64_t place) {
    return TARGETS ? out + (p.by_id ? static_cast<int64_t>(id) : place) * p.out_pitch : out + static_cast<int64_t>(id) * p.hidden;
}
__device__ __forceinline__ void tell_slot(const Sums &p, uint32_t id, int64_t place) {
    p.slot_of[id] = p.by_id ? static_cast<int32_t>(id) : static_cast<int32_t>(place);
    p.slot_of[p.vocab + id / kLossTile] = 0;
}

// A group of `cols` threads (a power of two) to a run; thread c of it holds
// columns VEC (c + cols blockIdx.y) and up.
template <int DT, int VEC, typename O, bool ADD, bool TARGETS>
__global__ void __launch_bounds__(kSumThreads)
    sum_runs_kernel(const Sums p, const typename Elem<DT>::T *dout, O *dtable, int cols) {
    constexpr int kAhead = ADD && sizeof(O) == 4 ? 4 : 8;  // rows (and sums to add to) asked for at a time
    extern __shared__ uint32_t lists[];
    pdl_wait();
    const uint32_t none = static_cast<uint32_t>(p.vocab);
    const int groups = kSumThreads / cols, group = threadIdx.x / cols, c = threadIdx.x % cols;
    uint32_t *key = lists + group * p.run;                                               // none past the end
    int32_t *pos = reinterpret_cast<int32_t *>(lists + (groups + group) * p.run);
    float *weight = reinterpret_cast<float *>(lists + (2 * groups + group) * p.run);     // (TARGETS)
    const int64_t run = static_cast<int64_t>(blockIdx.x) * groups + group;
    const int64_t i0 = run * p.run;
    for (int e = c; e < p.run; e += cols) {
        key[e] = i0 + e < p.n ? ld_dep(p.keys + i0 + e) : none;
        pos[e] = i0 + e < p.n ? ld_dep(p.order + i0 + e) : 0;
        if (TARGETS && key[e] != none) {
            pos[e] = ld_dep(p.row_of + pos[e]);
            weight[e] = ld_dep(p.weight + pos[e]);
        }
    }
    const uint32_t prev = i0 > 0 && i0 < p.n ? ld_dep(p.keys + i0 - 1) : none;
    const uint32_t next = i0 + p.run < p.n ? ld_dep(p.keys + i0 + p.run) : none;
    __syncthreads();
    if (key[0] == none) return;
    const uint32_t head = key[0] == prev ? prev : none;  // an id that came from the run before
    const int j = (c + cols * static_cast<int>(blockIdx.y)) * VEC;
    const bool in = j < p.hidden;
    float s[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) s[i] = 0.0f;
    auto keep = [&](int64_t row) {
        if (!in) return;
        float *o = p.part + row * p.pitch + j;
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = s[i];
    };
    for (int e0 = 0; e0 < p.run; e0 += kAhead) {
        uint32_t k[kAhead + 1];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) k[e] = key[e0 + e];
        k[kAhead] = e0 + kAhead < p.run ? key[e0 + kAhead] : next;
        Pack<DT, VEC> v[kAhead];
        Out<VEC, O> old[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            if (in && k[e] != none) v[e].load(dout + pos[e0 + e] * p.dout_stride + j);
            if (ADD && in && k[e] != none && k[e] != k[e + 1] && k[e] != head)
                old[e].load(dtable + static_cast<int64_t>(k[e]) * p.hidden + j);
        }
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            if (k[e] == none) continue;
            if (in) v[e].add(s, TARGETS ? weight[e0 + e] : 1.0f);
            if (k[e] == k[e + 1]) continue;
            // the id's last position
            if (k[e] == head) keep(2 * run);
            else if (in) old[e].store(sum_row<TARGETS>(p, dtable, k[e], i0 + e0 + e) + j, s, p.scale, ADD);
            if (TARGETS && k[e] != head && c == 0 && blockIdx.y == 0) tell_slot(p, k[e], i0 + e0 + e);
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[i] = 0.0f;
        }
    }
    if (key[p.run - 1] != none && key[p.run - 1] == next) {  // the last id goes on
        keep(next == head ? 2 * run : 2 * run + 1);
        if (next != head && c == 0 && blockIdx.y == 0) p.cross[atomicAdd(p.n_cross, 1u)] = static_cast<int32_t>(run);
    }
}

// The ids that cross runs: an item is one of them and kJoinCols columns, a warp to an
// item.  One with more than 32 further runs is shared by the CTA's warps, whose sums are
// joined in their order.  (Items of a CTA of 512 threads each: 61 us for 262,144 positions.)
template <typename O, bool TARGETS>
__global__ void __launch_bounds__(32 * kJoinWarps)
    join_runs_kernel(const Sums p, O *dtable, int col_blocks, bool vec) {
    __shared__ float4 part[kJoinWarps][32];
    __shared__ int ends[kJoinWarps];
    __shared__ int64_t large[kJoinWarps];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n_cross = ld_dep(p.n_cross), items = n_cross * col_blocks;
    auto starts = [&](int64_t run, uint32_t id) { return run * p.run < p.n && ld_dep(p.keys + run * p.run) == id; };
    // runs first, first + step, ... of those from `run` to run + more
    auto sum = [&](int64_t run, int64_t more, int first, int step, int j) -> float4 {
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (j < p.hidden) {
#pragma unroll 8
            for (int64_t r = first; r <= more; r += step) {
                const float4 a = ld_dep(reinterpret_cast<const float4 *>(p.part + (2 * (run + r) + (r == 0 ? 1 : 0)) * p.pitch + j));
                s.x += a.x, s.y += a.y, s.z += a.z, s.w += a.w;
            }
        }
        return s;
    };
    auto finish = [&](uint32_t id, int64_t run, int j, const float4 &s) {
        const float f[4] = {s.x, s.y, s.z, s.w};
        const int64_t place = (run + 1) * p.run - 1;
        O *o = sum_row<TARGETS>(p, dtable, id, place) + j;
        if (TARGETS && j == 0) tell_slot(p, id, place);
        if (vec && j < p.hidden) {  // hidden % 4 == 0: four values are 8 or 16 aligned bytes
            using W = typename Word<4 * sizeof(O)>::T;
            alignas(16) O v[4];
            if (p.accumulate) *reinterpret_cast<W *>(v) = *reinterpret_cast<const W *>(o);
#pragma unroll
            for (int k = 0; k < 4; ++k) put_rn(&v[k], fmaf(f[k], p.scale, p.accumulate ? wide(v[k]) : 0.0f));
            *reinterpret_cast<W *>(o) = *reinterpret_cast<const W *>(v);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (j + k < p.hidden) put_rn(o + k, fmaf(f[k], p.scale, p.accumulate ? wide(o[k]) : 0.0f));
        }
    };
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kJoinWarps; i0 < items; i0 += static_cast<int64_t>(gridDim.x) * kJoinWarps) {
        const int64_t item = i0 + warp;  // columns outermost, so that a large id's items go to different CTAs
        int64_t left = -1;
        if (item < items) {
            const int64_t run = ld_dep(p.cross + item % n_cross);
            const int j = static_cast<int>(item / n_cross) * kJoinCols + lane * 4;
            const uint32_t id = ld_dep(p.keys + (run + 1) * p.run - 1);
            const uint32_t m = __ballot_sync(0xFFFFFFFFu, starts(run + 1 + lane, id));
            if (m == 0xFFFFFFFFu) left = item;
            else finish(id, run, j, sum(run, __popc(m), 0, 1, j));
        }
        if (lane == 0) large[warp] = left;
        __syncthreads();
        for (int w = 0; w < kJoinWarps; ++w) {
            if (large[w] < 0) continue;
            const int64_t run = ld_dep(p.cross + large[w] % n_cross);
            const int j = static_cast<int>(large[w] / n_cross) * kJoinCols + lane * 4;
            const uint32_t id = ld_dep(p.keys + (run + 1) * p.run - 1);
            int64_t more = 0;
            for (;;) {
                const uint32_t m = __ballot_sync(0xFFFFFFFFu, starts(run + 1 + more + threadIdx.x, id));
                if (lane == 0) ends[warp] = __popc(m);
                __syncthreads();
                int n = 0;
                for (int k = 0; k < kJoinWarps; ++k) n += ends[k];
                more += n;
                __syncthreads();
                if (n < 32 * kJoinWarps) break;
            }
            part[warp][lane] = sum(run, more, warp, kJoinWarps, j);
            __syncthreads();
            if (warp == 0) {
                float4 s = part[0][lane];
                for (int k = 1; k < kJoinWarps; ++k) {
                    const float4 a = part[k][lane];
                    s.x += a.x, s.y += a.y, s.z += a.z, s.w += a.w;
                }
                finish(id, run, j, s);
            }
            __syncthreads();
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
struct Layout {
    size_t keys[2], order[2], counts, cross, n_cross, part, bytes;
    int64_t runs;
    int run, pitch, tiles;
};
Layout layout_of(int32_t hidden, int64_t n) {
    Layout l = {};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += align256(bytes);
        return o;
    };
    // Short runs spread few positions over the chip (8,192 positions added to a bf16 gradient: 23 us in
    // runs of 32, whose ids' rows are read one after another); long ones leave fewer sums to
    // join (262,144 positions in runs of 32: 58 MB of them beside 470 MB of rows).
    l.run = n <= kRankMost ? 16 : n <= 65536 ? 32 : n <= (1 << 17) ? 64 : kMostRun;
    l.runs = (n + l.run - 1) / l.run;
    l.pitch = static_cast<int>(round_up(hidden, 8));
    for (int i = 0; i < (n > kRankMost ? 2 : 1); ++i) {
        l.keys[i] = take(n * 4);
        l.order[i] = take(n * 4);
    }
    if (n > kRankMost) {
        const int64_t rounds = (n + kRound - 1) / kRound;
        l.tiles = static_cast<int>(rounds < kMostTiles ? rounds : kMostTiles);
        l.counts = take(static_cast<size_t>(l.tiles) * kBins * 4);
    }
    l.n_cross = take(4);
    l.cross = take(l.runs * 4);
    l.part = take(static_cast<size_t>(l.runs > 1 ? 2 * l.runs : 0) * l.pitch * 4);
    l.bytes = at;
    return l;
}

Zero zeros_of(void *p, size_t bytes) {
    const size_t n16 = bytes / 16;
    return {static_cast<uint4 *>(p), n16, static_cast<uint8_t *>(p) + n16 * 16, static_cast<int>(bytes % 16), 0};
}
// CTAs of `threads` that write zeros.
unsigned zero_ctas(const Zero &z, int threads) {
    const size_t each = static_cast<size_t>(kZeroWords) * threads;
    return static_cast<unsigned>((z.n16 + each - 1) / each) + (z.n16 == 0 && z.ntail ? 1u : 0u);
}

template <int DT, int VEC, typename O, bool ADD, bool TARGETS>
cudaError_t launch_sums(const Sums &s, const void *rows, O *out, int64_t runs, cudaStream_t stream) {
    int cols = 8;
    while (cols < kSumThreads && cols * VEC < s.hidden) cols *= 2;
    const int groups = kSumThreads / cols;
    const dim3 grid(static_cast<unsigned>((runs + groups - 1) / groups),
                    static_cast<unsigned>((s.hidden + cols * VEC - 1) / (cols * VEC)));
    const size_t smem = static_cast<size_t>((TARGETS ? 3 : 2) * groups) * s.run * 4;
    return launch_pdl(sum_runs_kernel<DT, VEC, O, ADD, TARGETS>, grid, dim3(kSumThreads), smem, stream, s,
                      static_cast<const typename Elem<DT>::T *>(rows), out, cols);
}
template <typename O, bool TARGETS>
cudaError_t launch_join(const Sums &s, O *out, int64_t runs, cudaStream_t stream) {
    DeviceInfo dev;
    const cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    const int col_blocks = (s.hidden + kJoinCols - 1) / kJoinCols;
    const int64_t most = (runs * col_blocks + kJoinWarps - 1) / kJoinWarps, cap = 4ll * dev.num_sms;
    return launch_pdl(join_runs_kernel<O, TARGETS>, dim3(static_cast<unsigned>(most < cap ? most : cap)), dim3(32 * kJoinWarps), 0,
                      stream, s, out, col_blocks, s.hidden % 4 == 0);
}

template <int DT, int VEC, typename O>
cudaError_t sum_runs(const EmbedGradArgs &a, const Sums &s, int64_t runs, cudaStream_t stream) {
    O *out = static_cast<O *>(a.dtable);
    return a.accumulate ? launch_sums<DT, VEC, O, true, false>(s, a.dout, out, runs, stream)
                        : launch_sums<DT, VEC, O, false, false>(s, a.dout, out, runs, stream);
}

template <typename O>
cudaError_t sums(const EmbedGradArgs &a, const Sums &s, int64_t runs, cudaStream_t stream) {
    // eight values at a time where every row of dout and of the table starts on the words they make
    const size_t es = a.dout_dtype == LHS_F32 ? 4 : 2;
    const bool wide8 = a.hidden % 8 == 0 && reinterpret_cast<uintptr_t>(a.dout) % 16 == 0 &&
                       static_cast<size_t>(a.dout_stride) * es % 16 == 0;
    cudaError_t e;
    if (a.dout_dtype == LHS_F32)
        e = wide8 ? sum_runs<LHS_F32, 8, O>(a, s, runs, stream) : sum_runs<LHS_F32, 1, O>(a, s, runs, stream);
    else if (a.dout_dtype == LHS_F16)
        e = wide8 ? sum_runs<LHS_F16, 8, O>(a, s, runs, stream) : sum_runs<LHS_F16, 1, O>(a, s, runs, stream);
    else
        e = wide8 ? sum_runs<LHS_BF16, 8, O>(a, s, runs, stream) : sum_runs<LHS_BF16, 1, O>(a, s, runs, stream);
    if (e != cudaSuccess || runs < 2) return e;
    return launch_join<O, false>(s, static_cast<O *>(a.dtable), runs, stream);
}

// Orders the ids, and writes zeros beside that; `s` gets the sorted keys and positions, and what sums
// of runs need besides.
cudaError_t order_ids(const int32_t *ids, int64_t n, int64_t vocab, int32_t ignore, const Layout &l, uint8_t *ws,
                      void *zeros, size_t zero_bytes, int32_t *err, Sums *s, cudaStream_t stream) {
    uint32_t *keys[2] = {reinterpret_cast<uint32_t *>(ws + l.keys[0]), reinterpret_cast<uint32_t *>(ws + l.keys[1])};
    int32_t *order[2] = {reinterpret_cast<int32_t *>(ws + l.order[0]), reinterpret_cast<int32_t *>(ws + l.order[1])};
    s->n_cross = reinterpret_cast<uint32_t *>(ws + l.n_cross);
    cudaError_t e = cudaSuccess;
    int last = 0;
    if (n <= kRankMost) {
        Zero z = zeros_of(zeros, zero_bytes);
        z.first = static_cast<int>((n + 31) / 32);
        e = launch_pdl(rank_ids_kernel, dim3(z.first + zero_ctas(z, kRankThreads)), dim3(kRankThreads),
                       round_up(n, 32) * 4, stream, ids, static_cast<int>(n), static_cast<uint32_t>(vocab), ignore, keys[0], order[0],
                       s->n_cross, z, err);
        if (e != cudaSuccess) return e;
    } else {
        int bits = 1;
        while ((vocab >> bits) != 0) ++bits;  // keys are 0 .. vocab
        const int passes = (bits + kDigitBits - 1) / kDigitBits;
        Pass p = {};
        p.counts = reinterpret_cast<uint32_t *>(ws + l.counts);
        p.n = n;
        p.tiles = l.tiles;
        p.per = round_up((n + l.tiles - 1) / l.tiles, kRound);
        p.vocab = static_cast<uint32_t>(vocab);
        p.ignore = ignore;
        p.n_cross = s->n_cross;
        p.err = err;
        // the moves take the zeros (20 us a pass for 262,144 ids, as 136 MB of zeros do; a count takes 5)
        auto share = [&](int i) {  // in whole words; the last takes the rest
            const size_t each = zero_bytes / 16 / passes * 16;
            Zero z = zeros_of(static_cast<uint8_t *>(zeros) + i * each, i + 1 < passes ? each : zero_bytes - i * each);
            z.first = l.tiles;
            return z;
        };
        for (int i = 0; i < passes; ++i) {
            p.shift = bits * i / passes;
            p.bits = bits * (i + 1) / passes - p.shift;
            p.ids = i == 0 ? ids : nullptr;
            p.keys_in = keys[(i & 1) ^ 1];
            p.order_in = order[(i & 1) ^ 1];
            p.keys_out = keys[i & 1];
            p.order_out = order[i & 1];
            e = launch_pdl(count_digits_kernel, dim3(l.tiles), dim3(kSortThreads), 0, stream, p);
            if (e != cudaSuccess) return e;
            const Zero z = share(i);
            e = launch_pdl(move_digits_kernel, dim3(l.tiles + zero_ctas(z, kSortThreads)), dim3(kSortThreads), 0, stream, p, z);
            if (e != cudaSuccess) return e;
            last = i & 1;
        }
    }
    s->keys = keys[last];
    s->order = order[last];
    s->n = n;
    s->run = l.run;
    s->pitch = l.pitch;
    s->vocab = vocab;
    s->part = reinterpret_cast<float *>(ws + l.part);
    s->cross = reinterpret_cast<int32_t *>(ws + l.cross);
    return e;
}

}  // namespace

cudaError_t launch_zero(void *p, size_t bytes, cudaStream_t stream) {
    const Zero z = zeros_of(p, bytes);
    return launch_pdl(zero_kernel, dim3(zero_ctas(z, 512)), dim3(512), 0, stream, z);
}

size_t embed_grad_workspace(int32_t hidden, int64_t n) { return layout_of(hidden, n).bytes; }

cudaError_t launch_embed_grad(const EmbedGradArgs &a, cudaStream_t stream) {
    const size_t es = a.dtable_dtype == LHS_F32 ? 4 : 2;
    const size_t table_bytes = a.accumulate ? 0 : static_cast<size_t>(a.vocab) * a.hidden * es;
    if (a.n == 0) return a.accumulate ? cudaSuccess : launch_zero(a.dtable, table_bytes, stream);
    const Layout l = layout_of(a.hidden, a.n);
    Sums s = {};
    const cudaError_t e = order_ids(a.ids, a.n, a.vocab, a.ignore, l, a.ws, a.dtable, table_bytes, a.err, &s, stream);
    if (e != cudaSuccess) return e;
    s.hidden = a.hidden;
    s.scale = a.scale;
    s.dout_stride = a.dout_stride;
    s.accumulate = a.accumulate;
    if (a.dtable_dtype == LHS_F32) return sums<float>(a, s, l.runs, stream);
    if (a.dtable_dtype == LHS_F16) return sums<__half>(a, s, l.runs, stream);
    return sums<__nv_bfloat16>(a, s, l.runs, stream);
}

cudaError_t launch_target_rows(const TargetRowsArgs &a, cudaStream_t stream) {
    const Layout l = layout_of(a.Hp, a.T);
    Sums s = {};
    cudaError_t e = order_ids(a.targets, a.T, a.V, a.ignore, l, a.ws, nullptr, 0, a.err, &s, stream);
    if (e != cudaSuccess) return e;
    s.hidden = a.Hp;
    s.scale = 1.0f;
    s.dout_stride = a.Hp;
    s.row_of = a.pos;
    s.weight = a.coef;
    s.slot_of = a.slot_of;
    s.out_pitch = a.pitch;
    s.by_id = a.V <= a.T;
    e = a.bf16 ? launch_sums<LHS_BF16, 8, float, false, true>(s, a.x, a.rows, l.runs, stream)
               : launch_sums<LHS_F16, 8, float, false, true>(s, a.x, a.rows, l.runs, stream);
    if (e != cudaSuccess || l.runs < 2) return e;
    return launch_join<float, true>(s, a.rows, l.runs, stream);
}

}  // namespace lhs
