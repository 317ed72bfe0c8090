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
//  * Sums.  A group of threads walks 32 sorted positions over the columns that
//    it holds.  A run of one id that lies within them is finished there.  One
//    that crosses their ends leaves an f32 sum for each 32, which a last kernel
//    joins in a fixed order, spread over threads: the hottest id of natural
//    text names a tenth of all positions.
//  * Rows that no id names are zeroed by further CTAs of the launches that order
//    the ids, which use little of the chip (8,192 ids: 402 MB of zeros beside a
//    few us of comparisons).
#include "train.cuh"

namespace lhs {
namespace {

constexpr int kRankMost = 8192;     // ids whose places are counted
constexpr int kRankThreads = 256;   // 32 ids to a CTA, its warps share the others
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9;
constexpr int kBins = 1 << kDigitBits;
constexpr int kSortSteps = 8;       // keys of a thread in a round
constexpr int kRound = kSortThreads * kSortSteps;
constexpr int kMostTiles = 128;     // each reads the counts of all
constexpr int kRun = 32;            // sorted positions that a group of threads sums
constexpr int kSumThreads = 128;
constexpr int kJoinCols = 64;       // threads along the columns, four columns each
constexpr int kJoinRows = 8;        // threads that share a column's sums

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Zeros that CTAs `first` and up of a launch write.
struct Zero {
    uint4 *p;
    size_t n16;       // 16-byte words
    uint8_t *tail;    // what is left of the last one
    int ntail;
    int first;
};
__device__ __forceinline__ void write_zeros(const Zero &z) {
    const size_t step = static_cast<size_t>(gridDim.x - z.first) * blockDim.x;
    for (size_t i = static_cast<size_t>(blockIdx.x - z.first) * blockDim.x + threadIdx.x; i < z.n16; i += step)
        __stcs(z.p + i, make_uint4(0u, 0u, 0u, 0u));
    if (static_cast<int>(blockIdx.x) == z.first && static_cast<int>(threadIdx.x) < z.ntail) z.tail[threadIdx.x] = 0;
}

__global__ void __launch_bounds__(256) zero_kernel(const Zero z) {
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
    extern __shared__ uint32_t all[];  // the keys, to a multiple of 32 with the largest value
    __shared__ int part[kRankThreads / 32][32];
    pdl_wait();
    pdl_trigger();
    if (static_cast<int>(blockIdx.x) >= z.first) return write_zeros(z);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kRankThreads / 32;
    const int padded = (n + 31) / 32 * 32;
    bool bad = false;
    for (int i = threadIdx.x; i < padded; i += kRankThreads) {
        const int32_t id = i < n ? ld_dep(ids + i) : ignore;
        const uint32_t k = key_of(id, vocab, ignore);
        if (k == vocab && id != ignore) bad = true;
        all[i] = i < n ? k : 0xFFFFFFFFu;
    }
    if (bad && blockIdx.x == 0) set_err(err, LHS_ERRBIT_BAD_TOKEN);
    if (blockIdx.x == 0 && threadIdx.x == 0) *n_cross = 0u;
    __syncthreads();
    const int i = blockIdx.x * 32 + lane;
    const uint32_t k = all[i < padded ? i : 0];
    int rank = 0;
    // words of four keys; those of other CTAs' positions lie wholly before or behind this one's
    for (int w = warp; w < padded / 4; w += warps) {
        const uint4 a = reinterpret_cast<const uint4 *>(all)[w];
        if (w < static_cast<int>(blockIdx.x) * 8) {
            rank += (a.x <= k) + (a.y <= k) + (a.z <= k) + (a.w <= k);
        } else if (w >= static_cast<int>(blockIdx.x) * 8 + 8) {
            rank += (a.x < k) + (a.y < k) + (a.z < k) + (a.w < k);
        } else {
            const int j = w * 4;
            rank += (a.x < k || (a.x == k && j < i)) + (a.y < k || (a.y == k && j + 1 < i)) +
                    (a.z < k || (a.z == k && j + 2 < i)) + (a.w < k || (a.w == k && j + 3 < i));
        }
    }
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

__global__ void __launch_bounds__(kSortThreads) count_digits_kernel(const Pass p, const Zero z) {
    __shared__ uint32_t bins[kBins];
    pdl_wait();
    pdl_trigger();
    if (static_cast<int>(blockIdx.x) >= z.first) return write_zeros(z);
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
// VEC consecutive values of a row, widened.
template <int DT, int VEC>
struct Pack;
template <int DT>
struct Pack<DT, 1> {
    typename Elem<DT>::T v;
    __device__ __forceinline__ void load(const typename Elem<DT>::T *p) { v = ld_dep(p); }
    __device__ __forceinline__ void add(float (&s)[1]) const { s[0] += Elem<DT>::widen(v); }
};
template <>
struct Pack<LHS_F32, 8> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = ld_dep(reinterpret_cast<const float4 *>(p));
        b = ld_dep(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void add(float (&s)[8]) const {
        s[0] += a.x, s[1] += a.y, s[2] += a.z, s[3] += a.w;
        s[4] += b.x, s[5] += b.y, s[6] += b.z, s[7] += b.w;
    }
};
template <int DT>
struct Pack<DT, 8> {
    uint4 w;
    __device__ __forceinline__ void load(const uint16_t *p) { w = ld_dep(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void add(float (&s)[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[2 * i] += Elem<DT>::widen(static_cast<uint16_t>(u[i]));
            s[2 * i + 1] += Elem<DT>::widen(static_cast<uint16_t>(u[i] >> 16));
        }
    }
};

// N sums scaled, added to what the gradient held if asked, and stored.
template <int N, typename O>
__device__ __forceinline__ void finish(O *o, const float (&s)[N], float scale, bool accumulate) {
    alignas(16) O v[N];
    if (N == 8) {
        uint4 *w = reinterpret_cast<uint4 *>(v);
        uint4 *g = reinterpret_cast<uint4 *>(o);
        if (accumulate) {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(v) / 16); ++i) w[i] = g[i];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) put_rn(&v[i], fmaf(s[i], scale, accumulate ? wide(v[i]) : 0.0f));
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(v) / 16); ++i) g[i] = w[i];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) put_rn(o + i, fmaf(s[i], scale, accumulate ? wide(o[i]) : 0.0f));
    }
}

struct Sums {
    const uint32_t *keys;
    const int32_t *order;
    int64_t n;
    int hidden, pitch;      // f32 sums of a run: rows of pitch, a multiple of 8
    uint32_t vocab;
    float scale;
    int64_t dout_stride;
    bool accumulate;
    float *part;            // [2 x runs x pitch]: of a run's first id where it came from before, of its
                            // last where it goes on
    uint32_t *n_cross;      // runs whose last id starts there and goes on
    int32_t *cross;
};

// A group of `cols` threads (a power of two) to a run; thread c of it holds
// columns VEC (c + cols blockIdx.y) and up.
template <int DT, int VEC, typename O>
__global__ void __launch_bounds__(kSumThreads)
    sum_runs_kernel(const Sums p, const typename Elem<DT>::T *dout, O *dtable, int cols) {
    constexpr int kAhead = 8;  // rows asked for at a time
    __shared__ uint32_t key[kSumThreads / 8][kRun];
    __shared__ int32_t pos[kSumThreads / 8][kRun];
    pdl_wait();
    const int group = threadIdx.x / cols, c = threadIdx.x % cols;
    const int64_t run = static_cast<int64_t>(blockIdx.x) * (kSumThreads / cols) + group;
    const int64_t i0 = run * kRun;
    const int len = i0 < p.n ? static_cast<int>(p.n - i0 < kRun ? p.n - i0 : kRun) : 0;
    for (int e = c; e < kRun; e += cols) {
        key[group][e] = e < len ? ld_dep(p.keys + i0 + e) : p.vocab;
        pos[group][e] = e < len ? ld_dep(p.order + i0 + e) : 0;
    }
    __syncthreads();
    if (len == 0 || key[group][0] == p.vocab) return;
    const uint32_t prev = i0 > 0 ? ld_dep(p.keys + i0 - 1) : p.vocab;
    const uint32_t next = i0 + kRun < p.n ? ld_dep(p.keys + i0 + kRun) : p.vocab;
    const int j = (c + cols * static_cast<int>(blockIdx.y)) * VEC;
    const bool in = j < p.hidden;
    float s[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) s[i] = 0.0f;
    uint32_t cur = key[group][0];
    bool head = cur == prev;
    auto keep = [&](int64_t row) {
        if (!in) return;
        float *o = p.part + row * p.pitch + j;
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = s[i];
    };
    for (int e0 = 0; e0 < kRun; e0 += kAhead) {
        Pack<DT, VEC> v[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
            if (in && key[group][e0 + e] != p.vocab) v[e].load(dout + pos[group][e0 + e] * p.dout_stride + j);
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            const uint32_t k = key[group][e0 + e];
            if (k != cur) {
                if (cur != p.vocab) {
                    if (head) keep(2 * run);
                    else if (in) finish<VEC>(dtable + static_cast<int64_t>(cur) * p.hidden + j, s, p.scale, p.accumulate);
                }
                head = false;
                cur = k;
#pragma unroll
                for (int i = 0; i < VEC; ++i) s[i] = 0.0f;
            }
            if (in && k != p.vocab) v[e].add(s);
        }
    }
    if (cur == p.vocab) return;
    if (cur == next) {
        keep(head ? 2 * run : 2 * run + 1);
        if (!head && c == 0 && blockIdx.y == 0) p.cross[atomicAdd(p.n_cross, 1u)] = static_cast<int32_t>(run);
    } else if (head) {
        keep(2 * run);
    } else if (in) {
        finish<VEC>(dtable + static_cast<int64_t>(cur) * p.hidden + j, s, p.scale, p.accumulate);
    }
}

// The ids that cross runs: an item is one of them and 4 kJoinCols columns.  The
// sums of its runs are dealt out to kJoinRows threads, whose results are joined in
// their order.
template <typename O>
__global__ void __launch_bounds__(kJoinCols *kJoinRows)
    join_runs_kernel(const Sums p, O *dtable, int col_blocks, bool vec) {
    constexpr int kThreads = kJoinCols * kJoinRows;
    __shared__ float4 part[kJoinRows][kJoinCols];
    __shared__ int ends[kThreads / 32];
    pdl_wait();
    const int c = threadIdx.x % kJoinCols, row = threadIdx.x / kJoinCols;
    const int64_t items = static_cast<int64_t>(ld_dep(p.n_cross)) * col_blocks;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t run = ld_dep(p.cross + item / col_blocks);
        const uint32_t id = ld_dep(p.keys + run * kRun + kRun - 1);
        // runs after the first that start with the id
        int64_t more = 0;
        for (;;) {
            const int64_t i = (run + 1 + more + threadIdx.x) * kRun;
            const bool on = i < p.n && ld_dep(p.keys + i) == id;
            const uint32_t m = __ballot_sync(0xFFFFFFFFu, on);
            if ((threadIdx.x & 31) == 0) ends[threadIdx.x / 32] = __popc(m);
            __syncthreads();
            int n = 0;
            for (int w = 0; w < kThreads / 32; ++w) n += ends[w];
            more += n;
            __syncthreads();
            if (n < kThreads) break;
        }
        const int j = (static_cast<int>(item % col_blocks) * kJoinCols + c) * 4;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (j < p.hidden) {
#pragma unroll 8
            for (int64_t r = row; r <= more; r += kJoinRows) {
                const float4 a = ld_dep(reinterpret_cast<const float4 *>(p.part + (2 * (run + r) + (r == 0 ? 1 : 0)) * p.pitch + j));
                s.x += a.x, s.y += a.y, s.z += a.z, s.w += a.w;
            }
        }
        part[row][c] = s;
        __syncthreads();
        if (row == 0 && j < p.hidden) {
            for (int r = 1; r < kJoinRows && r <= more; ++r) {
                const float4 a = part[r][c];
                s.x += a.x, s.y += a.y, s.z += a.z, s.w += a.w;
            }
            const float f[4] = {s.x, s.y, s.z, s.w};
            O *o = dtable + static_cast<int64_t>(id) * p.hidden + j;
            if (vec) {  // hidden % 4 == 0: four values are 8 or 16 aligned bytes
                alignas(16) O v[4];
                if (sizeof(O) == 4) {
                    if (p.accumulate) *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(o);
                } else if (p.accumulate) {
                    *reinterpret_cast<uint2 *>(v) = *reinterpret_cast<const uint2 *>(o);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) put_rn(&v[k], fmaf(f[k], p.scale, p.accumulate ? wide(v[k]) : 0.0f));
                if (sizeof(O) == 4) *reinterpret_cast<uint4 *>(o) = *reinterpret_cast<const uint4 *>(v);
                else *reinterpret_cast<uint2 *>(o) = *reinterpret_cast<const uint2 *>(v);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (j + k < p.hidden) put_rn(o + k, fmaf(f[k], p.scale, p.accumulate ? wide(o[k]) : 0.0f));
            }
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
    int pitch, tiles;
};
Layout layout_of(int32_t hidden, int64_t n) {
    Layout l = {};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += align256(bytes);
        return o;
    };
    l.runs = (n + kRun - 1) / kRun;
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
// CTAs of `threads` that write zeros: enough to fill the chip, no more than there is to write.
unsigned zero_ctas(const Zero &z, int threads, const DeviceInfo &dev) {
    const size_t want = (z.n16 + threads - 1) / threads, most = static_cast<size_t>(dev.num_sms) * 2048 / threads;
    return static_cast<unsigned>(want < most ? want : most) + (want == 0 && z.ntail ? 1u : 0u);
}

template <int DT, int VEC, typename O>
cudaError_t sum_runs(const EmbedGradArgs &a, const Sums &s, int64_t runs, cudaStream_t stream) {
    int cols = 8;
    while (cols < kSumThreads && cols * VEC < a.hidden) cols *= 2;
    const int groups = kSumThreads / cols;
    const dim3 grid(static_cast<unsigned>((runs + groups - 1) / groups),
                    static_cast<unsigned>((a.hidden + cols * VEC - 1) / (cols * VEC)));
    return launch_pdl(sum_runs_kernel<DT, VEC, O>, grid, dim3(kSumThreads), 0, stream, s,
                      static_cast<const typename Elem<DT>::T *>(a.dout), static_cast<O *>(a.dtable), cols);
}

template <typename O>
cudaError_t sums(const EmbedGradArgs &a, const Sums &s, int64_t runs, const DeviceInfo &dev, cudaStream_t stream) {
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
    const int col_blocks = (a.hidden + 4 * kJoinCols - 1) / (4 * kJoinCols);
    const int64_t most = runs * col_blocks, cap = 4ll * dev.num_sms;
    return launch_pdl(join_runs_kernel<O>, dim3(static_cast<unsigned>(most < cap ? most : cap)),
                      dim3(kJoinCols * kJoinRows), 0, stream, s, static_cast<O *>(a.dtable), col_blocks, a.hidden % 4 == 0);
}

}  // namespace

cudaError_t launch_zero(void *p, size_t bytes, cudaStream_t stream) {
    DeviceInfo dev;
    const cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    const Zero z = zeros_of(p, bytes);
    return launch_pdl(zero_kernel, dim3(zero_ctas(z, 256, dev)), dim3(256), 0, stream, z);
}

size_t embed_grad_workspace(int32_t hidden, int64_t n) { return layout_of(hidden, n).bytes; }

cudaError_t launch_embed_grad(const EmbedGradArgs &a, cudaStream_t stream) {
    const size_t es = a.dtable_dtype == LHS_F32 ? 4 : 2;
    const size_t table_bytes = a.accumulate ? 0 : static_cast<size_t>(a.vocab) * a.hidden * es;
    if (a.n == 0) return a.accumulate ? cudaSuccess : launch_zero(a.dtable, table_bytes, stream);
    DeviceInfo dev;
    cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    const Layout l = layout_of(a.hidden, a.n);
    uint32_t *keys[2] = {reinterpret_cast<uint32_t *>(a.ws + l.keys[0]), reinterpret_cast<uint32_t *>(a.ws + l.keys[1])};
    int32_t *order[2] = {reinterpret_cast<int32_t *>(a.ws + l.order[0]), reinterpret_cast<int32_t *>(a.ws + l.order[1])};
    Sums s = {};
    s.n_cross = reinterpret_cast<uint32_t *>(a.ws + l.n_cross);
    const uint32_t vocab = static_cast<uint32_t>(a.vocab);
    int last = 0;
    if (a.n <= kRankMost) {
        Zero z = zeros_of(a.dtable, table_bytes);
        z.first = static_cast<int>((a.n + 31) / 32);
        const unsigned grid = z.first + zero_ctas(z, kRankThreads, dev);
        e = launch_pdl(rank_ids_kernel, dim3(grid), dim3(kRankThreads), round_up(a.n, 32) * 4, stream, a.ids,
                       static_cast<int>(a.n), vocab, a.ignore, keys[0], order[0], s.n_cross, z, a.err);
        if (e != cudaSuccess) return e;
    } else {
        int bits = 1;
        while ((a.vocab >> bits) != 0) ++bits;  // keys are 0 .. vocab
        const int passes = (bits + kDigitBits - 1) / kDigitBits;
        Pass p = {};
        p.counts = reinterpret_cast<uint32_t *>(a.ws + l.counts);
        p.n = a.n;
        p.tiles = l.tiles;
        p.per = round_up((a.n + l.tiles - 1) / l.tiles, kRound);
        p.vocab = vocab;
        p.ignore = a.ignore;
        p.n_cross = s.n_cross;
        p.err = a.err;
        const int launches = 2 * passes;
        auto share = [&](int i) {  // of the zeros, in whole words; the last takes the rest
            const size_t each = table_bytes / 16 / launches * 16;
            Zero z = zeros_of(static_cast<uint8_t *>(a.dtable) + i * each, i + 1 < launches ? each : table_bytes - i * each);
            z.first = l.tiles;
            return z;
        };
        for (int i = 0; i < passes; ++i) {
            p.shift = bits * i / passes;
            p.bits = bits * (i + 1) / passes - p.shift;
            p.ids = i == 0 ? a.ids : nullptr;
            p.keys_in = keys[(i & 1) ^ 1];
            p.order_in = order[(i & 1) ^ 1];
            p.keys_out = keys[i & 1];
            p.order_out = order[i & 1];
            Zero z = share(2 * i);
            e = launch_pdl(count_digits_kernel, dim3(l.tiles + zero_ctas(z, kSortThreads, dev)), dim3(kSortThreads), 0,
                           stream, p, z);
            if (e != cudaSuccess) return e;
            z = share(2 * i + 1);
            e = launch_pdl(move_digits_kernel, dim3(l.tiles + zero_ctas(z, kSortThreads, dev)), dim3(kSortThreads), 0,
                           stream, p, z);
            if (e != cudaSuccess) return e;
            last = i & 1;
        }
    }
    s.keys = keys[last];
    s.order = order[last];
    s.n = a.n;
    s.hidden = a.hidden;
    s.pitch = l.pitch;
    s.vocab = vocab;
    s.scale = a.scale;
    s.dout_stride = a.dout_stride;
    s.accumulate = a.accumulate;
    s.part = reinterpret_cast<float *>(a.ws + l.part);
    s.cross = reinterpret_cast<int32_t *>(a.ws + l.cross);
    if (a.dtable_dtype == LHS_F32) return sums<float>(a, s, l.runs, dev, stream);
    if (a.dtable_dtype == LHS_F16) return sums<__half>(a, s, l.runs, dev, stream);
    return sums<__nv_bfloat16>(a, s, l.runs, dev, stream);
}

}  // namespace lhs
