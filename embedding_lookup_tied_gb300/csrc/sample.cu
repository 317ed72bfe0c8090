// sample.cu — one token per row of logits, drawn with temperature, top-k,
// top-p and min-p from a given random number (ADR-0008 "Remote Embeddings and
// lm_head Service", POST /v1/logits, "raw logits mode for beam search /
// sampling").
//
// Mathematics.  All three filters keep a head of the row in the order (logit
// descending, id ascending), so together they keep the entries whose 64-bit
// (order key, inverted id) is at least a threshold; top-k finds it by counts,
// top-p by sums of weights.  The draw inverts the running sum of the kept
// weights in id order.  Weights are 2^S exp((logit - max) / T) as 64-bit
// integers (see Weight), so every sum is exact, whatever the order in which
// warps, CTAs and atomics form it, and two passes over a row agree to the last
// bit.  A weight is cut to whole units, of which the largest has 2^(S-1) at least, so
// a sum is up to its number of entries in units below its value (2^-43 of the
// largest weight an entry for a vocabulary of 2^18).
//
// A cluster of CTAs owns a row and holds it in its shared memory: HBM is read
// once (bulk copies), and every later pass is a lane's own 16-byte words from
// shared memory.  Rows too long for 16 CTAs (more than 52 words a thread, 851,968
// f32 logits) are read from L2 or HBM in every pass.
//  * top-k: at least k entries lie in or above the bin that holds the k-th
//    largest of the threads' maxima, and few more do, so that bound gathers a
//    short list; one CTA sorts it and does the rest (k, p, min-p, the draw).
//  * top-p alone: one pass counts the entries by bins of 1/16 octave; the
//    counts bracket the bin in which the weights reach p of their sum, a pass
//    sums the bracket's bins, and what lies above and below it, exactly, and
//    the entries of the one bin left (or of 1/256 of it) are sorted.
//  * Where a list does not fit (equal logits by the thousand), the threshold is
//    found digit by digit (8 bits) from histograms over the order key.
//  * The draw: each warp's sum over its piece of the row, the pieces in id
//    order; the CTA whose warp's piece holds the answer walks it.
//
// What bounds it: latency.  A row of 1 MB is 0.15 us of HBM time, but 8 to 14
// exchanges across the cluster of about 0.7 us each, and passes of 1 to 7 us
// over 64 logits a lane (ncu, 256 rows of 262,144 f32 with mixed filters: 29% of
// issue slots, 3.2 of 4 warps a scheduler active, a third of the stalls at
// barriers).  Measured: 1 x 151,936 f32 with all filters 10.6 us; 8 x 262,144 f32
// with top-p 53 us; 256 x 262,144 f32 393 us mixed, 171 us min-p, 249 us with the
// temperature alone, 279 us top-k, 895 us top-p; a row that is not resident, 1 x
// 1,200,000 f32, 61 us with the temperature alone, 44 us top-k, 214 us top-p.  Tried and slower: CTAs of 512
// threads (426 -> 453 us mixed), two words side by side (441 -> 455 us), clusters
// of at most 8 (441 -> 499 us).
#include <cooperative_groups.h>

#include <mutex>

#include "decode.cuh"

namespace cg = cooperative_groups;

namespace lhs {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kList = 512;                    // entries one CTA ranks
constexpr int kDigits = 256;                  // bins of a digit of the order key
constexpr int kBins = 512;                    // of 1/16 octave of weight; the last takes all that is below
constexpr float kBinsPerOctave = 16.0f;
constexpr int kParts = 256;                   // of a bin that holds too many entries
constexpr int kMaxSmem = 224 * 1024;
constexpr uint32_t kKeyInf = 0xFF800000u;     // order key of +inf; these lie above:
constexpr uint32_t kKeyNan = 0xFFFFFFFEu;     // a NaN
constexpr uint32_t kKeyLate = 0xFFFFFFFFu;    // a piece of the row that has not arrived in time
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;  // order key of -inf

// round(2^61 * 2^(j/16))
__constant__ const uint64_t kPow16[16] = {
    0x2000000000000000ull, 0x216AB0D9F3121EC5ull, 0x22E57078FAA2F5BAull, 0x2470F4DCEAC470CEull,
    0x260DFC14636E2A5Cull, 0x27BD4C982468446Bull, 0x297FB5AA6C544E3Bull, 0x2B560FBA90A852B2ull,
    0x2D413CCCFE779921ull, 0x2F4228E7D6030DB0ull, 0x3159CA845541B6B7ull, 0x3389230547E12039ull,
    0x35D13F32B5A75ABDull, 0x383337BB0AA53844ull, 0x3AB031B9F7490E4Cull, 0x3D495F454921B30Bull};

// A logit's weight exp(l / T) over its row's scale, as an integer: 2^(S - G) *
// 2^(l c), c = log2(e) / T, G the integer next above c times the largest logit.
//
// c is two floats, l c = p + z with p = RN(l c_hi) and z the rest.  With K the
// nearest integer to 16 p, x = l c - K/16 is small (|x| <= 1/32 and a little),
// p - K/16 is exact, and
//   2^(l c) = 2^(K div 16) * 2^((K mod 16)/16) * 2^x,
// the middle factor from a table in 62 bits and 2^x = 1 + x ln2 + x^2 q(x)
// from its Taylor series: x ln2 in two floats, the rest (below 2^-12) in one.
// The factor's distance from 1 is below 2^-5.5 and is held as a 32-bit
// integer in units of 2^-36.  Together about 2^-36 of the weight, unbiased; then
// it is cut down to whole units, which is the larger error for weights below 2^-7
// of the largest (up to 2^-20 of a weight of 2^-23, S = 44).  Rounding would add
// a 64-bit addition and a shift to each weight, for sums that are already
// finer than u, a binary32 number (262,144 logits of N(0, 5) at temperature 0.8:
// running shares off by up to 2^-28).
// Where c times the largest logit passes 2^10 the rounding of l c_lo would
// show; there logits are first taken relative to the largest, and those that
// weigh anything are so near to it that the difference is exact.
// (No branch, so that the weights of a word's logits are worked out side by
// side: 33 issue slots a weight with 16 warps on an SM.)
struct Weight {
    float ref, low;    // what logits are relative to; below `low` they weigh 0
    float c_hi, c_lo;
    int shift;         // 61 - S + G
    const uint64_t *pow16;  // kPow16 in shared memory: 16 pairs of words, one to a bank

    __device__ __forceinline__ void init(float max, float c_hi_, float c_lo_, int S, const uint64_t *table) {
        c_hi = c_hi_;
        c_lo = c_lo_;
        ref = fabsf(max * c_hi) < 1024.0f ? 0.0f : max;
        low = max - static_cast<float>(S) / c_hi;
        const float top = (max - ref) * c_hi;
        shift = 61 - S + (__float2int_rn(top * 16.0f) >> 4) + 1;
        pow16 = table;
    }
    // 2^cut times the weight, before it is cut to whole units.
    __device__ __forceinline__ uint64_t whole(float logit, int &cut) const {
        const float l = __fsub_rn(logit, ref);
        const float p = __fmul_rn(l, c_hi);
        const float z = __fmaf_rn(l, c_lo, __fmaf_rn(l, c_hi, -p));
        const float magic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer
        const float y = __fmaf_rn(p, 16.0f, magic);
        const int K = static_cast<int>(__float_as_uint(y) - 0x4B400000u);
        const float r = __fmaf_rn(__fsub_rn(y, magic), -0.0625f, p);  // exact
        const float x = __fadd_rn(r, z), xl = __fadd_rn(__fsub_rn(r, x), z);
        constexpr float kLn2Hi = 0.6931471824645996f * 0x1p36f, kLn2Lo = -1.9046542e-9f * 0x1p36f;
        const float a = __fmul_rn(x, kLn2Hi);
        const float al = __fmaf_rn(x, kLn2Hi, -a) + __fmaf_rn(x, kLn2Lo, xl * kLn2Hi);
        float q = __fmaf_rn(x, 0.0013333558f * 0x1p36f, 0.009618129f * 0x1p36f);
        q = __fmaf_rn(x, q, 0.05550411f * 0x1p36f);
        q = __fmaf_rn(x, q, 0.24022651f * 0x1p36f);
        const int delta = __float2int_rn(a) + __float2int_rn(__fmaf_rn(x * x, q, al));  // (2^x - 1) 2^36
        const uint64_t f = pow16[K & 15];
        const uint64_t w =
            f + static_cast<uint64_t>((static_cast<int64_t>(static_cast<int>(f >> 32)) * delta) >> 4);
        // (below `low`, also at -inf, the rest may be anything, but w stays below 2^63)
        cut = logit < low ? 63 : min(shift - (K >> 4), 63);
        return w;
    }
    __device__ __forceinline__ uint64_t operator()(float logit) const {
        int cut;
        const uint64_t w = whole(logit, cut);
        return w >> cut;
    }
};

// What a row's parameters come to, worked out by one thread of each CTA while
// the row is on its way.  No 64-bit floating point: its unit here is slow.
struct RowScale {
    float c_hi, c_lo;   // log2(e) / T
    float span;         // differences from the largest logit beyond it are below min-p for certain
    uint64_t U, P, M;   // u, top-p and min-p in units of 2^-64
};

struct alignas(16) Shared {
    union {
        struct {
            uint64_t list[kList];   // entries; the digit histograms where no list fits
            uint64_t sums[kBins];   // a histogram's sums over the cluster
        };
        uint32_t copies[kBins][4];  // counts in the making: a lane's copy is lane mod 4
        uint32_t limbs[kBins][4];   // weights in the making: 15 bits to a limb, three used
    };
    uint64_t mass[kBins];
    uint32_t count[kBins];
    uint64_t slot[2][kMaxCluster];  // one value from each CTA of the cluster, two exchanges
    uint64_t warp_sum[kWarps];
    uint64_t above, in;
    uint64_t pow16[16];
    uint64_t arrived[kWarps];       // each warp's piece of the row has
    RowScale scale;
    int32_t bin;
    int32_t found;
    int32_t gathered;
};
static_assert(kDigits <= kList, "the digit histograms take the list's place");
static_assert(sizeof(Shared) % 16 == 0, "the row's words follow it");

__device__ __forceinline__ uint64_t warp_add(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t up = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += up;
    }
    return v;
}

// Sum over the CTA, leaving the warps' sums in warp_sum until the next use.
__device__ __forceinline__ uint64_t cta_sum(Shared &sm, uint64_t v) {
    v = warp_add(v);
    if ((threadIdx.x & 31) == 0) sm.warp_sum[threadIdx.x >> 5] = v;
    __syncthreads();
    uint64_t s = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s += sm.warp_sum[i];
    return s;
}
// Exclusive scan over the CTA's threads, and the sum of all; the caller syncs
// before the next use.
__device__ __forceinline__ uint64_t cta_scan(Shared &sm, uint64_t v, uint64_t &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t incl = warp_scan(v, lane);
    if (lane == 31) sm.warp_sum[warp] = incl;
    __syncthreads();
    uint64_t before = incl - v;
    all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const uint64_t x = sm.warp_sum[w];
        if (w < warp) before += x;
        all += x;
    }
    return before;
}

// The n entries of the list in descending order.  An entry's place is the number
// of larger ones: every pair is compared, two keys to a load (no rounds of a
// sort to wait for, and short lists are the rule).  CTA-collective.
__device__ __forceinline__ void sort_list(Shared &sm, int n) {
    const int tid = threadIdx.x;
    constexpr int E = kList / kThreads;
    if (tid == 0 && n < kList) sm.list[n] = 0;  // the last pair's other half
    __syncthreads();
    uint64_t key[E];
    int place[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        key[e] = tid + e * kThreads < n ? sm.list[tid + e * kThreads] : ~0ull;
        place[e] = 0;
    }
    if ((tid & ~31) < n) {  // else none of the warp's
        const ulonglong2 *pairs = reinterpret_cast<const ulonglong2 *>(sm.list);
        if (n <= kThreads) {
#pragma unroll 4
            for (int j = 0; j < (n + 1) / 2; ++j) {
                const ulonglong2 k = pairs[j];
                place[0] += (k.x > key[0] ? 1 : 0) + (k.y > key[0] ? 1 : 0);
            }
        } else {
#pragma unroll 4
            for (int j = 0; j < (n + 1) / 2; ++j) {
                const ulonglong2 k = pairs[j];
#pragma unroll
                for (int e = 0; e < E; ++e) place[e] += (k.x > key[e] ? 1 : 0) + (k.y > key[e] ? 1 : 0);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (tid + e * kThreads < n) sm.list[place[e]] = key[e];
    __syncthreads();
}

// What stays: entries with a key of at least `edge`.
struct Edge {
    float value;  // logits above it stay, those equal to it up to id `last`
    int last;
    __device__ __forceinline__ bool stays(float l, int id) const { return l > value || (l == value && id <= last); }
    __device__ __forceinline__ void set(uint64_t key) {
        value = key_value(key);
        last = key_id(key);
    }
};

// Bins from the top of a row down; a larger logit never lies in a later bin.
struct Bins {
    float largest, per_bin;
    __device__ __forceinline__ float place(float l) const { return fminf((largest - l) * per_bin, kBins - 1.0f); }
    static __device__ __forceinline__ int at(float place) {  // truncated by the addition
        return static_cast<int>(__float_as_uint(__fadd_rz(place, 8388608.0f)) - 0x4B000000u);
    }
};

// The weights of a word's logits that stay (EDGED) and are at least min-p's
// (FLOORED); false where all are 0 for certain.
template <bool EDGED, bool FLOORED, int VE>
struct Weigh {
    const Weight &weight;
    const Edge &edge;
    float largest, span;
    uint64_t floor_w;
    __device__ __forceinline__ bool operator()(const float (&x)[VE], int id, uint64_t (&w)[VE]) const {
        if (EDGED || FLOORED) {
            float most = x[0];
#pragma unroll
            for (int e = 1; e < VE; ++e) most = fmaxf(most, x[e]);
            if ((EDGED && most < edge.value) || (FLOORED && largest - most > span)) return false;
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            w[e] = weight(x[e]);
            if (EDGED && !edge.stays(x[e], id + e)) w[e] = 0;
            if (FLOORED && w[e] < floor_w) w[e] = 0;
        }
        return true;
    }
};
struct One {
    __device__ __forceinline__ uint64_t operator()(float) const { return 1; }
};

// One row, as one CTA of its cluster sees it.  The row's 16-byte words (as
// addresses fall, so the first and last may be partly another's: those elements
// are not read and count as -inf) are dealt out to warps in contiguous pieces.
template <int DT, bool RESIDENT>
struct RowView {
    using E = Elem<DT>;
    using T = typename E::T;
    static constexpr int VE = 16 / static_cast<int>(sizeof(T));
    Shared &sm;
    cg::cluster_group cl;
    int rank, ranks;
    uint4 *hold;      // this lane's words in shared memory, 32 apart
    int steps;        // words per lane
    int word0;        // this lane's first word; the next are 32 further on
    int vocab;
    const uint4 *base;  // the word that holds the row's first element
    int skip;           // elements of that word before it
    int flip;           // which exchange slots come next

    // Word w of the row, -inf where its elements are not the row's.
    __device__ __forceinline__ uint4 fetch(int w) const {
        const int64_t first = static_cast<int64_t>(w) * VE - skip;  // id of the word's first element
        if (first >= vocab || first + VE <= 0) return outside();
        return first < 0 || first + VE > vocab ? part(w) : ld_dep(base + w);
    }
    // A word that is partly the row's: its elements one by one, nothing else is read.
    __device__ __forceinline__ uint4 part(int w) const {
        const int64_t at = static_cast<int64_t>(w) * VE;
        const T *x = reinterpret_cast<const T *>(base) + at;
        uint32_t r[4] = {outside().x, outside().x, outside().x, outside().x};
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            if (at + e < skip || at + e - skip >= vocab) continue;
            if constexpr (VE == 4) {
                r[e] = __float_as_uint(ld_dep(x + e));
            } else {
                const uint32_t v = ld_dep(x + e);
                r[e >> 1] = e & 1 ? (r[e >> 1] & 0xFFFFu) | v << 16 : (r[e >> 1] & 0xFFFF0000u) | v;
            }
        }
        return make_uint4(r[0], r[1], r[2], r[3]);
    }
    // Whether the row starts (ends) inside this warp's first (last) word, of n.
    __device__ __forceinline__ bool starts_inside(int w0) const { return w0 == 0 && skip > 0; }
    __device__ __forceinline__ bool ends_inside(int w0, int n) const {
        return n > 0 && static_cast<int64_t>(w0 + n) * VE - skip > vocab;
    }
    static __device__ __forceinline__ uint4 outside() {  // -inf
        const uint32_t w = DT == LHS_F32 ? 0xFF800000u : DT == LHS_F16 ? 0xFC00FC00u : 0xFF80FF80u;
        return make_uint4(w, w, w, w);
    }
    static __device__ __forceinline__ void widen(const uint4 &u, float (&v)[VE]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        if (DT == LHS_F32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i) v[i] = E::widen(static_cast<T>(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu));
        }
    }
    // f(values, id of the first) for each of this lane's words, in id order.
    template <typename F>
    __device__ __forceinline__ void each(const F &f) const {
#pragma unroll 1
        for (int s = 0; s < steps; ++s) {
            float v[VE];
            widen(RESIDENT ? hold[s * 32] : fetch(word0 + s * 32), v);
            f(v, (word0 + s * 32) * VE - skip);
        }
    }
    // Starts the copy of this warp's piece of the row (the words that are wholly the row's).
    __device__ __forceinline__ void start() const {
        if (!RESIDENT || (threadIdx.x & 31)) return;
        const int n = piece();
        uint64_t *bar = &sm.arrived[threadIdx.x >> 5];
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the last row's reads
        const int from = starts_inside(word0) ? 1 : 0, whole = n - from - (ends_inside(word0, n) ? 1 : 0);
        mbar_arrive_expect_tx(bar, whole > 0 ? whole * 16 : 0);
        if (whole > 0) bulk_load(hold + from, base + word0 + from, whole * 16, bar);
    }
    // What the copy leaves out, while it is on its way: the row's ends, and -inf for
    // words of the piece beyond them.
    __device__ __forceinline__ void ends() const {
        if (!RESIDENT) return;
        const int lane = threadIdx.x & 31, n = piece(), w0 = word0 - lane;
        // an element to a lane: the first VE have the piece's first word, the next its last
        const bool first = lane < VE, cut = first ? starts_inside(w0) : ends_inside(w0, n);
        if (n > 0 && lane < 2 * VE && cut) {
            const int w = first ? 0 : n - 1, e = lane % VE;
            const int64_t at = static_cast<int64_t>(w0 + w) * VE + e;
            T x;
            if constexpr (DT == LHS_F32) x = -INFINITY;
            else x = static_cast<T>(outside().x);
            if (at >= skip && at - skip < vocab) x = ld_dep(reinterpret_cast<const T *>(base) + at);
            reinterpret_cast<T *>(hold - lane + w)[e] = x;
        }
        // of this lane's words, lane, lane + 32, ..
        for (int w = n + ((lane - n) & 31); w < steps * 32; w += 32) hold[w - lane] = outside();
        __syncwarp();
    }
    // Words of the warp's piece that hold elements of the row.
    __device__ __forceinline__ int piece() const {
        const int64_t words = (static_cast<int64_t>(skip) + vocab + VE - 1) / VE;
        const int64_t n = words - (word0 - static_cast<int>(threadIdx.x & 31));
        return static_cast<int>(n < 0 ? 0 : n < steps * 32 ? n : steps * 32);
    }
    // The row's first reading, once its piece has arrived: this lane's largest logit as
    // an order key (kKeyNan where one is NaN, kKeyLate where the piece has not arrived).
    __device__ __forceinline__ uint32_t read(uint32_t parity, int32_t *err) {
        float top = -INFINITY;
        uint32_t magnitude = 0;  // above the bits of inf: a NaN
        if (RESIDENT) {
            if (!mbar_wait(&sm.arrived[threadIdx.x >> 5], parity, kWaitTimeoutNs)) {
                set_err(err, LHS_ERRBIT_TIMEOUT);
                return kKeyLate;
            }
        }
#pragma unroll 4
        for (int s = 0; s < steps; ++s) {
            float v[VE];
            widen(RESIDENT ? hold[s * 32] : fetch(word0 + s * 32), v);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                top = fmaxf(top, v[e]);
                magnitude = max(magnitude, __float_as_uint(v[e]) & 0x7FFFFFFFu);
            }
        }
        return magnitude > 0x7F800000u ? kKeyNan : order_key32(top);
    }

    // Every CTA's v, in this CTA's shared memory.
    __device__ __forceinline__ const uint64_t *exchange(uint64_t v) {
        uint64_t *slots = sm.slot[flip];
        flip ^= 1;
        if (static_cast<int>(threadIdx.x) < ranks) cl.map_shared_rank(slots, threadIdx.x)[rank] = v;
        cl.sync();
        return slots;
    }
    // A histogram's (BINS of count or mass) sums over the cluster, into sums:
    // each CTA adds up its share of the bins, one source to a lane, and
    // hands the sums to all.
    template <int BINS, typename H>
    __device__ __forceinline__ void add_up(H *hist) {
        cl.sync();
#pragma unroll
        for (int i0 = 0; i0 < BINS; i0 += kThreads) {
            const int i = i0 + threadIdx.x, from = i & (ranks - 1);  // ranks: a power of two
            if (i >= BINS) break;                                    // whole warps
            const int bin = (i & ~(ranks - 1)) / ranks + rank * (BINS / ranks);
            uint64_t x = cl.map_shared_rank(hist, from)[bin];
            for (int o = 1; o < ranks; o <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
            cl.map_shared_rank(sm.sums, from)[bin] = x;
        }
        cl.sync();
    }
    // The bin in which the sums up to it reach need = need_of(all of them) (>= 1):
    // its number, and in sm.above / sm.in the sums before and of it.  BINS where
    // they do not.
    template <int BINS, typename H, typename F>
    __device__ __forceinline__ int crossing(H *hist, uint64_t &need, const F &need_of) {
        if (threadIdx.x == 0) sm.bin = BINS;
        add_up<BINS>(hist);
        constexpr int B = (BINS + kThreads - 1) / kThreads;
        uint64_t h[B], mine = 0;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int bin = threadIdx.x * B + b;
            h[b] = bin < BINS ? sm.sums[bin] : 0ull;
            mine += h[b];
        }
        uint64_t all, above = cta_scan(sm, mine, all);
        need = need_of(all);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (above < need && above + h[b] >= need) {
                sm.bin = static_cast<int>(threadIdx.x) * B + b;
                sm.above = above;
                sm.in = h[b];
            }
            above += h[b];
        }
        __syncthreads();
        return sm.bin;
    }

    template <int BINS, typename H>
    __device__ __forceinline__ int crossing(H *hist, uint64_t need) {
        return crossing<BINS>(hist, need, [&](uint64_t) { return need; });
    }

    // Entries that `take` takes, as keys: into this CTA's list, its number (of
    // which kList at most are held) into sm.gathered; their number over the
    // cluster.  take(values, id): a bit for each of a word's logits.
    template <typename F>
    __device__ __forceinline__ int64_t gather(const F &take) {
        if (threadIdx.x == 0) sm.gathered = 0;
        __syncthreads();
        each([&](const float (&v)[VE], int id) {
            uint32_t mask = take(v, id);
            if (mask == 0) return;
            const int n = __popc(mask);
            int at = atomicAdd(&sm.gathered, n);
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if ((mask >> e) & 1u) {
                    if (at < kList) sm.list[at] = topk_key(v[e], id + e);
                    ++at;
                }
        });
        __syncthreads();
        const uint64_t *all = exchange(static_cast<uint64_t>(sm.gathered));
        int64_t n = 0;
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i)
            if (i < ranks) n += static_cast<int64_t>(all[i]);
        return n;
    }
    // CTA 0: the other CTAs' entries (gathered, kList in all at most) behind its own.
    __device__ __forceinline__ void pull(const uint64_t *counts) {
        // a warp takes every kWarps-th CTA's list
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        int at = static_cast<int>(counts[0]);
        for (int r = 1; r < ranks; ++r) {
            const int n = static_cast<int>(counts[r]);
            if (r % kWarps == warp) {
                const uint64_t *src = cl.map_shared_rank(sm.list, r);
                for (int i = lane; i < n; i += 32) sm.list[at + i] = src[i];
            }
            at += n;
        }
        __syncthreads();
    }
    __device__ __forceinline__ const uint64_t *last_exchange() const { return sm.slot[flip ^ 1]; }

    // The key at which the sums of value over the entries that `take` takes, in
    // descending order of keys, reach need (>= 1, at most their sum).
    template <typename F, typename G>
    __device__ __forceinline__ uint64_t cut(const F &take, const G &value, uint64_t need) {
        const int64_t n = gather(take);
        if (n <= kList) {
            uint64_t key = 0;
            if (rank == 0) {
                pull(last_exchange());
                const int m = static_cast<int>(n);
                sort_list(sm, m);
                constexpr int P = kList / kThreads;
                uint64_t w[P], mine = 0;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const int at = threadIdx.x * P + i;
                    w[i] = at < m ? value(key_value(sm.list[at])) : 0ull;
                    mine += w[i];
                }
                uint64_t all, above = cta_scan(sm, mine, all);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    if (above < need && above + w[i] >= need) sm.above = sm.list[threadIdx.x * P + i];
                    above += w[i];
                }
                __syncthreads();
                key = sm.above;
            }
            return exchange(key)[0];
        }
        __syncthreads();
        // digit by digit, then the id among equal logits
        static_assert(kDigits <= kThreads, "one digit to a thread");
        uint32_t prefix = 0, mask = 0;
        uint64_t in = 0;
        for (int sh = 24; sh >= 0; sh -= 8) {
            if (threadIdx.x < kDigits) sm.list[threadIdx.x] = 0;
            __syncthreads();
            each([&](const float (&v)[VE], int id) {
                const uint32_t taken = take(v, id);
                if (taken == 0) return;
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const uint32_t k = order_key32(v[e]);
                    if (((taken >> e) & 1u) && (k & mask) == prefix)
                        atomicAdd(reinterpret_cast<unsigned long long *>(&sm.list[(k >> sh) & 0xFFu]), value(v[e]));
                }
            });
            // bins from the top, one to a thread
            add_up<kDigits>(sm.list);
            const uint64_t h = threadIdx.x < kDigits ? sm.sums[kDigits - 1 - threadIdx.x] : 0ull;
            uint64_t all, above = cta_scan(sm, h, all);
            if (above < need && above + h >= need) {
                sm.bin = kDigits - 1 - static_cast<int>(threadIdx.x);
                sm.above = above;
                sm.in = h;
            }
            __syncthreads();
            prefix |= static_cast<uint32_t>(sm.bin) << sh;
            mask |= 0xFFu << sh;
            need -= sm.above;
            in = sm.in;
            __syncthreads();
        }
        const float edge = key_value(static_cast<uint64_t>(prefix) << 32);
        const uint64_t one = value(edge), m = (need + one - 1) / one;  // of in / one equal logits
        int last = 0x7FFFFFFF;
        if (m < in / one) {
            locate(
                [&](const float (&v)[VE], int id, uint64_t (&w)[VE]) {
                    const uint32_t taken = take(v, id);
#pragma unroll
                    for (int e = 0; e < VE; ++e) w[e] = v[e] == edge ? (taken >> e) & 1u : 0u;
                    return taken != 0;
                },
                [&](uint64_t) { return m - 1; },
                [&](int id, float, uint64_t) {
                    for (int r = 0; r < ranks; ++r) *cl.map_shared_rank(&sm.found, r) = id;
                });
            cl.sync();
            last = sm.found;
        }
        return topk_key(edge, last);
    }

    // How many of this CTA's entries that stay lie in each bin, into count.  Four
    // copies of the counts: a warp's 32 logits meet in few bins.
    __device__ __forceinline__ void count_bins(const Bins &bins, const Edge &edge) {
        uint32_t *copies = &sm.copies[0][0];
        for (int i = threadIdx.x; i < 4 * kBins; i += kThreads) copies[i] = 0;
        __syncthreads();
        each([&](const float (&x)[VE], int id) {
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (x[e] > -INFINITY && edge.stays(x[e], id + e))
                    atomicAdd(copies + 4 * Bins::at(bins.place(x[e])) + (threadIdx.x & 3), 1u);
        });
        __syncthreads();
        for (int i = threadIdx.x; i < kBins; i += kThreads) {
            const uint4 c = *reinterpret_cast<const uint4 *>(sm.copies[i]);
            sm.count[i] = c.x + c.y + c.z + c.w;
        }
    }
    // Sums of weights by bins, into mass: start, add from any thread, finish.
    // 64-bit additions to shared memory are loops of compare and swap; where
    // a CTA's share of the row is resident (below 2^17 entries) a weight's three
    // limbs of 15 bits are added without waiting for an answer.
    __device__ __forceinline__ void mass_start(int bins) {
        for (int i = threadIdx.x; i < bins; i += kThreads) {
            sm.mass[i] = 0;
            if (RESIDENT) *reinterpret_cast<uint4 *>(sm.limbs[i]) = make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
    }
    __device__ __forceinline__ void mass_add(int bin, uint64_t w) {
        if constexpr (RESIDENT) {
            atomicAdd(&sm.limbs[bin][0], static_cast<uint32_t>(w) & 0x7FFFu);
            atomicAdd(&sm.limbs[bin][1], static_cast<uint32_t>(w >> 15) & 0x7FFFu);
            atomicAdd(&sm.limbs[bin][2], static_cast<uint32_t>(w >> 30));
        } else {
            atomicAdd(reinterpret_cast<unsigned long long *>(&sm.mass[bin]), w);
        }
    }
    __device__ __forceinline__ void mass_finish(int bins) {
        __syncthreads();
        if constexpr (RESIDENT) {
            for (int i = threadIdx.x; i < bins; i += kThreads)
                sm.mass[i] += sm.limbs[i][0] + (static_cast<uint64_t>(sm.limbs[i][1]) << 15) +
                              (static_cast<uint64_t>(sm.limbs[i][2]) << 30);
        }
    }

    // The key at which the sums of value over bin b's entries (n of them stay by
    // `in`) reach need: where they are many, the bin in 256 parts and the
    // entries of the part.
    template <typename G>
    __device__ __forceinline__ uint64_t narrow(const Bins &bins, int b, uint64_t n, uint64_t need, const Edge &in,
                                               const G &value) {
        const float first = static_cast<float>(b);
        auto within = [&](const float (&x)[VE], int id) {
            uint32_t mask = 0;
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float at = bins.place(x[e]) - first;
                mask |= at >= 0.0f && at < 1.0f && x[e] > -INFINITY && in.stays(x[e], id + e) ? 1u << e : 0u;
            }
            return mask;
        };
        if (n <= kList) return cut(within, value, need);
        __syncthreads();
        mass_start(kParts);
        each([&](const float (&x)[VE], int id) {
            const uint32_t mask = within(x, id);
            if (mask == 0) return;
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if ((mask >> e) & 1u)
                    mass_add(Bins::at((bins.place(x[e]) - first) * static_cast<float>(kParts)), value(x[e]));
        });
        mass_finish(kParts);
        const int part = crossing<kParts>(sm.mass, need);
        const float from = static_cast<float>(part), past = from + 1.0f;
        const uint64_t rest = need - sm.above;
        return cut(
            [&](const float (&x)[VE], int id) {
                uint32_t mask = within(x, id);
                if (mask == 0) return mask;
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float at = (bins.place(x[e]) - first) * static_cast<float>(kParts);
                    if (!(at >= from && at < past)) mask &= ~(1u << e);
                }
                return mask;
            },
            value, rest);
    }

    // All weights that stay into mass: bins ba .. bb one by one, those above
    // them in bin 0 and those below in the last (which leaves the sums up to
    // each bin of the bracket, and of all, as they are).
    template <bool EDGED>
    __device__ __forceinline__ void bracket(const Bins &bins, const Weigh<EDGED, false, VE> &weigh, int ba, int bb) {
        const float from = static_cast<float>(ba), past = bb < kBins - 1 ? static_cast<float>(bb + 1) : INFINITY;
        uint64_t over = 0, under = 0;
        mass_start(kBins);
        each([&](const float (&x)[VE], int id) {
            uint64_t w[VE];
            if (!weigh(x, id, w)) return;
            uint32_t inside = 0;
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float at = bins.place(x[e]);
                over += at < from ? w[e] : 0ull;
                under += at >= past ? w[e] : 0ull;
                inside |= at >= from && at < past && w[e] ? 1u << e : 0u;
            }
            if (inside == 0) return;
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if ((inside >> e) & 1u) mass_add(Bins::at(bins.place(x[e])), w[e]);
        });
        over = warp_add(over);
        under = warp_add(under);
        if ((threadIdx.x & 31) == 0) {
            if (over) atomicAdd(reinterpret_cast<unsigned long long *>(&sm.mass[0]), over);
            if (under) atomicAdd(reinterpret_cast<unsigned long long *>(&sm.mass[kBins - 1]), under);
        }
        mass_finish(kBins);
    }

    // The first id at which the running sum of weights passes target(total):
    // the one thread that finds it calls found(id, logit, total).
    // value(values, id, weights): false where all of a word's weights are 0.
    template <typename F, typename G, typename H>
    __device__ __forceinline__ void locate(const F &value, const G &target, const H &found) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        uint64_t s = 0;
        each([&](const float (&v)[VE], int id) {
            uint64_t x[VE];
            if (!value(v, id, x)) return;
#pragma unroll
            for (int e = 0; e < VE; ++e) s += x[e];
        });
        const uint64_t *all = exchange(cta_sum(sm, s));
        uint64_t before = 0, total = 0;
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i) {
            if (i < rank) before += all[i];
            if (i < ranks) total += all[i];
        }
        const uint64_t t = target(total);
        // the warp whose piece holds the answer; the whole CTA walks that piece
        int at = -1;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const uint64_t x = sm.warp_sum[w];
            if (at < 0 && t >= before && t < before + x) at = w;
            if (at < 0) before += x;
        }
        __syncthreads();
        if (at >= 0) {
            const int words = steps * 32;
            const int w0 = word0 - lane + (at - warp) * words;  // the piece's first word
            const uint4 *src = hold - lane + (at - warp) * words;
            for (int i0 = 0; i0 < words; i0 += kThreads) {
                const int i = i0 + threadIdx.x;
                float v[VE];
                widen(i < words ? (RESIDENT ? src[i] : fetch(w0 + i)) : outside(), v);
                const int id = (w0 + i) * VE - skip;
                uint64_t x[VE], mine_i = 0;
                const bool some = value(v, id, x);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    if (!some) x[e] = 0;
                    mine_i += x[e];
                }
                uint64_t all_i, run = before + cta_scan(sm, mine_i, all_i);
                if (t >= run && t < run + mine_i) {
                    int at_id = -1;
                    float at_logit = 0.0f;
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        run += x[e];
                        if (at_id < 0 && run > t) {
                            at_id = id + e;
                            at_logit = v[e];
                        }
                    }
                    found(at_id, at_logit, total);
                }
                before += all_i;
                __syncthreads();
            }
        }
    }
};

// A fraction 0 <= f < 1 in units of 2^-64 (exact above 2^-40).
__device__ __forceinline__ uint64_t fraction64(float f) { return __float2ull_rz(f * 0x1p64f); }
// a / b to about 2^-24 of itself, a, b > 0, in two floats a number.
__device__ __forceinline__ float quotient(uint64_t a, uint64_t b) {
    const float ah = __ull2float_rn(a), bh = __ull2float_rn(b);
    const float al = __ll2float_rn(static_cast<int64_t>(a - __float2ull_rn(ah)));
    const float bl = __ll2float_rn(static_cast<int64_t>(b - __float2ull_rn(bh)));
    const float q = __fdiv_rn(ah, bh);
    const float rest = __fmaf_rn(-q, bh, ah) + __fmaf_rn(-q, bl, al);
    return q + __fdiv_rn(rest, bh);
}
// The drawn token's weight over the total of those that stayed.  Its weight is
// taken before it is cut to whole units: an unlikely token has few of them.
__device__ __forceinline__ float probability(const Weight &weight, float logit, uint64_t total) {
    int cut;
    const uint64_t w = weight.whole(logit, cut);
    return quotient(w, total) * __uint_as_float(static_cast<uint32_t>(127 - cut) << 23);
}
// The least integer that is at least P 2^-64 of all (1 at least).
__device__ __forceinline__ uint64_t share_of(uint64_t P, uint64_t all) {
    const uint64_t need = __umul64hi(P, all) + (P * all != 0 ? 1 : 0);
    return need ? need : 1;
}

// A row that the filters have narrowed to the n <= kList entries of the list, in
// any order, in one CTA: top-k of them, top-p, min-p and the draw.
__device__ __forceinline__ void finish_list(Shared &sm, const Weight &weight, int n, int k, float top_p,
                                            uint64_t floor_w, int32_t *id, float *prob) {
    constexpr int E = kList / kThreads;
    const int first = threadIdx.x * E, most = k < n ? k : n;
    sort_list(sm, n);
    uint64_t w[E], mine = 0, all;
    uint64_t entry[E];
    uint32_t id_key[E];  // inverted ids, 0 for none
#pragma unroll
    for (int e = 0; e < E; ++e) {
        entry[e] = first + e < most ? sm.list[first + e] : 0ull;
        w[e] = entry[e] ? weight(key_value(entry[e])) : 0ull;
        id_key[e] = static_cast<uint32_t>(entry[e]);
        mine += w[e];
    }
    uint64_t above = cta_scan(sm, mine, all);
    const uint64_t need = top_p < 1.0f ? share_of(sm.scale.P, all) : ~0ull;
    // those that stay (a head of the list), then their places in ascending order of ids
    int kept = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const bool stays = above < need && w[e] >= floor_w && w[e] > 0;
        above += w[e];
        if (!stays) id_key[e] = 0;
        kept += stays;
        sm.count[first + e] = id_key[e];
    }
    __syncthreads();
    int place[E] = {};
    if (__any_sync(0xFFFFFFFFu, kept > 0)) {
        const uint4 *four = reinterpret_cast<const uint4 *>(sm.count);
#pragma unroll 4
        for (int j = 0; j < (most + 3) / 4; ++j) {
            const uint4 k4 = four[j];
#pragma unroll
            for (int e = 0; e < E; ++e)
                place[e] += (k4.x > id_key[e] ? 1 : 0) + (k4.y > id_key[e] ? 1 : 0) + (k4.z > id_key[e] ? 1 : 0) +
                            (k4.w > id_key[e] ? 1 : 0);
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm.mass[first + e] = 0;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (id_key[e]) {
            sm.mass[place[e]] = w[e];
            sm.list[place[e]] = entry[e];
        }
    __syncthreads();
    mine = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        w[e] = sm.mass[first + e];
        mine += w[e];
    }
    above = cta_scan(sm, mine, all);
    const uint64_t t = __umul64hi(sm.scale.U, all);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (above <= t && t < above + w[e]) {
            const uint64_t drawn = sm.list[first + e];
            *id = key_id(drawn);
            if (prob) *prob = probability(weight, key_value(drawn), all);
        }
        above += w[e];
    }
}

template <int DT, bool RESIDENT>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p, const int S, const int steps) {
    using View = RowView<DT, RESIDENT>;
    constexpr int VE = View::VE;
    extern __shared__ __align__(16) uint8_t dyn_smem[];
    Shared &sm = *reinterpret_cast<Shared *>(dyn_smem);
    cg::cluster_group cl = cg::this_cluster();
    const int rank = static_cast<int>(cl.block_rank()), ranks = static_cast<int>(cl.num_blocks());
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid < 16) sm.pow16[tid] = kPow16[tid];
    if (lane == 0) {
        mbar_init(&sm.arrived[warp], 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_trigger();
    pdl_wait();
    cl.sync();  // the peers run: their shared memory may be written

    View v{sm, cl, rank, ranks, nullptr, steps, (rank * kWarps + warp) * steps * 32 + lane, p.vocab, nullptr, 0, 0};
    v.hold = reinterpret_cast<uint4 *>(dyn_smem + sizeof(Shared)) + warp * steps * 32 + lane;

    uint32_t parity = 0;
    for (int64_t r = blockIdx.x / ranks; r < p.rows; r += gridDim.x / ranks, parity ^= 1u) {
        const uintptr_t row = reinterpret_cast<uintptr_t>(static_cast<const typename View::T *>(p.logits) + r * p.stride);
        v.base = reinterpret_cast<const uint4 *>(row & ~uintptr_t(15));
        v.skip = static_cast<int>((row & 15) / sizeof(typename View::T));
        v.start();
        const float u = ld_dep(p.u + r);
        float T = p.temperature ? ld_dep(p.temperature + r) : 1.0f;
        const float top_p = p.top_p ? ld_dep(p.top_p + r) : 1.0f;
        const float min_p = p.min_p ? ld_dep(p.min_p + r) : 0.0f;
        int k = p.top_k ? ld_dep(p.top_k + r) : 0;
        v.ends();
        const bool bad_param = !(T >= 0.0f && T <= 3.4028234663852886e38f) || !(top_p > 0.0f && top_p <= 1.0f) ||
                               !(min_p >= 0.0f && min_p <= 1.0f) || !(u >= 0.0f && u < 1.0f);
        if (T == 0.0f) {  // greedy
            T = 1.0f;
            k = 1;
        }
        T = fminf(fmaxf(T, 0x1p-100f), 0x1p100f);
        if (k <= 0 || k >= p.vocab) k = p.vocab;

        if (tid == 0) {
            constexpr float kLog2eHi = 1.44269502162933349609375f, kLog2eLo = 1.925963033500e-8f;
            const float c_hi = __fdiv_rn(kLog2eHi, T);
            RowScale &x = sm.scale;
            x.c_hi = c_hi;
            x.c_lo = __fdiv_rn(__fmaf_rn(-c_hi, T, kLog2eHi) + kLog2eLo, T);
            x.span = min_p > 0.0f ? (0.001f - log2f(min_p)) / c_hi : INFINITY;
            x.U = fraction64(u);
            x.P = fraction64(top_p);
            x.M = fraction64(min_p);
        }
        // the row's largest logit (as an order key: NaN lies above +inf, a late piece above that)
        const uint32_t lane_top = v.read(parity, p.err);
        uint32_t top = __reduce_max_sync(0xFFFFFFFFu, lane_top);
        if (lane == 0) sm.warp_sum[warp] = top;
        for (int i = tid; i < kBins; i += kThreads) sm.count[i] = 0;
        __syncthreads();
        for (int i = 0; i < kWarps; ++i) top = max(top, static_cast<uint32_t>(sm.warp_sum[i]));
        const uint64_t *tops = v.exchange(top);
        for (int i = 0; i < ranks; ++i) top = max(top, static_cast<uint32_t>(tops[i]));
        if (top == kKeyLate) {
            // the whole cluster gives up, after one more wait for its copies: no id for this row and
            // those that it would have come to
            if (RESIDENT) mbar_wait(&sm.arrived[warp], parity, kWaitTimeoutNs);
            if (rank == 0 && tid == 0)
                for (; r < p.rows; r += gridDim.x / ranks) {
                    p.ids[r] = -1;
                    if (p.probs) p.probs[r] = 0.0f;
                }
            break;
        }
        if (bad_param || top >= kKeyInf || top <= kKeyNegInf) {
            if (rank == 0 && tid == 0) {
                p.ids[r] = -1;
                if (p.probs) p.probs[r] = 0.0f;
                const int bits = (bad_param ? LHS_ERRBIT_BAD_PARAM : 0) |
                                 (top >= kKeyInf ? LHS_ERRBIT_NONFINITE : 0);
                if (bits) set_err(p.err, bits);
            }
            __syncthreads();
            continue;
        }
        const float largest = key_value(static_cast<uint64_t>(top) << 32);
        Weight weight;
        weight.init(largest, sm.scale.c_hi, sm.scale.c_lo, S, sm.pow16);
        const uint64_t heaviest = weight(largest);
        const uint64_t floor_w = min_p >= 1.0f ? heaviest : min_p > 0.0f ? share_of(sm.scale.M, heaviest) : 0ull;
        const Bins bins = {largest, weight.c_hi * kBinsPerOctave};

        Edge edge = {-INFINITY, 0x7FFFFFFF};
        bool edged = false;
        if (k < p.vocab) {
            // at least k entries lie in the bins up to the one in which the k-th of the lanes' maxima does
            const float lane_max = key_value(static_cast<uint64_t>(lane_top) << 32);
            constexpr int kHalf = kBins / 2;  // bins twice as wide
            if (lane_top > kKeyNegInf) atomicAdd(&sm.count[Bins::at(bins.place(lane_max) * 0.5f)], 1u);
            const int bound = v.template crossing<kHalf>(sm.count, static_cast<uint64_t>(k));
            if (bound < kHalf - 1) {
                const float past = static_cast<float>(2 * (bound + 1));
                const int64_t n = v.gather([&](const float (&x)[VE], int) {
                    uint32_t mask = 0;
#pragma unroll
                    for (int e = 0; e < VE; ++e) mask |= bins.place(x[e]) < past ? 1u << e : 0u;
                    return mask;
                });
                if (n <= kList) {
                    if (rank == 0) {
                        v.pull(v.last_exchange());
                        finish_list(sm, weight, static_cast<int>(n), k, top_p, floor_w, p.ids + r,
                                    p.probs ? p.probs + r : nullptr);
                    }
                    if (r + gridDim.x / ranks < p.rows) cl.sync();  // the lists have been read
                    continue;
                }
            }
            cl.sync();
            // the bin of the k-th entry, then the entry
            v.count_bins(bins, edge);
            const int b = v.template crossing<kBins>(sm.count, static_cast<uint64_t>(k));
            if (b < kBins)  // else fewer than k are not masked: all of them stay
                edge.set(v.narrow(bins, b, sm.in, static_cast<uint64_t>(k) - sm.above, Edge{-INFINITY, 0x7FFFFFFF}, One()));
            edged = true;
            cl.sync();
        }
        if (top_p < 1.0f) {
            v.count_bins(bins, edge);
            if (tid == 0) {
                sm.bin = 0;
                sm.found = kBins - 1;
            }
            v.template add_up<kBins>(sm.count);
            // The bins that may be the one in which the sum of weights reaches p of all.  A bin's
            // weights lie between 2^(S - (b + 1) / 16) and 2^(S - b / 16), the last one's anywhere
            // below that, the largest taken as 2^S: bounds for the sums up to each bin and for all.
            // The largest is 2^(S - 1) units at least and each weight less than a unit below its
            // value, hence two of these less for each entry (which is what counts in rows of 2^28
            // and more, where small weights are a unit or two).
            constexpr int B = kBins / kThreads;
            static_assert(B * kThreads == kBins, "whole bins to a thread");
            uint64_t high[B], low[B], h0 = 0, l0 = 0, h_all, l_all;
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int bin = tid * B + b;
                const uint64_t c = sm.sums[bin];
                const float x = static_cast<float>(c) * exp2f(static_cast<float>(S) - bin / kBinsPerOctave);
                high[b] = static_cast<uint64_t>(x * 1.0001f) + c;
                const uint64_t l = static_cast<uint64_t>(x * 0.9575f);  // 2^(-1/16) = 0.95760..
                low[b] = bin < kBins - 1 && l > 2 * c ? l - 2 * c : 0ull;
                h0 += high[b];
                l0 += low[b];
            }
            uint64_t hs = cta_scan(sm, h0, h_all);
            __syncthreads();
            uint64_t ls = cta_scan(sm, l0, l_all);
            const uint64_t least = share_of(sm.scale.P, l_all), most = share_of(sm.scale.P, h_all);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (hs < least && hs + high[b] >= least) sm.bin = tid * B + b;
                if (ls < most && ls + low[b] >= most) sm.found = tid * B + b;
                hs += high[b];
                ls += low[b];
            }
            __syncthreads();
            const int ba = sm.bin, bb = sm.found;
            // (how many entries each has, for below)
            for (int i = tid; i < kBins; i += kThreads) sm.count[i] = static_cast<uint32_t>(sm.sums[i]);
            __syncthreads();
            if (edged) v.bracket(bins, Weigh<true, false, VE>{weight, edge, largest, 0.0f, 0}, ba, bb);
            else v.bracket(bins, Weigh<false, false, VE>{weight, edge, largest, 0.0f, 0}, ba, bb);
            const uint64_t P = sm.scale.P;
            uint64_t need;
            const int b = v.template crossing<kBins>(sm.mass, need, [&](uint64_t all) { return share_of(P, all); });
            const uint64_t rest = need - sm.above;
            const Edge kept = edge;
            edge.set(v.narrow(bins, b, b < kBins ? sm.count[b] : 0, rest, kept, weight));
            edged = true;
        }
        const float span = sm.scale.span;
        const uint64_t U = sm.scale.U;
        auto target = [&](uint64_t total) { return __umul64hi(U, total); };
        auto drawn = [&](int id, float logit, uint64_t total) {
            p.ids[r] = id;
            if (p.probs) p.probs[r] = probability(weight, logit, total);
        };
        if (edged) v.locate(Weigh<true, true, VE>{weight, edge, largest, span, floor_w}, target, drawn);
        else if (floor_w) v.locate(Weigh<false, true, VE>{weight, edge, largest, span, floor_w}, target, drawn);
        else v.locate(Weigh<false, false, VE>{weight, edge, largest, span, floor_w}, target, drawn);
        __syncthreads();
    }
    cl.sync();  // no CTA leaves while a peer may address its shared memory
}

template <int DT, bool RESIDENT>
cudaError_t launch_kernel(const SampleParams &p, int S, int steps, int ranks, cudaStream_t stream) {
    const size_t smem = sizeof(Shared) + (RESIDENT ? static_cast<size_t>(steps) * kThreads * 16 : 0);
    auto kern = sample_kernel<DT, RESIDENT>;
    {
        DeviceInfo dev;
        cudaError_t e = device_info(&dev);
        if (e != cudaSuccess) return e;
        static std::mutex mu;
        static bool done[64] = {};
        std::lock_guard<std::mutex> lock(mu);
        if (!done[dev.device]) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
            if (e != cudaSuccess) return e;
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            done[dev.device] = true;
        }
    }
    const int64_t clusters = p.rows < (1 << 20) ? p.rows : (1 << 20);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p, S, steps);
}

template <int DT>
cudaError_t launch(const SampleParams &p, cudaStream_t stream) {
    constexpr int VE = 16 / static_cast<int>(sizeof(typename Elem<DT>::T));
    int bits = 0;
    while ((1ll << bits) < p.vocab) ++bits;
    const int S = 62 - bits < 45 ? 62 - bits : 45;  // a row's sum stays below 2^62
    // words of a row, one more where a row may start inside its first
    const bool aligned = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && (p.stride % VE == 0 || p.rows == 1);
    const int64_t words = (static_cast<int64_t>(p.vocab) + VE - 1) / VE + (aligned ? 0 : 1);
    // The smallest cluster that leaves room for two CTAs on an SM (64 rows of 151,936 in bf16, min-p:
    // 31 us in clusters of 4, 65 us of 16); a larger one while SMs would be idle and a lane still has
    // more than two words (4 rows of 8,192: 13.2 us in clusters of 4, 15.2 us of 2).
    DeviceInfo dev;
    const cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    auto steps_of = [&](int ranks) { return (words + ranks * kThreads - 1) / (ranks * kThreads); };
    int ranks = 1;
    while (ranks < kMaxCluster &&
           (static_cast<int64_t>(sizeof(Shared)) + steps_of(ranks) * kThreads * 16 > kMaxSmem / 2 ||
            (p.rows * ranks < dev.num_sms && steps_of(ranks) > 2)))
        ranks *= 2;
    const int64_t steps = steps_of(ranks);
    if (sizeof(Shared) + steps * kThreads * 16 <= kMaxSmem)
        return launch_kernel<DT, true>(p, S, static_cast<int>(steps), ranks, stream);
    return launch_kernel<DT, false>(p, S, static_cast<int>(steps), ranks, stream);
}

}  // namespace

cudaError_t launch_sample(const SampleParams &p, int32_t dtype, cudaStream_t stream) {
    switch (dtype) {
    case LHS_F32: return launch<LHS_F32>(p, stream);
    case LHS_F16: return launch<LHS_F16>(p, stream);
    default: return launch<LHS_BF16>(p, stream);
    }
}

}  // namespace lhs
