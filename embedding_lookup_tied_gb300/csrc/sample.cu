// sample.cu — one token per row of logits, drawn with temperature, top-k,
// top-p and min-p from a given random number (ADR-0008 "Remote Embeddings and
// lm_head Service", POST /v1/logits, "raw logits mode for beam search /
// sampling").
//
// Mathematics.  All three filters keep a head of the row in the order (logit
// descending, id ascending), so together they keep the ids whose (order key,
// inverted id) is at least a threshold; top-k finds it by counts, top-p by
// sums of weights.  The draw inverts the running sum of the kept weights in id
// order.  Weights are 2^S exp((logit - max) / T) as 64-bit integers (see
// Weight), so every sum is exact, whatever the order in which warps, CTAs and
// atomics form it, and two passes over a row agree to the last bit.
//
// A cluster of CTAs owns a row; each warp owns one contiguous piece of it.
// The threshold is found digit by digit (11, 11 and 10 bits of the 32-bit
// order key) from histograms of counts or weights in shared memory, which the
// cluster's CTAs read from one another.
#include <cooperative_groups.h>

#include "decode.cuh"

namespace cg = cooperative_groups;

namespace lhs {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kBinsPerThread = kBins / kThreads;
constexpr uint32_t kKeyInf = 0xFF800000u;     // order key of +inf; NaN lies above
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;  // order key of -inf

// round(2^62 * 2^(-j/16))
__constant__ const uint64_t kPow16[16] = {
    0x4000000000000000ull, 0x3D495F454921B30Bull, 0x3AB031B9F7490E4Cull, 0x383337BB0AA53844ull,
    0x35D13F32B5A75ABDull, 0x3389230547E12039ull, 0x3159CA845541B6B7ull, 0x2F4228E7D6030DB0ull,
    0x2D413CCCFE779921ull, 0x2B560FBA90A852B2ull, 0x297FB5AA6C544E3Bull, 0x27BD4C982468446Bull,
    0x260DFC14636E2A5Cull, 0x2470F4DCEAC470CEull, 0x22E57078FAA2F5BAull, 0x216AB0D9F3121EC5ull};

// The weight 2^S * 2^(-(max - l) * c), c = log2(e) / T, as an integer.
//
// d = max - l is held as the rounded difference and its error, t = d * c as
// two floats, so an argument is good to about 2^-46 of itself.  With n the
// nearest integer to 16 t and x = t - n/16 (|x| <= 1/32),
//   2^-t = 2^-(n div 16) * 2^(-(n mod 16)/16) * 2^-x,
// the middle factor from a table in 62 bits and 2^-x = 1 - x ln2 + x^2 q(x)
// from its Taylor series: x ln2 in two floats, the rest (below 2^-12) in one.
// The factor's distance from 1 is below 2^-5.5 and is held as a 32-bit
// integer in units of 2^-36.  Together about 2^-36 of the weight, unbiased.
struct Weight {
    float max, c_hi, c_lo, far;
    int shift;  // 62 - S
    const uint64_t *pow16;  // kPow16 in shared memory: 16 pairs of words, one to a bank

    __device__ __forceinline__ void init(float max_, float temperature, int S, const uint64_t *table) {
        max = max_;
        const double c = 1.4426950408889634 / static_cast<double>(temperature);
        c_hi = static_cast<float>(c);
        c_lo = static_cast<float>(c - static_cast<double>(c_hi));
        far = static_cast<float>(S + 1) / c_hi;
        shift = 62 - S;
        pow16 = table;
    }
    __device__ __forceinline__ uint64_t operator()(float l) const {
        const float s = __fsub_rn(max, l);
        if (!(s <= far)) return 0ull;  // also -inf
        const float bv = __fsub_rn(s, max), av = __fsub_rn(s, bv);
        const float e = __fsub_rn(__fsub_rn(max, av), __fadd_rn(l, bv));
        const float th = __fmul_rn(s, c_hi);
        const float tl = __fmaf_rn(s, c_hi, -th) + __fmaf_rn(s, c_lo, e * c_hi);
        const float magic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer
        const float y = __fmaf_rn(th, 16.0f, magic);
        const int n = static_cast<int>(__float_as_uint(y) - 0x4B400000u);
        const float r = __fmaf_rn(__fsub_rn(y, magic), -0.0625f, th);  // exact
        const float x = __fadd_rn(r, tl), xl = __fadd_rn(__fsub_rn(r, x), tl);
        constexpr float kLn2Hi = 0.6931471824645996f, kLn2Lo = -1.9046542e-9f;
        const float p = __fmul_rn(x, kLn2Hi);
        const float pl = __fmaf_rn(x, kLn2Hi, -p) + __fmaf_rn(x, kLn2Lo, xl * kLn2Hi);
        float q = __fmaf_rn(x, -0.0013333558f, 0.009618129f);
        q = __fmaf_rn(x, q, -0.05550411f);
        q = __fmaf_rn(x, q, 0.24022651f);
        const float z = __fmaf_rn(x * x, q, -pl);
        const int delta = __float2int_rn(z * 0x1p36f) - __float2int_rn(p * 0x1p36f);  // 2^-x - 1
        const uint64_t f = pow16[n & 15];
        const uint64_t w = f + static_cast<uint64_t>(
            (static_cast<int64_t>(static_cast<int>(f >> 32)) * delta) >> 4);
        return w >> min(shift + (n >> 4), 63);
    }
};

struct Shared {
    uint64_t hist[kBins];
    uint64_t slot[2][kMaxCluster];  // one value from each CTA of the cluster, two exchanges
    uint64_t warp_sum[kWarps];
    uint64_t cross_above, cross_in;
    uint64_t pow16[16];
    int32_t cross_bin;
    int32_t found;
};

__device__ __forceinline__ uint64_t warp_add(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// One row, as one CTA of its cluster sees it.
template <int DT>
struct RowView {
    using E = Elem<DT>;
    Shared &sm;
    cg::cluster_group cl;
    int rank, ranks;
    const typename E::T *row;
    int lo, hi;  // this warp's piece
    int flip;    // which exchange slots come next

    __device__ __forceinline__ float at(int i) const { return E::widen(ld_dep(row + i)); }

    // Every CTA's v, in this CTA's shared memory.
    __device__ __forceinline__ const uint64_t *exchange(uint64_t v) {
        uint64_t *slots = sm.slot[flip];
        flip ^= 1;
        if (static_cast<int>(threadIdx.x) < ranks) cl.map_shared_rank(slots, threadIdx.x)[rank] = v;
        cl.sync();
        return slots;
    }
    // Sum over the CTA of per-warp sums; leaves them in warp_sum.
    __device__ __forceinline__ uint64_t cta_sum(uint64_t lane_sum) {
        const uint64_t w = warp_add(lane_sum);
        if ((threadIdx.x & 31) == 0) sm.warp_sum[threadIdx.x >> 5] = w;
        __syncthreads();
        uint64_t s = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) s += sm.warp_sum[i];
        return s;
    }
    template <typename F>
    __device__ __forceinline__ uint64_t row_sum(const F &value) {
        uint64_t s = 0;
        for (int i = lo + (threadIdx.x & 31); i < hi; i += 32) s += value(at(i), i);
        const uint64_t mine = cta_sum(s);
        const uint64_t *all = exchange(mine);
        uint64_t t = 0;
        for (int i = 0; i < ranks; ++i) t += all[i];
        __syncthreads();
        return t;
    }

    // The largest order key at which the sum of value over the keys from it
    // upwards reaches `need` (>= 1, at most the row's sum).  need: what is
    // left of it for that key's own elements; in: their sum.
    template <typename F>
    __device__ __forceinline__ uint32_t threshold(const F &value, uint64_t &need, uint64_t &in) {
        uint32_t prefix = 0, mask = 0;
        const int shifts[3] = {21, 10, 0};
        for (int level = 0; level < 3; ++level) {
            const int sh = shifts[level];
            const uint32_t digit = level < 2 ? 0x7FFu : 0x3FFu;
            for (int i = threadIdx.x; i < kBins; i += kThreads) sm.hist[i] = 0;
            __syncthreads();
            for (int i = lo + (threadIdx.x & 31); i < hi; i += 32) {
                const float l = at(i);
                const uint32_t k = order_key32(l);
                if ((k & mask) != prefix) continue;
                const uint64_t v = value(l, i);
                if (v) atomicAdd(reinterpret_cast<unsigned long long *>(&sm.hist[(k >> sh) & digit]), v);
            }
            cl.sync();
            // bins from the top: thread t holds bins kBins - 1 - t * kBinsPerThread - (0 ..)
            uint64_t h[kBinsPerThread], mine = 0;
#pragma unroll
            for (int b = 0; b < kBinsPerThread; ++b) {
                const int bin = kBins - 1 - (threadIdx.x * kBinsPerThread + b);
                h[b] = 0;
                for (int r = 0; r < ranks; ++r) h[b] += cl.map_shared_rank(sm.hist, r)[bin];
                mine += h[b];
            }
            uint64_t incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (static_cast<int>(threadIdx.x & 31) >= o) incl += up;
            }
            if ((threadIdx.x & 31) == 31) sm.warp_sum[threadIdx.x >> 5] = incl;
            __syncthreads();
            uint64_t above = incl - mine;
            for (int w = 0; w < static_cast<int>(threadIdx.x >> 5); ++w) above += sm.warp_sum[w];
#pragma unroll
            for (int b = 0; b < kBinsPerThread; ++b) {
                if (above < need && above + h[b] >= need) {
                    sm.cross_bin = kBins - 1 - (threadIdx.x * kBinsPerThread + b);
                    sm.cross_above = above;
                    sm.cross_in = h[b];
                }
                above += h[b];
            }
            cl.sync();  // also: every CTA has read this one's histogram
            prefix |= static_cast<uint32_t>(sm.cross_bin) << sh;
            mask |= digit << sh;
            need -= sm.cross_above;
            in = sm.cross_in;
            __syncthreads();
        }
        return prefix;
    }

    // The first id at which the running sum of value passes target(total).
    template <typename F, typename G>
    __device__ __forceinline__ int locate(const F &value, const G &target, uint64_t &total) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        uint64_t s = 0;
        for (int i = lo + lane; i < hi; i += 32) s += value(at(i), i);
        const uint64_t mine = cta_sum(s);
        const uint64_t *all = exchange(mine);
        uint64_t before = 0;
        total = 0;
        for (int i = 0; i < ranks; ++i) {
            if (i < rank) before += all[i];
            total += all[i];
        }
        const uint64_t t = target(total);
        for (int w = 0; w < warp; ++w) before += sm.warp_sum[w];
        if (t >= before && t < before + sm.warp_sum[warp]) {  // in this warp's piece
            for (int i0 = lo; i0 < hi; i0 += 32) {
                const int i = i0 + lane;
                uint64_t incl = i < hi ? value(at(i), i) : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                    if (lane >= o) incl += up;
                }
                const unsigned hit = __ballot_sync(0xFFFFFFFFu, before + incl > t);
                if (hit) {
                    if (lane < ranks) *cl.map_shared_rank(&sm.found, lane) = i0 + __ffs(hit) - 1;
                    break;
                }
                before += __shfl_sync(0xFFFFFFFFu, incl, 31);
            }
        }
        cl.sync();
        return sm.found;
    }
};

// A fraction of 0 <= f < 1 in units of 2^-64 (exact above 2^-40).
__device__ __forceinline__ uint64_t fraction64(float f) {
    return static_cast<uint64_t>(static_cast<double>(f) * 0x1p64);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p, const int S) {
    __shared__ Shared sm;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = static_cast<int>(cl.block_rank()), ranks = static_cast<int>(cl.num_blocks());
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid < 16) sm.pow16[tid] = kPow16[tid];
    pdl_trigger();
    pdl_wait();
    cl.sync();  // the peers run: their shared memory may be written

    const int seg = ((p.vocab + ranks * kWarps - 1) / (ranks * kWarps) + 31) & ~31;
    const int64_t first = static_cast<int64_t>(rank * kWarps + warp) * seg;
    const int lo = static_cast<int>(first < p.vocab ? first : p.vocab);
    const int hi = static_cast<int>(first + seg < p.vocab ? first + seg : p.vocab);
    RowView<DT> v{sm, cl, rank, ranks, nullptr, lo, hi, 0};

    for (int64_t r = blockIdx.x / ranks; r < p.rows; r += gridDim.x / ranks) {
        v.row = static_cast<const typename Elem<DT>::T *>(p.logits) + r * p.stride;
        const float u = ld_dep(p.u + r);
        float T = p.temperature ? ld_dep(p.temperature + r) : 1.0f;
        const float top_p = p.top_p ? ld_dep(p.top_p + r) : 1.0f;
        const float min_p = p.min_p ? ld_dep(p.min_p + r) : 0.0f;
        int k = p.top_k ? ld_dep(p.top_k + r) : 0;
        const bool bad_param = !(T >= 0.0f && T <= 3.4028234663852886e38f) || !(top_p > 0.0f && top_p <= 1.0f) ||
                               !(min_p >= 0.0f && min_p <= 1.0f) || !(u >= 0.0f && u < 1.0f);
        if (T == 0.0f) {  // greedy
            T = 1.0f;
            k = 1;
        }
        T = fminf(fmaxf(T, 0x1p-100f), 0x1p100f);

        // the row's largest logit (as an order key: NaN lies above +inf)
        uint32_t top = 0;
        for (int i = lo + lane; i < hi; i += 32) top = max(top, order_key32(v.at(i)));
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if (lane == 0) sm.warp_sum[warp] = top;
        __syncthreads();
        for (int i = 0; i < kWarps; ++i) top = max(top, static_cast<uint32_t>(sm.warp_sum[i]));
        const uint64_t *tops = v.exchange(top);
        for (int i = 0; i < ranks; ++i) top = max(top, static_cast<uint32_t>(tops[i]));
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
        Weight weight;
        weight.init(key_value(static_cast<uint64_t>(top) << 32), T, S, sm.pow16);

        // what stays: keys above `edge`, and those equal to it up to id `last`
        uint32_t edge = 0;
        int last = 0x7FFFFFFF;
        auto stays = [&](uint32_t key, int i) { return key > edge || (key == edge && i <= last); };
        if (k > 0 && k < p.vocab) {
            uint64_t need = static_cast<uint64_t>(k), in = 0;
            const uint32_t e = v.threshold([](float, int) { return uint64_t(1); }, need, in);
            if (need < in) {
                uint64_t total;
                last = v.locate([&](float l, int) { return uint64_t(order_key32(l) == e); },
                                [&](uint64_t) { return need - 1; }, total);
            }
            edge = e;
        }
        if (top_p < 1.0f) {
            auto kept = [&](float l, int i) { return stays(order_key32(l), i) ? weight(l) : uint64_t(0); };
            const uint64_t all = v.row_sum(kept), P = fraction64(top_p);
            uint64_t need = __umul64hi(P, all) + (P * all != 0 ? 1 : 0), in = 0;
            if (need == 0) need = 1;
            const uint32_t e = v.threshold(kept, need, in);
            const uint64_t one = weight(key_value(static_cast<uint64_t>(e) << 32));
            const uint64_t m = (need + one - 1) / one;  // of the in / one equal logits
            if (m < in / one) {
                uint64_t total;
                last = v.locate([&](float l, int i) {
                                    const uint32_t key = order_key32(l);
                                    return uint64_t(key == e && stays(key, i));
                                },
                                [&](uint64_t) { return m - 1; }, total);
            } else if (e != edge) {
                last = 0x7FFFFFFF;
            }
            edge = e;
        }
        const uint64_t floor_w = static_cast<uint64_t>(ceil(ldexp(static_cast<double>(min_p), S)));
        uint64_t total;
        const uint64_t U = fraction64(u);
        const int id = v.locate(
            [&](float l, int i) {
                if (!stays(order_key32(l), i)) return uint64_t(0);
                const uint64_t w = weight(l);
                return w >= floor_w ? w : uint64_t(0);
            },
            [&](uint64_t t) { return __umul64hi(U, t); }, total);
        if (rank == 0 && tid == 0) {
            p.ids[r] = id;
            if (p.probs) p.probs[r] = static_cast<float>(static_cast<double>(weight(v.at(id))) /
                                                         static_cast<double>(total));
        }
        __syncthreads();
    }
    cl.sync();  // no CTA leaves while a peer may address its shared memory
}

template <int DT>
cudaError_t launch(const SampleParams &p, cudaStream_t stream) {
    int bits = 0;
    while ((1ll << bits) < p.vocab) ++bits;
    const int S = 62 - bits < 45 ? 62 - bits : 45;  // a row's sum stays below 2^62
    int ranks = 1;
    while (ranks < kMaxCluster && static_cast<int64_t>(ranks) * 8192 < p.vocab) ranks *= 2;
    const int64_t clusters = p.rows < (1 << 20) ? p.rows : (1 << 20);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * ranks));
    cfg.blockDim = dim3(kThreads);
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
    return cudaLaunchKernelEx(&cfg, sample_kernel<DT>, p, S);
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
