// i8_matmul.cu — the lm_head as a product in 8 bits: logits[t][c] =
// (sum_j a[t][j] w[c][j]) * a_scale[t] * w_scale[c], integers summed exactly
// (ADR-0008 "Remote Embeddings and lm_head Service", POST /v1/logits, over a
// table and residuals in the i8 form of ADR-0009 "Wire Format Evolution").
//
// The 5th-generation tensor cores of this chip multiply f16 far faster than
// integers, and an 8-bit code is exact in f16, as is a product of two in the
// f32 accumulator.  So the table stays in 8 bits in HBM and on its way into
// shared memory, and is widened to f16 on the SM, straight into tensor memory:
//   TMA -> shared memory (codes) -> registers (f16) -> TMEM (operand A),
// while the tokens, few next to the table's rows, are written out as f16 once
// by a first kernel and staged by TMA as operand B.  A pair of CTAs owns 256
// channels x up to 256 tokens (tcgen05 cta_group::2: each CTA holds 128
// channels and half of the tokens' tile).
//
// Roles in a CTA: one warp streams the table, one the tokens, one issues the
// MMAs, and 8 or 16 widen the codes and take the sums out, in groups of four
// warps that take the stages in turn (a stage's waits, loads, widening and
// TMEM store are one chain of about 1,000 clocks).
//
// Exact sums.  f32 sums of integers are exact while they stay within 2^24.  A
// partial sum over some k is at most 128 * sum|a|; the first kernel leaves,
// for each token, the largest sum|a| over 128 codes, b, so n = floor(2^24 /
// (128 b)) blocks of 128 (at least 8) may be summed in the tensor cores.  Longer
// sums are taken out every n blocks and added up as 32-bit integers.
//
// What bounds it.  256 x 262,144 x 5,120: the tensor cores (387 us, 1,775
// TFLOP/s, the sustained bf16 rate and a little more; 429 us back to back for
// seconds, under the power cap; HBM alone would take 238 us).  628 x 151,936 x
// 896 (143 us; 99 us by that rate): a tile is seven stages, and the warps that
// widen also write its 224 results a channel, about 4,300 of its 11,300 clocks;
// the tensor cores are busy 56% of the time.  64 x 262,144 x 768 (50 us; 35 us of
// HBM): the widening chain (48 us with the MMAs left out).
// Tried and not kept: results of 16 bits written two channels to a word (no
// change), a tile's results written between the next tile's stages (143 -> 235
// us), tiles of at most 128 or 192 tokens (batch 392 -> 503 us).
#include <mutex>

#include "i8_common.cuh"

namespace lhs {

namespace {

__host__ __device__ constexpr int64_t align_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// Workspace: the tokens as f16 [tokens][kpad] (zeros past hidden), their
// scales, and each one's largest sum|a| over a block of 128 codes.
struct Layout {
    int kpad;
    int64_t scales, peaks, bytes;
};
Layout layout_of(int hidden, int64_t tokens) {
    Layout l;
    l.kpad = static_cast<int>(align_up(hidden, kStageK));
    l.scales = align_up(tokens * l.kpad * 2, 256);
    l.peaks = l.scales + align_up(tokens * 4, 256);
    l.bytes = l.peaks + align_up(tokens * 4, 256);
    return l;
}

// ---------------------------------------------------------------------------
// tokens: codes as f16, scale, peak
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 256;
constexpr int kPrepWarps = kPrepThreads / 32;
constexpr int kPrepSteps = 6;  // blocks of 128 a warp keeps in registers: rows up to 6,144 values

// Four codes (small integers) as f16, and the warp's sum of their magnitudes.
__device__ __forceinline__ int store_codes(__half *dst, const int (&q)[4]) {
    const __half2 a = __floats2half2_rn(static_cast<float>(q[0]), static_cast<float>(q[1]));
    const __half2 b = __floats2half2_rn(static_cast<float>(q[2]), static_cast<float>(q[3]));
    *reinterpret_cast<uint2 *>(dst) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    return __reduce_add_sync(0xFFFFFFFFu, abs(q[0]) + abs(q[1]) + abs(q[2]) + abs(q[3]));
}

// One CTA per wide token; a warp takes blocks of 128 values, four to a lane,
// and keeps the first kPrepSteps of them in registers between the maximum and
// the codes.
template <int DT>
__global__ void __launch_bounds__(kPrepThreads)
    i8_prep_wide_kernel(const typename Elem<DT>::T *x, int64_t x_stride, bool vec, int64_t tokens, int hidden,
                        int kpad, __half *codes, float *scales, int32_t *peaks, int32_t *err) {
    __shared__ float sm_m[kPrepWarps];
    __shared__ int sm_f[kPrepWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int blocks = kpad / kStageK;
    pdl_wait();
    pdl_trigger();  // after the wait: the product streams the table before its own, and an earlier
                    // kernel of the stream may be the one that quantised it
    for (int64_t r = blockIdx.x; r < tokens; r += gridDim.x) {
        const typename Elem<DT>::T *row = x + r * x_stride;
        float v[kPrepSteps][4];
        float m = 0.0f;
        int bad = 0;
        auto scan = [&](const float (&w)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (isfinite(w[i])) m = fmaxf(m, fabsf(w[i]));
                else bad = 1;
            }
        };
#pragma unroll
        for (int s = 0; s < kPrepSteps; ++s)
            if (warp + s * kPrepWarps < blocks)
                load4<DT>(row, (warp + s * kPrepWarps) * kStageK + lane * 4, hidden, vec, v[s]);
#pragma unroll
        for (int s = 0; s < kPrepSteps; ++s)
            if (warp + s * kPrepWarps < blocks) scan(v[s]);
        for (int b = warp + kPrepSteps * kPrepWarps; b < blocks; b += kPrepWarps) {
            float w[4];
            load4<DT>(row, b * kStageK + lane * 4, hidden, vec, w);
            scan(w);
        }
        block_max_or(m, bad, sm_m, sm_f);
        const float scale = bad ? 0.0f : __fdiv_rn(m, 127.0f);
        const float rcp = __frcp_rn(scale);
        int peak = 0;
        auto emit = [&](const float (&w)[4], int b) {
            int q[4];
            i8_codes<4>(w, scale, rcp, q);
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = static_cast<int8_t>(q[i]);
            peak = max(peak, store_codes(codes + r * kpad + b * kStageK + lane * 4, q));
        };
#pragma unroll
        for (int s = 0; s < kPrepSteps; ++s)
            if (warp + s * kPrepWarps < blocks) emit(v[s], warp + s * kPrepWarps);
        for (int b = warp + kPrepSteps * kPrepWarps; b < blocks; b += kPrepWarps) {
            float w[4];
            load4<DT>(row, b * kStageK + lane * 4, hidden, vec, w);
            emit(w, b);
        }
        if (lane == 0) sm_f[warp] = peak;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kPrepWarps; ++w) peak = max(peak, sm_f[w]);
            peaks[r] = peak;
            scales[r] = scale;
            if (bad) set_err(err, LHS_ERRBIT_NONFINITE);
        }
        __syncthreads();
    }
}

// One CTA per coded token.
__global__ void __launch_bounds__(kPrepThreads)
    i8_prep_coded_kernel(const lhs_i8 a, bool words, int kpad, __half *codes, float *scales, int32_t *peaks,
                         int32_t *err) {
    __shared__ int sm_f[kPrepWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();  // after the wait, as above
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int8_t *row = a.codes + r * a.stride;
        int peak = 0;
        for (int b = warp; b < kpad / kStageK; b += kPrepWarps) {
            const int j = b * kStageK + lane * 4;
            int q[4];
            if (words && j + 4 <= a.hidden) {
                const uint32_t w = ld_dep(reinterpret_cast<const uint32_t *>(row + j));
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = static_cast<int8_t>(w >> (8 * i));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = j + i < a.hidden ? ld_dep(row + j + i) : 0;
            }
            peak = max(peak, store_codes(codes + r * kpad + j, q));
        }
        if (lane == 0) sm_f[warp] = peak;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kPrepWarps; ++w) peak = max(peak, sm_f[w]);
            peaks[r] = peak;
            scales[r] = coded_scale(a, r, err);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------
constexpr int kPairRows = 2 * kCtaRows;             // a CTA's are its TMEM lanes
constexpr int kTmemCols = 512;
constexpr int kSlotCols = kStageK / 2;              // of one stage's widened codes
constexpr int kPeakBlocks = (1 << 24) / kStageK;    // n = kPeakBlocks / peak

// By the most tokens of a tile: the groups of four warps that widen codes (a
// group takes every kGroups-th stage, and an equal part of the sums), the
// ring depths that fill shared memory, and how tensor memory is split.
template <int NMAX>
struct Tile {
    static constexpr int kGroups = NMAX == 256 ? 2 : 4;
    static constexpr int kConvWarps = 4 * kGroups;
    static constexpr int kThreads = 32 * (kConvWarps + 4);  // + table producer, token producer, MMA issuer, idle
    static constexpr int kAccs = NMAX == 256 ? 1 : 2;
    static constexpr int kColA = kAccs * NMAX;               // first column of the widened codes
    static constexpr int kSlots = 4;                         // stages the MMAs may hold, a multiple of the groups
    static constexpr int kTokenStageBytes = NMAX / 2 * kStageK * 2;  // this CTA's half of the tokens
    static constexpr int kTableStages = (208 * 1024 - kSlots * kTokenStageBytes) / kTableStageBytes;
    static constexpr int kAhead = kSlots - 1;                // stages widened before a finished sum is taken out
    static constexpr int kPart = NMAX / kGroups;             // tokens whose sums a warp takes out
};

template <int NMAX>
struct Smem {
    using T = Tile<NMAX>;
    static_assert(T::kSlots % T::kGroups == 0 && T::kTableStages >= T::kSlots && T::kColA + T::kSlots * kSlotCols <= kTmemCols,
                  "see the waits of the widening warps");
    uint8_t table[T::kTableStages][kTableStageBytes];
    uint8_t token[T::kSlots][T::kTokenStageBytes];
    uint64_t table_full[T::kTableStages], table_empty[T::kTableStages];
    uint64_t full[T::kSlots], empty[T::kSlots];  // a stage's operands, widened codes and tokens
    uint64_t acc_full[2], acc_empty[2];
    uint32_t tmem_base;
    int abort_flag;
};

struct Params {
    const uint8_t *w_scales;
    int64_t w_scale_stride;
    int64_t channels, tokens;
    int n;         // tokens per tile, a multiple of 32
    int blocks;    // of tokens
    int nk;        // stages per tile
    int64_t items; // channel tiles x token blocks
    const float *scales;
    const int32_t *peaks;
    void *out;
    int64_t out_stride;
    int out_dtype;
    int32_t *err;
};

__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(uint32_t smem_addr, uint32_t cta) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr), "r"(cta));
    return r;
}
// TMA load into this CTA's shared memory, counted on a barrier of either CTA.
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, uint32_t bar_cluster,
                                                 int32_t c0, int32_t c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(c0), "r"(c1)
        : "memory");
}
// Arrive on a barrier of either CTA.  What it orders is tensor memory, by the
// tcgen05 waits and fences around it; a release at cluster scope would add a
// fence of all memory, which held every stage up by about 0.5 us.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
// Low word of the shared-memory matrix descriptor; the high word is constant:
// K-major, 128-byte swizzle, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | (1u << 16); }
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

// One lane of the warp, for the instructions below: the whole warp runs the
// loop around them, so that their operands stay in uniform registers (in a
// branch of one lane every operand of every MMA was moved there first, about
// 85 clocks an MMA).
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p)::"memory");
    return p;
}
// A in TMEM (the widened codes of both CTAs, same columns), B in shared memory.
__device__ __forceinline__ void umma_f16_ts(uint32_t elected, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 b, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(elected), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void umma_commit_both(uint32_t elected, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::
            "r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(0x3)), "r"(elected)
        : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// 8 consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float *v) {
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// 32 consecutive columns of this thread's TMEM lane, written.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
// The tile a pair works on: channels from 256 tile, tokens from n block.  Items
// (tile, block), blocks innermost, are dealt out to the pairs in turn; a step
// is worked out once, so that no tile waits for a division.
struct Item {
    int64_t tile;
    int block, blocks, step_block;
    int64_t step_tile;
    __device__ __forceinline__ Item(int64_t first, int64_t step, int blocks_) : blocks(blocks_) {
        tile = first / blocks;
        block = static_cast<int>(first - tile * blocks);
        step_tile = step / blocks;
        step_block = static_cast<int>(step - step_tile * blocks);
    }
    __device__ __forceinline__ void next() {
        tile += step_tile;
        block += step_block;
        if (block >= blocks) {
            block -= blocks;
            ++tile;
        }
    }
};

// A place in a ring of N slots and the parity of its phase.
template <int N>
struct Ring {
    int i = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) {
            i = 0;
            parity ^= 1u;
        }
    }
};

// Whether the phase is over, acquiring what both CTAs of the pair released.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// The same look without a wait.
__device__ __forceinline__ bool mbar_test_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// Bounded wait that gives up at once when the CTA has already aborted.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, int *abort_flag, int32_t *err) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if (*reinterpret_cast<const volatile int *>(abort_flag)) return false;
    const uint64_t t0 = global_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait_cluster(bar, parity)) return true;
        if (global_ns() - t0 > kWaitTimeoutNs) break;
    }
    set_err(err, LHS_ERRBIT_TIMEOUT);
    *reinterpret_cast<volatile int *>(abort_flag) = 1;
    return false;
}

// Blocks of 128 codes that may be summed in f32.  Warp-collective.
__device__ __forceinline__ int blocks_per_sum(const Params &p, int lane) {
    int peak = 0;
    for (int64_t t = lane; t < p.tokens; t += 32) peak = max(peak, ld_dep(p.peaks + t));
    peak = __reduce_max_sync(0xFFFFFFFFu, peak);
    return peak ? kPeakBlocks / peak : p.nk;
}

template <int NMAX>
__global__ void __launch_bounds__(Tile<NMAX>::kThreads, 1)
    i8_matmul_kernel(const __grid_constant__ CUtensorMap tm_table, const __grid_constant__ CUtensorMap tm_token,
                     const Params p) {
    using T = Tile<NMAX>;
    constexpr int SW = T::kTableStages, SX = T::kSlots, ACCS = T::kAccs, kConvWarps = T::kConvWarps;
    extern __shared__ uint8_t dyn_smem[];
    Smem<NMAX> &sm = *reinterpret_cast<Smem<NMAX> *>(smem_align<1024>(dyn_smem));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int64_t cl = blockIdx.x >> 1, clusters = gridDim.x >> 1;
    const int64_t mine = cl < p.items ? (p.items - cl + clusters - 1) / clusters : 0;  // tiles of this pair
    const int64_t total = mine * p.nk;                                                 // stages

    if (tid == 0) {
        for (int s = 0; s < SW; ++s) {
            mbar_init(&sm.table_full[s], 1);
            mbar_init(&sm.table_empty[s], 4);
        }
        for (int s = 0; s < SX; ++s) {
            mbar_init(&sm.full[s], 1 + 2 * 4);  // leader: both CTAs' bytes, and a group of warps of each
            mbar_init(&sm.empty[s], 1);         // the leader's commit, to both
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.acc_full[s], 1);
            mbar_init(&sm.acc_empty[s], 2 * kConvWarps);
        }
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kConvWarps + 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sm.tmem_base)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_sync_all();  // the peer's barriers exist
    const uint32_t tmem = sm.tmem_base;
    pdl_trigger();

    // The warps that hold sums take registers from the others: 8 x 216 + 4 x
    // 72 a lane are what 12 warps are launched with at 168, 16 x 104 + 4 x 64
    // what 20 are at 96.
    if (warp < kConvWarps) {
        if constexpr (NMAX == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        pdl_wait();
        const int chunk = blocks_per_sum(p, lane);
        // ---------------- widen the codes, take the sums out ----------------
        const int q = warp & 3, g = warp >> 2;  // TMEM lane quarter; group
        const int row = q * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        const int part = p.n / T::kGroups;
        // the sums of this channel against the group's part of the tile's tokens: f32 while they
        // are exact in it, 32-bit integers (whole) once they are not
        float acc[T::kPart];
        bool whole = false;
#pragma unroll
        for (int c = 0; c < T::kPart; ++c) acc[c] = 0.0f;
        Ring<SW> sw;
        Ring<T::kSlots> sa;
        Ring<ACCS> sc;
        Ring<T::kGroups> turn;
        Item it(cl, clusters, p.blocks);
        int kd = 0, in = 0;  // stage of the tile, of the sum, that the sums have got to
        // the tile's scales, asked for one tile ahead
        int64_t ch = 0, t0 = 0;
        float ws = 0.0f, as[(T::kPart + 31) / 32];
        auto ask = [&]() {
            ch = it.tile * kPairRows + static_cast<int64_t>(rank) * kCtaRows + row;
            t0 = static_cast<int64_t>(it.block) * p.n + g * part;
            if (ch < p.channels) ws = ld_dep(reinterpret_cast<const float *>(p.w_scales + ch * p.w_scale_stride));
#pragma unroll
            for (int i = 0; i < (T::kPart + 31) / 32; ++i)
                if (t0 + i * 32 + lane < p.tokens) as[i] = ld_dep(p.scales + t0 + i * 32 + lane);
        };
#pragma unroll
        for (int i = 0; i < (T::kPart + 31) / 32; ++i) as[i] = 0.0f;
        if (total > 0) ask();
        for (int64_t j = 0; j < total + T::kAhead; ++j) {
            if (j < total && turn.i == g) {
                // in this order: once the slot is free, every stage up to kSlots before this one has been
                // widened, so the copy before this one in the same place of the table's ring (at least
                // kSlots back, and perhaps another group's) has landed, and the wait for this one cannot
                // take that one's phase for its own
                bool ok = wait_or_abort(&sm.empty[sa.i], sa.parity ^ 1u, &sm.abort_flag, p.err);
                ok = ok && wait_or_abort(&sm.table_full[sw.i], sw.parity, &sm.abort_flag, p.err);
                if (!__all_sync(0xFFFFFFFFu, ok)) break;  // the tcgen05 instructions are warp-collective
                tc_fence_after();
                const uint8_t *src = sm.table[sw.i] + row * kStageK;
                const uint32_t dst = tmem + lanes + T::kColA + sa.i * kSlotCols;
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    uint32_t f[32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // 16-byte piece 4o + i of this row, swizzled
                        const uint4 u = *reinterpret_cast<const uint4 *>(src + (((4 * o + i) ^ (row & 7)) << 4));
                        widen4(u.x ^ 0x80808080u, f[8 * i], f[8 * i + 1]);
                        widen4(u.y ^ 0x80808080u, f[8 * i + 2], f[8 * i + 3]);
                        widen4(u.z ^ 0x80808080u, f[8 * i + 4], f[8 * i + 5]);
                        widen4(u.w ^ 0x80808080u, f[8 * i + 6], f[8 * i + 7]);
                    }
                    tmem_st32(dst + o * 32, f);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.table_empty[sw.i]);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_u32(&sm.full[sa.i]), 0));
            }
            sw.next();
            sa.next();
            turn.next();
            if (j < T::kAhead) continue;
            // stage j - kAhead: does a sum end with it?
            ++in;
            ++kd;
            const bool tile_done = kd == p.nk;
            if (in < chunk && !tile_done) continue;
            const bool ok = wait_or_abort(&sm.acc_full[sc.i], sc.parity, &sm.abort_flag, p.err);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_after();
            const uint32_t src = tmem + lanes + sc.i * NMAX + g * part;
            if (kd == in) {  // the tile's first sum
                whole = false;
#pragma unroll
                for (int c = 0; c < T::kPart; c += 8) {
                    if (c >= part) break;
                    tmem_ld8(src + c, &acc[c]);
                }
            } else {
                // f32 still holds the new sums exactly where all of them stay below 2^24 (a
                // larger one would round to 2^24 at least)
                float big = 0.0f;
                if (!whole) {
#pragma unroll
                    for (int c = 0; c < T::kPart; c += 8) {
                        if (c >= part) break;
                        float v[8];
                        tmem_ld8(src + c, v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(acc[c + i] + v[i]));
                    }
                    if (__any_sync(0xFFFFFFFFu, big >= 16777216.0f)) {
                        whole = true;
#pragma unroll
                        for (int c = 0; c < T::kPart; ++c) acc[c] = __int_as_float(__float2int_rn(acc[c]));
                    }
                }
                if (!whole) {
#pragma unroll
                    for (int c = 0; c < T::kPart; c += 8) {
                        if (c >= part) break;
                        float v[8];
                        tmem_ld8(src + c, v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[c + i] += v[i];
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < T::kPart; c += 8) {
                        if (c >= part) break;
                        float v[8];
                        tmem_ld8(src + c, v);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            acc[c + i] = __int_as_float(__float_as_int(acc[c + i]) + __float2int_rn(v[i]));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_u32(&sm.acc_empty[sc.i]), 0));
            sc.next();
            in = 0;
            if (!tile_done) continue;
            kd = 0;
            const bool valid = ch < p.channels;
            const int64_t left = p.tokens - t0;
            const int cols = static_cast<int>(left < part ? left : part);
            if (whole) {
#pragma unroll
                for (int c = 0; c < T::kPart; ++c) acc[c] = static_cast<float>(__float_as_int(acc[c]));
            }
            auto emit = [&](auto *out) {
                out += t0 * p.out_stride + ch;
#pragma unroll
                for (int c = 0; c < T::kPart; ++c) {
                    if (c % 8 == 0 && c >= cols) break;
                    const float v = __fmul_rn(
                        __fmul_rn(acc[c], __shfl_sync(0xFFFFFFFFu, as[c / 32], c % 32)), ws);
                    if (valid && c < cols) put(out, v);
                    out += p.out_stride;
                }
            };
            if (p.out_dtype == LHS_F32) emit(static_cast<float *>(p.out));
            else if (p.out_dtype == LHS_F16) emit(static_cast<__half *>(p.out));
            else emit(static_cast<__nv_bfloat16 *>(p.out));
            it.next();
            ask();
        }
    } else {
        if constexpr (NMAX == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == kConvWarps) {
            // ---------------- table producer (does not wait for the tokens) ----------------
            if (lane == 0) {
                tma_prefetch_map(&tm_table);
                int64_t j = 0;
                Ring<SW> st;
                bool ok = true;
                Item it(cl, clusters, p.blocks);
                for (int64_t i = 0; i < mine && ok; ++i, it.next()) {
                    const int32_t row = static_cast<int32_t>(it.tile) * kPairRows + static_cast<int32_t>(rank) * kCtaRows;
                    for (int kc = 0; kc < p.nk; ++kc, ++j, st.next()) {
                        if (!wait_or_abort(&sm.table_empty[st.i], st.parity ^ 1u, &sm.abort_flag, p.err)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&sm.table_full[st.i], kTableStageBytes);
                        tma_load_2d(sm.table[st.i], &tm_table, &sm.table_full[st.i], kc * kStageK, row);
                    }
                }
                // the copies have landed
                for (int64_t i = j > SW ? j - SW : 0; i < j; ++i) mbar_wait(&sm.table_full[i % SW], (i / SW) & 1, kWaitTimeoutNs);
            }
        } else if (warp == kConvWarps + 1) {
            // ---------------- token producer ----------------
            if (lane == 0) {
                tma_prefetch_map(&tm_token);
                pdl_wait();
                const int half = p.n / 2;
                int64_t j = 0;
                Ring<SX> st;
                bool ok = true;
                Item it(cl, clusters, p.blocks);
                for (int64_t i = 0; i < mine && ok; ++i, it.next()) {
                    const int32_t row = it.block * p.n + static_cast<int32_t>(rank) * half;
                    for (int kc = 0; kc < p.nk; ++kc, ++j, st.next()) {
                        const int s = st.i;
                        if (!wait_or_abort(&sm.empty[s], st.parity ^ 1u, &sm.abort_flag, p.err)) {
                            ok = false;
                            break;
                        }
                        if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * half * kStageK * 2);
                        const uint32_t bar = cluster_addr(smem_u32(&sm.full[s]), 0);
                        tma_load_2d_pair(sm.token[s], &tm_token, bar, kc * kStageK, row);
                        tma_load_2d_pair(sm.token[s] + half * 128, &tm_token, bar, kc * kStageK + 64, row);
                    }
                }
                // the copies have landed and the last commits have arrived; after an abort, when some
                // never will, what is still under way has one more limit's time to land
                for (int64_t i = j > SX ? j - SX : 0; i < j; ++i)
                    if (!mbar_wait(&sm.empty[i % SX], (i / SX) & 1, kWaitTimeoutNs)) {
                        if (!*reinterpret_cast<volatile int *>(&sm.abort_flag)) set_err(p.err, LHS_ERRBIT_TIMEOUT);
                        break;
                    }
            }
        } else if (warp == kConvWarps + 2) {
            // ---------------- MMA issuer (the leader CTA only) ----------------
            pdl_wait();
            const int chunk = blocks_per_sum(p, lane);
            if (rank == 0) {
                const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(p.n >> 3) << 17) |
                                       (static_cast<uint32_t>(kPairRows >> 4) << 24);  // f16 x f16 -> f32
                const uint32_t half16 = static_cast<uint32_t>(p.n / 2) * 128 >> 4;  // half a stage, in descriptor units
                const uint32_t tm = __reduce_or_sync(0xFFFFFFFFu, tmem);
                const uint32_t elected = elect_one();
                Ring<SX> sx;
                Ring<ACCS> sc;
                bool ok = true, ready = false;
                for (int64_t it = 0; it < mine && ok; ++it) {
                    int in = 0;  // stages of the current sum
                    for (int kc = 0; kc < p.nk; ++kc) {
                        bool go = true;
                        if (in == 0) go = wait_or_abort(&sm.acc_empty[sc.i], sc.parity ^ 1u, &sm.abort_flag, p.err);
                        if (!ready) go = go && wait_or_abort(&sm.full[sx.i], sx.parity, &sm.abort_flag, p.err);
                        if (!__all_sync(0xFFFFFFFFu, go)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d = tm + sc.i * NMAX, a = tm + T::kColA + sx.i * kSlotCols;
                        const uint32_t b = desc_lo(smem_u32(sm.token[sx.i]));
                        uint64_t *done = &sm.empty[sx.i];
                        sx.next();
                        // a look at the next stage, whose answer the MMAs' issue hides
                        ready = mbar_test_cluster(&sm.full[sx.i], sx.parity);
#pragma unroll
                        for (int ks = 0; ks < kStageK / 16; ++ks)
                            umma_f16_ts(elected, d, a + ks * 8, b + (ks >> 2) * half16 + (ks & 3) * 2, idesc, (in | ks) != 0);
                        umma_commit_both(elected, done);
                        ready = __all_sync(0xFFFFFFFFu, ready);
                        ++in;
                        if (in == chunk || kc + 1 == p.nk) {
                            umma_commit_both(elected, &sm.acc_full[sc.i]);
                            in = 0;
                            sc.next();
                        }
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // the pair is done with its accumulators and barriers
    if (warp == kConvWarps + 2) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
    cluster_sync_all();  // neither CTA leaves while its peer may still address it
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
template <int NMAX>
cudaError_t launch_product(const CUtensorMap &tm_table, const CUtensorMap &tm_token, const Params &p,
                           const DeviceInfo &dev, cudaStream_t stream) {
    constexpr int smem = 1024 + static_cast<int>(sizeof(Smem<NMAX>));
    auto kern = i8_matmul_kernel<NMAX>;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(Tile<NMAX>::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    static std::mutex mu;
    static int pairs[64] = {};  // resident at once
    int fit;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!pairs[dev.device]) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            int n = dev.num_sms / 2, active = 0;
            cfg.gridDim = dim3(2 * n);
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&active, kern, &cfg) == cudaSuccess && active > 0 && active < n) n = active;
            (void)cudaGetLastError();
            pairs[dev.device] = n < 1 ? 1 : n;
        }
        fit = pairs[dev.device];
    }
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (p.items < fit ? p.items : fit)));
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, tm_table, tm_token, p);
}

template <int DT>
cudaError_t prep_wide(const I8Tokens &a, int hidden, const Layout &l, uint8_t *ws, int32_t *err, unsigned grid,
                      cudaStream_t stream) {
    constexpr int64_t size = DT == LHS_F32 ? 4 : 2;
    const bool vec = reinterpret_cast<uintptr_t>(a.x) % (4 * size) == 0 && a.x_stride % 4 == 0;
    return launch_pdl(i8_prep_wide_kernel<DT>, dim3(grid), dim3(kPrepThreads), 0, stream,
                      static_cast<const typename Elem<DT>::T *>(a.x), a.x_stride, vec, a.rows, hidden, l.kpad,
                      reinterpret_cast<__half *>(ws), reinterpret_cast<float *>(ws + l.scales),
                      reinterpret_cast<int32_t *>(ws + l.peaks), err);
}

}  // namespace

size_t i8_matmul_workspace(const lhs_i8 &table, int64_t tokens) {
    return static_cast<size_t>(layout_of(table.hidden, tokens).bytes);
}

cudaError_t launch_i8_matmul(const I8Tokens &a, const lhs_i8 &table, void *out, int32_t out_dtype,
                             int64_t out_stride, void *ws_, int32_t *err, cudaStream_t stream) {
    DeviceInfo dev;
    cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    if (i8_gemv_serves(table, a.rows)) return launch_i8_gemv(a, table, out, out_dtype, out_stride, err, dev, stream);
    uint8_t *ws = static_cast<uint8_t *>(ws_);
    const Layout l = layout_of(table.hidden, a.rows);

    Params p = {};
    p.w_scales = reinterpret_cast<const uint8_t *>(table.scales);
    p.w_scale_stride = table.scale_stride;
    p.channels = table.rows;
    p.tokens = a.rows;
    // token blocks of equal size, at most 256 tokens each
    p.blocks = static_cast<int>((a.rows + 255) / 256);
    p.n = static_cast<int>(align_up((a.rows + p.blocks - 1) / p.blocks, 32));
    p.nk = l.kpad / kStageK;
    p.items = (table.rows + kPairRows - 1) / kPairRows * p.blocks;
    p.scales = reinterpret_cast<const float *>(ws + l.scales);
    p.peaks = reinterpret_cast<const int32_t *>(ws + l.peaks);
    p.out = out;
    p.out_stride = out_stride;
    p.out_dtype = out_dtype;
    p.err = err;
    CUtensorMap tm_table, tm_token;
    if (!make_map(&tm_table, CU_TENSOR_MAP_DATA_TYPE_UINT8, table.codes, table.hidden, table.rows, table.stride,
                  kStageK, kCtaRows) ||
        !make_map(&tm_token, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ws, l.kpad, a.rows, static_cast<uint64_t>(l.kpad) * 2, 64,
                  p.n / 2))
        return cudaErrorInvalidValue;

    const unsigned pg = static_cast<unsigned>(a.rows < (1 << 20) ? a.rows : (1 << 20));
    if (!a.x) {
        const bool words = reinterpret_cast<uintptr_t>(a.coded.codes) % 4 == 0 && a.coded.stride % 4 == 0;
        e = launch_pdl(i8_prep_coded_kernel, dim3(pg), dim3(kPrepThreads), 0, stream, a.coded, words, l.kpad,
                       reinterpret_cast<__half *>(ws), reinterpret_cast<float *>(ws + l.scales),
                       reinterpret_cast<int32_t *>(ws + l.peaks), err);
    } else if (a.x_dtype == LHS_F32) {
        e = prep_wide<LHS_F32>(a, table.hidden, l, ws, err, pg, stream);
    } else if (a.x_dtype == LHS_F16) {
        e = prep_wide<LHS_F16>(a, table.hidden, l, ws, err, pg, stream);
    } else {
        e = prep_wide<LHS_BF16>(a, table.hidden, l, ws, err, pg, stream);
    }
    if (e != cudaSuccess) return e;
    if (p.n <= 32) return launch_product<32>(tm_table, tm_token, p, dev, stream);
    if (p.n <= 64) return launch_product<64>(tm_table, tm_token, p, dev, stream);
    if (p.n <= 128) return launch_product<128>(tm_table, tm_token, p, dev, stream);
    return launch_product<256>(tm_table, tm_token, p, dev, stream);
}

}  // namespace lhs
