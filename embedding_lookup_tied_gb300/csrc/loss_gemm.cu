// loss_gemm.cu — the products of the cross entropy and of its gradient, on the
// 5th-generation tensor cores (tcgen05 + TMEM).
//
// Four products share one kernel.  With X the packed residuals, W the table and
// g a piece of the logits' gradient ([tokens x rows of the piece]):
//   logits   z  = X W^T   M = tokens,  N = rows,   K = hidden   (statistics, or g)
//   dx      += g W        M = tokens,  N = hidden, K = rows of the piece
//   dtable   = g^T X      M = rows,    N = hidden, K = tokens
// A pair of CTAs owns a tile of 256 x up to 256 (cta_group::2): each stages its
// own 128 rows of A and half of B's columns, 64 of k at a time, by TMA with
// 128-byte swizzle, and receives the f32 sums of its rows in its TMEM, which
// holds two tiles, so that the next one's MMAs run while one is taken out.
// Operands whose k is not the contiguous index (W for dx, both for dtable) are
// staged as they lie and read "MN-major": no transposed copy is made.
//
// The gradient goes through the vocabulary in pieces, in one launch: the logits
// of a few pieces run ahead of their products.  (A launch for each piece left a
// tail of idle pairs at its end: 4.63 ms at 8,192 x 151,936 x 896 in pieces of 4,096
// rows.)  Items (tiles) come from one queue, in an order in which an
// item waits only for items before it: g for the products that read the slot
// which it overwrites, the products for the piece's g, and the sums of dx for the
// piece before (so that they are added up in order).  Pairs take items as they
// run, so what is waited for is always with a pair that runs, however many do.
// dx's tiles are few and their k is long, so they are split along k; each split
// adds up in f32 sums of its own, which one kernel joins in order at the end.
//
// The logits are never stored: statistics leave a tile as (maximum, sum of the
// other exponentials) of each token, g as 16-bit values that the products read
// back from L2 or HBM; of up to 128 tokens in two terms, the second in the rows of the
// tile's other half, with the residuals there too, so that both products add them up.
// Of more positions the targets' entries are kept apart in f32 (loss_queue.cuh): g holds what a
// logit of the tensor cores makes of one beyond that, and a tile of dtable adds the sums of
// its targets' rows before it rounds.
//
// What bounds it.  Many tokens: the tensor cores and the power cap.  8,192 x
// 151,936 x 896: statistics 1.21 ms (1,840 TFLOP/s; 1,660 for seconds on end),
// gradient 3.95 to 4.2 ms with its small kernels (1,590 to 1,690; 1,496 for seconds on end, where
// a library product of the same shape does 1,636); 2,048 x 262,144 x 5,376: 3.05 ms
// (1,890).  256 x 262,144 x 5,120: 1.56 ms for 1.18 at the sustained rate; the
// table is read twice and its gradient written, 1.2 ms of HBM.  One token, 151,936 x
// 896: statistics 49 us, 5.6 TB/s; gradient 196 us for 80: reading the table twice,
// and taking 2,376 tiles of its gradient out.
#include <mutex>
#include <type_traits>

#include "i8_common.cuh"
#include "train.cuh"

namespace lhs {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kCtaM = 128;                    // rows of a tile that a CTA holds (TMEM lanes)
constexpr int kBoxBytes = 64 * 64 * 2;        // what one TMA load brings: 64 x 64 values
constexpr int kOperandBytes = 2 * kBoxBytes;  // a CTA's part of A, or of B, of a stage
constexpr int kTmemCols = 512;
constexpr int kStoreBytes = 32 * 128;         // an epilogue warp's store: 32 rows of 128 bytes
constexpr int kQueue = 3;                     // items handed out ahead

enum { kStore16 = 0, kStore32 = 1, kAdd32 = 2, kPlain = 3 };  // how dtable is written

struct Params : LossShape {
    const LossMeta *meta;
    const int32_t *tgt;
    float l2;                // log2(e) / temperature
    uint32_t *queue;         // items handed out; 0 at the start
    int32_t *err;
    float2 *stats;           // statistics
    float *zt;
    float inv_t;             // 1 / temperature
    const float *lse, *gs;   // g
    const float *em;         // the targets' p - 1, or null
    const float *coef;       // what is kept apart of the targets' entries, or null
    const int32_t *slot_of;  // dtable: [V] rows of what it makes there, [tiles] whether there is one; or null
    const float *rows;
    int64_t rows_pitch;
    uint32_t *g_done;        // [pieces] warps that have written a tile of g
    uint32_t *read_done;     // [pieces] products that have read it
    uint32_t *dx_done;       // [tiles of dx x splits x kLossSyncWarps] pieces added up
    int dt_mode, dt_dtype;
    bool accumulate;
    void *dtable;
};

template <int MODE>
struct Conf {
    static constexpr bool kGrad = MODE == 1;
    static constexpr int kStages = kGrad ? 6 : 7;
    // Two warps to each quarter of TMEM's lanes take a tile out: half of its columns each for the
    // statistics, 64 in turn for the gradient's products.
    static constexpr int kEpiWarps = 8;
    static constexpr int kFirstEpi = 4;  // after the producer, the MMA issuer, the scheduler and an idle one
    static constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
    static constexpr int kOutBuffers = 1;
};


template <int MODE>
struct Smem {
    static constexpr int S = Conf<MODE>::kStages;
    uint8_t a[S][kOperandBytes];
    uint8_t b[S][kOperandBytes];
    uint8_t out[Conf<MODE>::kGrad ? Conf<MODE>::kEpiWarps : 1][Conf<MODE>::kOutBuffers][Conf<MODE>::kGrad ? kStoreBytes : 16];
    uint64_t full[S], empty[S];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t item_full[kQueue], item_empty[kQueue];
    Item item[kQueue];
    uint32_t tmem_base;
    int abort_flag;
};

// ---------------------------------------------------------------------------
// instructions
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The shared::cluster address of a variable of CTA `cta` of the pair.
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t cta) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(cta));
    return r;
}
// TMA load into this CTA's shared memory, counted on a barrier of either CTA.
__device__ __forceinline__ void tma_load_pair(void *dst, const CUtensorMap *map, uint32_t bar, int32_t c0, int32_t c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap *map, const void *src, int32_t c0, int32_t c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void tma_add(const CUtensorMap *map, const void *src, int32_t c0, int32_t c1) {
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Arrive on a barrier of either CTA for what tcgen05 waits and fences order.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait(uint64_t *bar, uint32_t parity) {
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
// Whether the phase is over, without a wait.
__device__ __forceinline__ bool test_wait(uint64_t *bar, uint32_t parity) {
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
    if (try_wait(bar, parity)) return true;
    if (*reinterpret_cast<const volatile int *>(abort_flag)) return false;
    const uint64_t t0 = global_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (try_wait(bar, parity)) return true;
        if (global_ns() - t0 > kWaitTimeoutNs) break;
    }
    set_err(err, LHS_ERRBIT_TIMEOUT);
    *reinterpret_cast<volatile int *>(abort_flag) = 1;
    return false;
}
// Counters in global memory that CTAs tell one another by.
__device__ __forceinline__ void add_release(uint32_t *p, uint32_t v) {
    asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void add_relaxed(uint32_t *p, uint32_t v) {
    asm volatile("red.relaxed.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t load_acquire(const uint32_t *p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
// What TMA reads or writes next comes after what this thread has acquired.
__device__ __forceinline__ void fence_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }
// Bounded wait of one thread until *p reaches `target`.
__device__ __forceinline__ bool wait_count(const uint32_t *p, uint32_t target, int *abort_flag, int32_t *err) {
    if (load_acquire(p) < target) {
        const uint64_t t0 = global_ns();
        while (load_acquire(p) < target) {
            if (*reinterpret_cast<const volatile int *>(abort_flag)) return false;
            if (global_ns() - t0 > kWaitTimeoutNs) {
                set_err(err, LHS_ERRBIT_TIMEOUT);
                *reinterpret_cast<volatile int *>(abort_flag) = 1;
                return false;
            }
            __nanosleep(64);
        }
    }
    fence_async_global();
    return true;
}
// One lane of the warp for the MMAs: the whole warp runs the loop around them,
// so that their operands stay in uniform registers.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p)::"memory");
    return p;
}
// Shared-memory matrix descriptors, 128-byte swizzle.  High word: groups of 8
// rows 1024 bytes apart (SBO).  Low word: address, and for an MN-major operand
// the distance of its second 64 columns, one box further on (LBO).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kLboK = 1u << 16, kLboMn = static_cast<uint32_t>(kBoxBytes >> 4) << 16;
// 16 of k further on: 32 bytes along the rows, or 16 rows of 128 bytes
constexpr uint32_t kStepK = 32 >> 4, kStepMn = 2048 >> 4;
__device__ __forceinline__ void umma(uint32_t elected, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                     uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(elected), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void commit_both(uint32_t elected, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::
            "r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(0x3)), "r"(elected)
        : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 32 consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// Twice 32 columns: both loads are under way before the first is waited for.
__device__ __forceinline__ void tmem_ld64(uint32_t lo, uint32_t hi, float (&v)[64]) {
    const uint32_t taddr[2] = {lo, hi};
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
#pragma unroll
    for (int o = 0; o < 2; ++o)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
            "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
            : "=r"(r[32 * o + 0]), "=r"(r[32 * o + 1]), "=r"(r[32 * o + 2]), "=r"(r[32 * o + 3]), "=r"(r[32 * o + 4]),
              "=r"(r[32 * o + 5]), "=r"(r[32 * o + 6]), "=r"(r[32 * o + 7]), "=r"(r[32 * o + 8]), "=r"(r[32 * o + 9]),
              "=r"(r[32 * o + 10]), "=r"(r[32 * o + 11]), "=r"(r[32 * o + 12]), "=r"(r[32 * o + 13]),
              "=r"(r[32 * o + 14]), "=r"(r[32 * o + 15]), "=r"(r[32 * o + 16]), "=r"(r[32 * o + 17]),
              "=r"(r[32 * o + 18]), "=r"(r[32 * o + 19]), "=r"(r[32 * o + 20]), "=r"(r[32 * o + 21]),
              "=r"(r[32 * o + 22]), "=r"(r[32 * o + 23]), "=r"(r[32 * o + 24]), "=r"(r[32 * o + 25]),
              "=r"(r[32 * o + 26]), "=r"(r[32 * o + 27]), "=r"(r[32 * o + 28]), "=r"(r[32 * o + 29]),
              "=r"(r[32 * o + 30]), "=r"(r[32 * o + 31])
            : "r"(taddr[o])
            : "memory");
    // the values are not there before this; nothing that uses them moves above it
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 64; ++i) asm volatile("" : "+r"(r[i]));
}
// 2^x, relative error below 2^-21: a thousandth of what g is rounded by, and of the order of an
// f32 logit's own rounding in a sum of exponentials.  Results below 2^-126 (of the row's largest, or
// as a probability) are 0: one instruction instead of several.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool BF>
__device__ __forceinline__ float round16(float x) {
    return BF ? __bfloat162float(__float2bfloat16_rn(x)) : __half2float(__float2half_rn(x));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if (BF) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// 16-byte piece i of row r of a store's 128-byte rows, swizzled.
__device__ __forceinline__ void put_piece(uint8_t *buf, int r, int i, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    *reinterpret_cast<uint4 *>(buf + r * 128 + ((i ^ (r & 7)) << 4)) = make_uint4(x, y, z, w);
}

// ---------------------------------------------------------------------------
// kernel
// ---------------------------------------------------------------------------
template <int MODE, bool BF>
__global__ void __launch_bounds__(Conf<MODE>::kThreads, 1)
    loss_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                const __grid_constant__ CUtensorMap tm_g, const __grid_constant__ CUtensorMap tm_g_out,
                const __grid_constant__ CUtensorMap tm_part, const __grid_constant__ CUtensorMap tm_dt, const Params p) {
    constexpr int S = Conf<MODE>::kStages, kEpiWarps = Conf<MODE>::kEpiWarps, kFirstEpi = Conf<MODE>::kFirstEpi,
                  kOutBuffers = Conf<MODE>::kOutBuffers;
    extern __shared__ uint8_t dyn_smem[];
    Smem<MODE> &sm = *reinterpret_cast<Smem<MODE> *>(smem_align<1024>(dyn_smem));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&sm.full[s], 1);   // leader: its producer's expect_tx; both CTAs' bytes
            mbar_init(&sm.empty[s], 1);  // the leader's commit, to both
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.acc_full[i], 1);
            mbar_init(&sm.acc_empty[i], 2 * kEpiWarps);
        }
        for (int i = 0; i < kQueue; ++i) {
            mbar_init(&sm.item_full[i], 1);
            mbar_init(&sm.item_empty[i], 2 + 1 + 2 * kEpiWarps);  // leader: producers, MMA issuer, epilogues
        }
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {  // with the peer's warp 1
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_sync_all();  // the peer's barriers exist
    const uint32_t tmem = sm.tmem_base;
    pdl_wait();
    const Work work = work_of<MODE>(p, ld_dep(&p.meta->count));

    // The next item, for one role (a warp, or the producer's lane); kind -1 at the end or after an abort.
    int slot = 0;
    uint32_t slot_parity = 0;
    auto next_item = [&](bool whole_warp) -> Item {
        Item t;
        t.kind = -1;
        const bool ok = wait_or_abort(&sm.item_full[slot], slot_parity, &sm.abort_flag, p.err);
        if (whole_warp ? !__all_sync(0xFFFFFFFFu, ok) : !ok) return t;
        t = sm.item[slot];
        // One lane hands the slot back, after every lane has read it: the vote needs a word of each of
        // the item's two loads from all of them (both conditions always hold), and what follows it is
        // ordered behind their reads.  (A release at cluster scope would wait for all memory, 0.5 us of
        // every item.)
        bool read = t.kind >= -1 && t.width <= kLossTile;
        if (whole_warp) {
            read = __all_sync(0xFFFFFFFFu, read);
            __syncwarp();
        }
        if ((!whole_warp || lane == 0) && read) arrive_cluster(cluster_addr(&sm.item_empty[slot], 0));
        if (++slot == kQueue) {
            slot = 0;
            slot_parity ^= 1u;
        }
        return t;
    };

    // The warps that hold sums take registers from the others: 8 x 224 + 4 x 56 a lane are what 12 warps
    // are launched with at 168.
    if (warp < kFirstEpi) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {
            // ---------------- TMA producer ----------------
            if (lane == 0) {
                uint32_t j = 0;  // stages issued
                bool ok = true;
                int seen = -1;   // the last piece whose g is known to be complete
                const int r = static_cast<int>(rank);
                for (;;) {
                    const Item t = next_item(false);
                    if (t.kind < 0) break;
                    const int half = t.width / 2, b_boxes = half > 64 ? 2 : 1;
                    // first coordinates of A and B: (x, y) of the box at stage 0, whether k runs along x,
                    // and the second box's offset
                    const CUtensorMap *ma, *mb;
                    int ax, ay, bx, by;
                    bool ak, bk;
                    if (MODE == 0 || t.kind == kLogits) {
                        ma = &tm_x, ax = 0, ay = t.m * kLossTile + r * kCtaM, ak = true;
                        mb = &tm_w, bx = 0, by = t.piece * static_cast<int>(p.piece) + t.n * kLossTile + r * half, bk = true;
                    } else {
                        if (t.piece > seen) {  // all of the piece's g
                            if (!wait_count(p.g_done + t.piece, work.blocks * tiles_of(p, t.piece) * kLossSyncWarps,
                                            &sm.abort_flag, p.err))
                                break;
                            seen = t.piece;
                        }
                        const int g0 = t.piece % p.slots * static_cast<int>(p.Tpad);
                        if (t.kind == kDx) {
                            ma = &tm_g, ax = 0, ay = g0 + t.m * kLossTile + r * kCtaM, ak = true;
                            mb = &tm_w, bx = t.n * kLossTile + r * half, by = t.piece * static_cast<int>(p.piece), bk = false;
                        } else {
                            ma = &tm_g, ax = t.m * kLossTile + r * kCtaM, ay = g0, ak = false;
                            mb = &tm_x, bx = t.n * kLossTile + r * half, by = 0, bk = false;
                        }
                    }
                    for (int kc = t.k0; kc < t.k1; ++kc, ++j) {
                        const int s = j % S;
                        if (j >= S && !wait_or_abort(&sm.empty[s], ((j / S) & 1) ^ 1, &sm.abort_flag, p.err)) {
                            ok = false;
                            break;
                        }
                        if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * (2 + b_boxes) * kBoxBytes);
                        const uint32_t bar = cluster_addr(&sm.full[s], 0);
                        const int k = kc * kTileK + (MODE == 1 && t.kind == kDtable && kc >= work.turn ? work.gap : 0);
                        const int axk = ak ? ax + k : ax, ayk = ak ? ay : ay + k;
                        tma_load_pair(sm.a[s], ma, bar, axk, ayk);
                        tma_load_pair(sm.a[s] + kBoxBytes, ma, bar, ak ? axk : axk + 64, ak ? ayk + 64 : ayk);
                        const int bxk = bk ? bx + k : bx, byk = bk ? by : by + k;
                        tma_load_pair(sm.b[s], mb, bar, bxk, byk);
                        if (b_boxes == 2)
                            tma_load_pair(sm.b[s] + kBoxBytes, mb, bar, bk ? bxk : bxk + 64, bk ? byk + 64 : byk);
                    }
                    if (!ok) break;
                }
                // drain: the pair has consumed every stage issued, so no copy, completion or commit is still
                // headed for either CTA (after an abort, when some never come, one more limit's time to land)
                for (uint32_t i = j > static_cast<uint32_t>(S) ? j - S : 0; i < j; ++i)
                    if (!mbar_wait(&sm.empty[i % S], (i / S) & 1, kWaitTimeoutNs)) {
                        if (!*reinterpret_cast<volatile int *>(&sm.abort_flag)) set_err(p.err, LHS_ERRBIT_TIMEOUT);
                        break;
                    }
            }
        } else if (warp == 1) {
            // ---------------- MMA issuer (the leader CTA only) ----------------
            if (rank == 0) {
                const uint32_t tm = __reduce_or_sync(0xFFFFFFFFu, tmem);
                const uint32_t elected = elect_one();
                uint32_t j = 0;
                int n_acc = 0;
                for (;;) {
                    const Item t = next_item(true);
                    if (t.kind < 0) break;
                    const bool a_mn = MODE == 1 && t.kind == kDtable, b_mn = MODE == 1 && t.kind != kLogits;
                    const uint32_t idesc = (1u << 4) | (BF ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) |
                                           (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(t.width >> 3) << 17) |
                                           (static_cast<uint32_t>((2 * kCtaM) >> 4) << 24);
                    const uint32_t la = a_mn ? kLboMn : kLboK, lb = b_mn ? kLboMn : kLboK;
                    const uint32_t sa = a_mn ? kStepMn : kStepK, sb = b_mn ? kStepMn : kStepK;
                    const int chunk = chunk_of<MODE>(t.kind);
                    bool ok = true;
                    for (int k0 = t.k0; k0 < t.k1 && ok; k0 += chunk) {
                        const int buf = n_acc & 1, k1 = k0 + chunk < t.k1 ? k0 + chunk : t.k1;
                        ok = wait_or_abort(&sm.acc_empty[buf], ((n_acc >> 1) & 1) ^ 1, &sm.abort_flag, p.err);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t d = tm + buf * (kTmemCols / 2);
                        for (int kc = k0; kc < k1; ++kc, ++j) {
                            const int s = j % S;
                            ok = wait_or_abort(&sm.full[s], (j / S) & 1, &sm.abort_flag, p.err);
                            ok = __all_sync(0xFFFFFFFFu, ok);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t a = ((smem_u32(sm.a[s]) >> 4) & 0x3FFFu) | la, b = ((smem_u32(sm.b[s]) >> 4) & 0x3FFFu) | lb;
#pragma unroll
                            for (int ks = 0; ks < kTileK / 16; ++ks)
                                umma(elected, d, a + ks * sa, b + ks * sb, idesc, kc != k0 || ks != 0);
                            commit_both(elected, &sm.empty[s]);
                        }
                        if (!ok) break;
                        commit_both(elected, &sm.acc_full[buf]);
                        ++n_acc;
                    }
                    if (!ok) break;
                }
            }
        } else if (warp == 2) {
            // ---------------- scheduler (the leader CTA only) ----------------
            if (rank == 0 && lane == 0) {
                Work w = work;
                set_divisors<MODE>(p, w);
                int q = 0;
                uint32_t parity = 1;
                uint32_t i = atomicAdd(p.queue, 1u);
                for (;;) {
                    Item t = {};
                    t.kind = -1;
                    uint32_t next = 0;
                    if (i < w.total) {
                        next = atomicAdd(p.queue, 1u);  // on its way while this one is worked out
                        t = item_of<MODE>(p, w, i);
                        // (asked here, items ahead: a warp that takes tiles out would wait for the answer,
                        // 256 x 262,144 x 5,120 1.48 -> 1.63 ms)
                        if (MODE == 1 && t.kind == kDtable && p.slot_of)
                            t.split = ld_dep(p.slot_of + p.V + t.piece * p.piece_tiles + t.m) >= 0;
                    }
                    if (!wait_or_abort(&sm.item_empty[q], parity, &sm.abort_flag, p.err)) break;
                    const int4 *v = reinterpret_cast<const int4 *>(&t);
#pragma unroll
                    for (uint32_t cta = 0; cta < 2; ++cta) {  // the words' arrival completes the phase
                        const uint32_t bar = cluster_addr(&sm.item_full[q], cta), dst = cluster_addr(&sm.item[q], cta);
                        asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar),
                                     "r"(static_cast<uint32_t>(sizeof(Item)))
                                     : "memory");
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            asm volatile(
                                "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                                    dst + 16 * h),
                                "r"(v[h].x), "r"(v[h].y), "r"(v[h].z), "r"(v[h].w), "r"(bar)
                                : "memory");
                    }
                    if (t.kind < 0) break;
                    i = next;
                    if (++q == kQueue) {
                        q = 0;
                        parity ^= 1u;
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        // ---------------- epilogue ----------------
        const int q = warp & 3, part = (warp - kFirstEpi) / 4;  // TMEM lane quarter; of the warps that share it
        constexpr int kParts = kEpiWarps / 4;
        const int row = static_cast<int>(rank) * kCtaM + q * 32 + lane;  // of the tile
        const int row0 = static_cast<int>(rank) * kCtaM + q * 32;
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        const float scale = MODE == 1 ? ld_dep(&p.meta->scale) : 1.0f, unscale = MODE == 1 ? ld_dep(&p.meta->unscale) : 1.0f;
        // the second CTA's rows hold what the rounding of the first one's left (see kLossTwin)
        const bool rest = MODE == 1 && rank == 1 && ld_dep(&p.meta->count) <= kLossTwin;
        int n_acc = 0, n_out = 0, free_seen = -1;
        uint32_t *told = nullptr;  // lane 0: whom to tell of the stores so far
        auto tell = [&]() {
            if (told) {
                bulk_wait_all();  // written, for whoever acquires it
                add_release(told, 1u);
                told = nullptr;
            }
        };
        // This warp has read an accumulator.
        auto release = [&](int buf) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(cluster_addr(&sm.acc_empty[buf], 0));
        };
        // A buffer of this warp's that no store reads any more.
        auto out_buffer = [&]() -> uint8_t * {
            if (lane == 0) bulk_wait_read<kOutBuffers - 1>();
            __syncwarp();
            return sm.out[MODE == 1 ? warp - kFirstEpi : 0][n_out % kOutBuffers];
        };
        auto send = [&](const CUtensorMap *map, const uint8_t *buf, int x, int y, bool add) {
            fence_async_shared();
            __syncwarp();
            if (lane == 0) {
                if (add) tma_add(map, buf, x, y);
                else tma_store(map, buf, x, y);
                bulk_commit();
            }
            ++n_out;
        };
        // Lane 0: a counter has reached `target`, at the latest after what this warp has to tell.
        auto after = [&](const uint32_t *count, uint32_t target) -> bool {
            if (load_acquire(count) < target) tell();
            return wait_count(count, target, &sm.abort_flag, p.err);
        };
        // 64 values of 16 bits of this lane's row, to (x, y).  The buffer is waited for when they are there.
        auto put_half = [&](const uint32_t (&w)[32], int x, int y, const CUtensorMap *map) {
            if (lane == 0) tell();
            uint8_t *out = out_buffer();
#pragma unroll
            for (int k = 0; k < 8; ++k) put_piece(out, lane, k, w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            send(map, out, x, y, false);
        };
        for (;;) {
            const Item t = next_item(true);
            if (t.kind < 0) break;
            int buf = n_acc & 1;
            // what the tile needs besides its sums, asked for before they are waited for
            int y = -1;
            bool none = false;  // a row past the last token
            float lse = 0.0f, gs = 0.0f, em = 0.0f, apart = 0.0f;
            int64_t v0 = 0;
            const int64_t tok = static_cast<int64_t>(t.m) * kLossTile + row;
            if (MODE == 0 || t.kind == kLogits) {
                v0 = t.piece * p.piece + static_cast<int64_t>(t.n) * kLossTile;
                const int target = ld_dep(p.tgt + tok);
                none = target < 0;
                y = target >= v0 && target < v0 + kLossTile ? static_cast<int>(target - v0) : -1;
                if (MODE == 1) {
                    lse = ld_dep(p.lse + tok);
                    gs = ld_dep(p.gs + tok) * scale;
                    if (p.em) em = ld_dep(p.em + tok);
                    if (p.coef) apart = ld_dep(p.coef + tok) * scale;
                }
            }
            int at = -1;  // where the row's sums of what is kept apart are
            if (MODE == 1 && t.kind == kDtable && t.split) {
                const int64_t v = t.piece * p.piece + static_cast<int64_t>(t.m) * kLossTile + row;
                if (v < p.V) at = ld_dep(p.slot_of + v);
            }
            // What was written and not yet told of is told of before anything is waited for that may
            // depend on it; where the tile is there already, after its first part, when the stores
            // have long completed.
            uint32_t *dx_done = nullptr;
            bool go = true;
            if (MODE == 1 && lane == 0) {
                if (t.kind == kLogits) {
                    // the slot is free once the products with the piece that was there have read it
                    const int old = t.piece - p.slots;
                    if (old > free_seen) {
                        go = after(p.read_done + old, n_products_of(p, work, old));
                        free_seen = old;
                    }
                } else if (t.kind == kDx) {
                    dx_done = p.dx_done + ((static_cast<int64_t>(t.m) * p.ht + t.n) * p.splits + t.split) * kLossSyncWarps +
                              rank * kEpiWarps + warp - kFirstEpi;
                    if (t.piece > 0) go = after(dx_done, t.piece);
                }
                if (told && !test_wait(&sm.acc_full[buf], (n_acc >> 1) & 1)) tell();
            }
            const bool ok = go && wait_or_abort(&sm.acc_full[buf], (n_acc >> 1) & 1, &sm.abort_flag, p.err);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;  // tcgen05.ld is warp-collective
            tc_fence_after();
            ++n_acc;
            if (MODE == 0) {
                // Statistics: the maximum m, the sum s of the exponentials below it and the number
                // of equals.  The maximum's own 1 is left out of the sum, so that a loss near 0 (the
                // target is the maximum, the rest small) keeps its relative accuracy.
                constexpr int kCols = kLossTile / kParts;
                float m = -INFINITY, s = 0.0f, z = 0.0f;
                int equal = 0;
                float sum[kCols];
                bool all = true;
                for (int k0 = t.k0;;) {
#pragma unroll
                    for (int c = 0; c < kCols; c += 32) {
                        float v[32];
                        tmem_ld32(tmem + lanes + buf * (kTmemCols / 2) + part * kCols + c, v);
#pragma unroll
                        for (int k = 0; k < 32; ++k) sum[c + k] = k0 == t.k0 ? v[k] : sum[c + k] + v[k];
                    }
                    release(buf);
                    k0 += kChunk;
                    if (k0 >= t.k1) break;
                    buf = n_acc & 1;
                    all = __all_sync(0xFFFFFFFFu, wait_or_abort(&sm.acc_full[buf], (n_acc >> 1) & 1, &sm.abort_flag, p.err));
                    if (!all) break;
                    tc_fence_after();
                    ++n_acc;
                }
                if (!all) break;
#pragma unroll
                for (int c = 0; c < kCols; c += 32) {
                    float *v = sum + c;
                    const int64_t left = p.V - v0 - part * kCols - c;
                    if (left <= 0) continue;
                    if (left < 32) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (k >= left) v[k] = -INFINITY;  // counted as equal only where nothing is above -inf
                    }
                    if (__any_sync(0xFFFFFFFFu, y >= 0 && (y >> 5) == (part * kCols + c) / 32)) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (y == part * kCols + c + k) z = v[k];
                    }
                    float top = m;
#pragma unroll
                    for (int k = 0; k < 32; ++k) top = fmaxf(top, v[k]);
                    if (top > m) {
                        s = m == -INFINITY ? s : (s + static_cast<float>(equal)) * ex2((m - top) * p.l2);
                        equal = 0;
                        m = top;
                    }
                    // (the difference first: m log2(e) by itself would be rounded to 2^-24 of itself, which is an
                    // error of all exponentials but the maximum's alike)
                    float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float e = ex2((v[k] - m) * p.l2);
                        if (v[k] == m) ++equal;
                        else s4[k & 3] += e;
                    }
                    s += (s4[0] + s4[1]) + (s4[2] + s4[3]);
                }
                p.stats[(static_cast<int64_t>(t.n) * kLossParts + part) * p.Tpad + tok] =
                    make_float2(m, m == -INFINITY ? s : s + static_cast<float>(equal - 1));
                if (y >= 0 && y / (kLossTile / kParts) == part) p.zt[tok] = z;
            } else {
                const int mode = t.kind == kLogits ? kStore16 : t.kind == kDtable ? p.dt_mode : t.piece == 0 ? kStore32 : kAdd32;
                const int left = p.H - t.n * kLossTile, cols = t.kind == kLogits || left > kLossTile ? kLossTile : left;
                // This warp's columns, 32 at a time, in their order: two stores of 64, or four of 32, in
                // turn with the other warp of its rows.  They are read at once, which hands the accumulator back
                // before they are worked on, 64 at a time by one copy of the code (two copies: 1 x 151,936 x 896
                // 196 -> 213 us; the second 64 read when the first are done: 201).
                static_assert(kParts == 2, "two warps to a row's columns");
                auto column = [&](int i) { return mode == kStore16 ? part * 64 + (i >> 1) * 128 + (i & 1) * 32 : part * 32 + i * 64; };
                auto load = [&](int b, float (&o)[64]) {
                    const uint32_t acc = tmem + lanes + buf * (kTmemCols / 2);
                    tmem_ld64(acc + column(2 * b), acc + column(2 * b + 1), o);
                };
                const int chunk = chunk_of<MODE>(t.kind);
                float v[64], next[64];
                load(0, v);
                load(1, next);
                release(buf);
                if (t.k1 - t.k0 > chunk) {
                    bool all = true;
                    for (int k0 = t.k0 + chunk; k0 < t.k1; k0 += chunk) {
                        // (the other warps, on whom the next sums wait too, may depend on what this one has to tell)
                        if (lane == 0) tell();
                        buf = n_acc & 1;
                        all = __all_sync(0xFFFFFFFFu, wait_or_abort(&sm.acc_full[buf], (n_acc >> 1) & 1, &sm.abort_flag, p.err));
                        if (!all) break;
                        tc_fence_after();
                        ++n_acc;
                        const uint32_t acc = tmem + lanes + buf * (kTmemCols / 2);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float more[32];
                            tmem_ld32(acc + column(i), more);
#pragma unroll
                            for (int k = 0; k < 32; ++k) (i < 2 ? v : next)[32 * (i & 1) + k] += more[k];
                        }
                        release(buf);
                    }
                    if (!all) break;
                }
                // what the blocks share: the target's entry; the place of a row of sums
                const bool nothing = __all_sync(0xFFFFFFFFu, none);  // (few tokens: three quarters of the warps)
                const bool dx = t.kind == kDx;
                const float u = dx ? 1.0f : unscale;
                const int h0 = t.n * kLossTile;
                // (a piece starts at a multiple of the tile, and rows past the table's end are not stored)
                const int64_t out_row = dx ? t.split * p.Tpad + static_cast<int64_t>(t.m) * kLossTile + row0
                                           : t.piece * p.piece + static_cast<int64_t>(t.m) * kLossTile + row0;
                const bool any = __any_sync(0xFFFFFFFFu, at >= 0);
                const float *targets = at >= 0 ? p.rows + at * p.rows_pitch + h0 : nullptr;
#pragma unroll 1
                for (int b = 0; b < 2; ++b) {
                    if (b == 1) {
#pragma unroll
                        for (int k = 0; k < 64; ++k) v[k] = next[k];
                    }
                    const int c = column(2 * b);
                    if (t.kind == kLogits) {
                        // g
                        const int64_t left = p.V - v0 - c;
                        const bool mine = y >= 0 && (y >> 6) == c / 64;
                        const bool special = left < 64 || __any_sync(0xFFFFFFFFu, none || mine);
                        uint32_t w[32];
                        if (nothing) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) w[k] = 0u;
                        } else {
                            float entry = 0.0f;  // the target's
                            if (__any_sync(0xFFFFFFFFu, mine)) {
                                float e = em;
                                if (!p.em) {
                                    float z = 0.0f;
#pragma unroll
                                    for (int k = 0; k < 64; ++k)
                                        if (y == c + k) z = v[k];
                                    const float l = fmaf(z, p.inv_t, -lse);
                                    e = p_minus_1(l, ex2(l * kLog2e));
                                }
                                entry = e * gs - apart;
                            }
                            // (the logarithm of the probability before it is scaled to base 2: lse times
                            // log2(e) would be rounded to 2^-24 of itself, which is an error of all of a row's
                            // probabilities alike)
#pragma unroll
                            for (int k = 0; k < 64; ++k) v[k] = ex2(fmaf(v[k], p.inv_t, -lse) * kLog2e) * gs;
                            if (special) {
#pragma unroll
                                for (int k = 0; k < 64; ++k) {
                                    if (y == c + k) v[k] = entry;
                                    if (none || k >= left) v[k] = 0.0f;
                                }
                            }
                            if (rest) {
#pragma unroll
                                for (int k = 0; k < 64; ++k) v[k] -= round16<BF>(v[k]);
                            }
#pragma unroll
                            for (int k = 0; k < 32; ++k) w[k] = pack16<BF>(v[2 * k], v[2 * k + 1]);
                        }
                        put_half(w, t.n * kLossTile + c, t.piece % p.slots * static_cast<int>(p.Tpad) + t.m * kLossTile + row0,
                                 &tm_g_out);
                        continue;
                    }
                    // sums of dx, or of dtable times the inverse of g's scale, and what is kept apart of this row's
                    if (any) {
#pragma unroll
                        for (int k = 0; k < 64; k += 4) {
                            float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            const int at_c = column(2 * b + k / 32) + k % 32;
                            if (targets && at_c < cols) a = ld_dep(reinterpret_cast<const float4 *>(targets + at_c));
                            v[k] = fmaf(v[k], u, a.x), v[k + 1] = fmaf(v[k + 1], u, a.y);
                            v[k + 2] = fmaf(v[k + 2], u, a.z), v[k + 3] = fmaf(v[k + 3], u, a.w);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 64; ++k) v[k] *= u;
                    }
                    if (mode == kStore16) {
                        if (c >= cols) continue;
                        uint32_t w[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) w[k] = pack16<BF>(v[2 * k], v[2 * k + 1]);
                        put_half(w, h0 + c, static_cast<int>(out_row), &tm_dt);
                        continue;
                    }
#pragma unroll 1
                    for (int i = 0; i < 2; ++i) {
                        const int c = column(2 * b + i);
                        if (c >= cols) break;
                        if (lane == 0) tell();
                        uint8_t *out = out_buffer();
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            if (s != i) continue;
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                put_piece(out, lane, k, __float_as_uint(v[32 * s + 4 * k]), __float_as_uint(v[32 * s + 4 * k + 1]),
                                          __float_as_uint(v[32 * s + 4 * k + 2]), __float_as_uint(v[32 * s + 4 * k + 3]));
                        }
                        if (mode != kPlain) {
                            send(dx ? &tm_part : &tm_dt, out, h0 + c, static_cast<int>(out_row), mode == kAdd32);
                            continue;
                        }
                        // a lane to a column: rows that TMA does not take, or sums in 16 bits
                        __syncwarp();
                        // (eight rows' loads under way at a time: 64 x 100,000 x 1,001 277 -> 199 us)
                        auto emit = [&](auto *dt) {
                            using O = std::remove_pointer_t<decltype(dt)>;
                            const bool in = c + lane < cols;
                            dt += out_row * p.H + h0 + c + lane;
                            for (int r0 = 0; r0 < 32; r0 += 8) {
                                O old[8];
                                if (p.accumulate) {
#pragma unroll
                                    for (int k = 0; k < 8; ++k)
                                        if (in && out_row + r0 + k < p.V) old[k] = dt[static_cast<int64_t>(r0 + k) * p.H];
                                }
                                float s[8];
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    s[k] = *reinterpret_cast<const float *>(out + (r0 + k) * 128 + (((lane >> 2) ^ k) << 4) + (lane & 3) * 4);
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    if (in && out_row + r0 + k < p.V)
                                        put_rn(dt + static_cast<int64_t>(r0 + k) * p.H, p.accumulate ? wide(old[k]) + s[k] : s[k]);
                            }
                        };
                        if (p.dt_dtype == LHS_F32) emit(static_cast<float *>(p.dtable));
                        else if (BF) emit(static_cast<__nv_bfloat16 *>(p.dtable));
                        else emit(static_cast<__half *>(p.dtable));
                        __syncwarp();
                    }
                }
            }
            if (MODE == 1 && lane == 0) {
                tell();  // (a warp without columns in this tile has not yet)
                if (t.kind == kLogits) told = p.g_done + t.piece;
                else if (t.kind == kDx) told = dx_done;
                // Both CTAs' MMAs are done, and with them their reads of g: the copies' bytes were counted
                // on the barrier that the MMAs waited for, and the MMAs on the one that this thread has.
                // What the counter has to keep apart is those reads and the stores of whoever overwrites
                // the slot.  The reads have returned what they read before the barriers' phases end, the
                // add depends on this thread's wait for them, and the stores on the add being seen (by
                // an acquire, and a fence for the async proxy): no store can reach back to a read that
                // has returned.  There is no write of this thread's that the others have to see, which is
                // all that a release would add (256 x 262,144 x 5,120: 1.48 -> 1.59 ms with one,
                // 1 x 151,936 x 896 194 -> 217 us).
                if (t.kind != kLogits && rank == 0 && warp == kFirstEpi) add_relaxed(p.read_done + t.piece, 1u);
            }
        }
        if (MODE == 1 && lane == 0) tell();
        if (MODE == 1 && lane == 0) bulk_wait_all();  // the stores are complete, and shared memory no longer read
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // the pair is done with its accumulators and barriers
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
    cluster_sync_all();  // neither CTA leaves while its peer may still address it
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
struct Maps {
    CUtensorMap x, w, g, g_out, part, dt;
};

bool make_box(CUtensorMap *map, int32_t dtype, const void *base, uint64_t cols, uint64_t rows, uint64_t pitch,
              uint32_t box_cols, uint32_t box_rows) {
    return make_map(map, dtype == LHS_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                         : dtype == LHS_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                    base, cols, rows, pitch, box_cols, box_rows);
}

template <int MODE, bool BF>
cudaError_t launch(const Maps &m, const Params &p, uint32_t items, cudaStream_t stream) {
    DeviceInfo dev;
    cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    constexpr int smem = 1024 + static_cast<int>(sizeof(Smem<MODE>));
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    static_assert(2 * Conf<MODE>::kEpiWarps == kLossSyncWarps && Conf<MODE>::kEpiWarps == 4 * kLossParts, "warps that take a tile out");
    auto kern = loss_kernel<MODE, BF>;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(Conf<MODE>::kThreads);
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
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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
    cfg.gridDim = dim3(2 * (items < static_cast<uint32_t>(fit) ? items : fit));
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, m.x, m.w, m.g, m.g_out, m.part, m.dt, p);
}

// What every launch of a call shares.
bool common(const LossArgs &a, const LossPlan &p, Maps *m, Params *k) {
    const int32_t dt = p.bf16 ? LHS_BF16 : LHS_F16;
    const void *w = p.H % 8 ? static_cast<const void *>(a.ws + p.off_w) : a.t.data;
    if (!make_box(&m->x, dt, a.ws + p.off_x, p.Hp, p.Tpad, static_cast<uint64_t>(p.Hp) * 2, 64, 64) ||
        !make_box(&m->w, dt, w, p.Hp, p.V, static_cast<uint64_t>(p.Hp) * 2, 64, 64))
        return false;
    m->g = m->g_out = m->part = m->dt = m->x;  // replaced where they are used
    k->meta = reinterpret_cast<const LossMeta *>(a.ws + p.off_meta);
    k->tgt = reinterpret_cast<const int32_t *>(a.ws + p.off_tgt);
    shape_of(p, p.grad, a.dx != nullptr, a.dtable != nullptr, k);
    k->l2 = kLog2e * a.inv_temperature;
    k->queue = reinterpret_cast<uint32_t *>(a.ws + p.off_sync);
    k->err = a.err;
    return true;
}

}  // namespace

cudaError_t launch_loss_stats(const LossArgs &a, const LossPlan &p, cudaStream_t stream) {
    Maps m;
    Params k = {};
    if (!common(a, p, &m, &k)) return cudaErrorInvalidValue;
    k.stats = reinterpret_cast<float2 *>(a.ws + p.off_stats);
    k.zt = reinterpret_cast<float *>(a.ws + p.off_zt);
    const uint32_t items = static_cast<uint32_t>(p.Tpad / kLossTile * p.vt);
    return p.bf16 ? launch<0, true>(m, k, items, stream) : launch<0, false>(m, k, items, stream);
}

cudaError_t launch_loss_products(const LossArgs &a, const LossPlan &p, cudaStream_t stream) {
    const int32_t dt = p.bf16 ? LHS_BF16 : LHS_F16;
    Maps m;
    Params k = {};
    if (!common(a, p, &m, &k)) return cudaErrorInvalidValue;
    k.inv_t = a.inv_temperature;
    k.lse = reinterpret_cast<const float *>(a.ws + p.off_lse);
    k.gs = reinterpret_cast<const float *>(a.ws + p.off_gs);
    if (a.loss_in) k.em = reinterpret_cast<const float *>(a.ws + p.off_em);
    if (p.apart) {
        k.coef = reinterpret_cast<const float *>(a.ws + p.off_coef);
        if (a.dtable) k.slot_of = reinterpret_cast<const int32_t *>(a.ws + p.off_slot);
        k.rows = reinterpret_cast<const float *>(a.ws + p.off_rows);
        k.rows_pitch = p.rows_pitch;
    }
    k.dtable = a.dtable;
    k.dt_dtype = a.dtable_dtype;
    k.accumulate = a.accumulate;
    if (a.dx && !make_box(&m.part, LHS_F32, a.ws + p.off_part, p.H, static_cast<uint64_t>(p.splits) * p.Tpad,
                          static_cast<uint64_t>(p.part_pitch) * 4, 32, 32))
        return cudaErrorInvalidValue;
    if (a.dtable) {
        // rows of whole 16-byte words go by TMA; sums in 16 bits are added to what the
        // gradient held before they are rounded, which TMA's addition would do after
        const bool f32 = a.dtable_dtype == LHS_F32;
        k.dt_mode = p.H % (f32 ? 4 : 8) || (a.accumulate && !f32) ? kPlain
                    : !f32                                        ? kStore16
                    : a.accumulate                                ? kAdd32
                                                                  : kStore32;
        if (k.dt_mode != kPlain && !make_box(&m.dt, a.dtable_dtype, a.dtable, p.H, p.V,
                                             static_cast<uint64_t>(p.H) * (f32 ? 4 : 2), f32 ? 32 : 64, 32))
            return cudaErrorInvalidValue;
    }
    const uint64_t pitch = static_cast<uint64_t>(p.piece) * 2, g_rows = static_cast<uint64_t>(p.slots) * p.Tpad;
    if (!make_box(&m.g, dt, a.ws + p.off_g, p.piece, g_rows, pitch, 64, 64) ||
        !make_box(&m.g_out, dt, a.ws + p.off_g, p.piece, g_rows, pitch, 64, 32))
        return cudaErrorInvalidValue;
    k.g_done = k.queue + 1;
    k.read_done = k.g_done + p.pieces;
    k.dx_done = k.read_done + p.pieces;
    // (as many pairs as have an item, at the most positions)
    const int64_t items = p.Tpad / kLossTile * p.vt;
    const uint32_t grid = static_cast<uint32_t>(items < 65536 ? items * (1 + k.ht) : 65536);
    return p.bf16 ? launch<1, true>(m, k, grid, stream) : launch<1, false>(m, k, grid, stream);
}

}  // namespace lhs
