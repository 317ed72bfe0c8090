// i8_gemv.cu — the 8-bit lm_head product of up to sixteen tokens: the table
// streams through shared memory once.
//
// With m tokens a table byte carries 2 m operations, far below the ridge, so
// the floor is the table's bytes at the HBM rate, 23.5 bytes a clock and SM or
// 697 clocks for a 16 KB stage of the ring.  What multiplies a stage must be
// well under that, because the ring is full when the warps start and what they
// cannot catch up on is time after the stream's end.
//  * Up to four tokens: four-way dot products on the codes as they are, about
//    64 clocks a token and stage.
//  * Up to sixteen: mma.sync.m16n8k16 in f16 (1,040 products a clock and SM
//    here; the integer form, m16n8k32 in s8, does 260, 504 clocks for a stage
//    of eight tokens).  The codes are widened in registers: a word of four
//    consecutive codes becomes two f16 pairs that serve as the k positions 2t,
//    2t+1, 2t+8 and 2t+9 of the fragment, for both operands alike, so no code
//    moves between lanes.  f32 sums of up to 1,024 products are exact; they
//    are added up as integers.
// (The tcgen05 kernel of i8_matmul.cu, whose operand has to pass through tensor
// memory, needs about 1,000 clocks for a stage of so few tokens.)
//
// One CTA per SM: two groups of eight warps, each warp with 16 of its group's
// tile of 128 rows, and a producer that keeps a ring of TMA boxes full for
// each, the two tiles' stages in turn.  A stage's wait, loads, widening and
// products are one chain of latencies, and two groups have two under way.
// (One ring for both would let a group that is ahead mistake the barrier of a
// slot whose earlier copy, the other group's, is still on its way for its own:
// a wait tells two phases apart, not three.)  The CTAs take the 128-row tiles
// in turn; the rows that do not fill a round of them are split evenly, in units
// of 16 rows with boxes of that size.  The tokens are quantised by every CTA
// for itself while its ring fills, so a call is one launch.
//
// Measured: 1 x 151,936 x 896 in 23.2 us (87% of the HBM rate; a stream this
// short is 3 us of start and end), 8 x 262,144 x 5,376 in 233 us (90%).
#include <mutex>

#include "i8_common.cuh"

namespace lhs {
namespace {

constexpr int kMaxTokens = 16;
constexpr int kGroups = 2;                 // of warps, each with a tile of its own
constexpr int kGroupWarps = 8;
constexpr int kWarps = kGroups * kGroupWarps;
constexpr int kConsumers = 32 * kWarps;
constexpr int kThreads = kConsumers + 32;  // + producer
constexpr int kUnitRows = 16;
constexpr int kUnitBytes = kUnitRows * kStageK;
constexpr int kMaxStages = 12;            // of both groups' rings
constexpr int kTokenBytes = 98 * 1024;     // tokens' codes at most, beside six stages
constexpr int kSmemBytes = 224 * 1024;

__host__ __device__ constexpr int round_up(int v, int a) { return (v + a - 1) / a * a; }
// Token rows 16 bytes past a multiple of 128: eight rows' 16-byte pieces lie
// in different banks.
__host__ __device__ constexpr int token_pitch(int hidden) { return round_up(hidden, kStageK) + 16; }

struct Head {
    uint64_t full[kMaxStages], empty[kMaxStages];
    float scale[kMaxTokens];
    float part[kWarps][kMaxTokens];
    int bad[kWarps];
    int abort_flag;
};

struct Params {
    I8Tokens a;
    bool vec;           // four wide values (or codes) of a token may be loaded at once
    const uint8_t *w_scales;
    int64_t w_scale_stride;
    int64_t channels;
    int hidden, nst;    // stages of each group's ring
    void *out;
    int64_t out_stride;
    int out_dtype;
    int32_t *err;
};

// The tiles of one CTA: `rounds` full ones, then `units` units of 16 rows.
struct Share {
    int64_t rounds, tail;
    int units;
    __device__ __forceinline__ Share(int64_t channels) {
        const int64_t round_rows = static_cast<int64_t>(gridDim.x) * kCtaRows;
        rounds = channels / round_rows;
        const int64_t u = (channels - rounds * round_rows + kUnitRows - 1) / kUnitRows;
        const int64_t u0 = u * blockIdx.x / gridDim.x, u1 = u * (blockIdx.x + 1) / gridDim.x;
        tail = rounds * round_rows + u0 * kUnitRows;
        units = static_cast<int>(u1 - u0);
    }
    __device__ __forceinline__ int64_t tiles() const { return rounds + (units > 0 ? 1 : 0); }
    __device__ __forceinline__ int64_t row(int64_t i) const {
        return i < rounds ? (i * gridDim.x + blockIdx.x) * kCtaRows : tail;
    }
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Token rows held in shared memory for m tokens: 1, 2, 4, 8 or 16.
__host__ __device__ constexpr int token_rows(int64_t m) { return m <= 1 ? 1 : m <= 2 ? 2 : m <= 4 ? 4 : m <= 8 ? 8 : 16; }

// DT: the tokens' type, or -1 for codes; R: token rows, zeros past the tokens.
// Rows for the f16 products have their codes' sign bits flipped (see widen4).
template <int DT, int R>
__device__ __forceinline__ void stage_tokens(const Params &p, uint8_t *tok, Head &sm, int tid) {
    const int warp = tid >> 5, lane = tid & 31;
    const int pitch = token_pitch(p.hidden), groups = (pitch - 16) / 4, m = static_cast<int>(p.a.rows);
    constexpr uint32_t flip = R > 4 ? 0x80808080u : 0u;
    if constexpr (DT < 0) {
        for (int i = tid; i < R * groups; i += kConsumers) {
            const int t = i / groups, j = (i - t * groups) * 4;
            uint32_t w = 0;
            if (t < m) {
                const int8_t *row = p.a.coded.codes + t * p.a.coded.stride;
                if (p.vec && j + 4 <= p.hidden) w = ld_dep(reinterpret_cast<const uint32_t *>(row + j));
                else
                    for (int e = 0; e < 4; ++e)
                        if (j + e < p.hidden) w |= static_cast<uint32_t>(static_cast<uint8_t>(ld_dep(row + j + e))) << (8 * e);
            }
            *reinterpret_cast<uint32_t *>(tok + t * pitch + j) = w ^ flip;
        }
        if (tid < R) sm.scale[tid] = tid < m ? coded_scale(p.a.coded, tid, blockIdx.x == 0 ? p.err : nullptr) : 0.0f;
        named_bar_sync(1, kConsumers);
    } else {
        using E = typename Elem<DT>::T;
        const E *x = static_cast<const E *>(p.a.x);
        // max|x| of every token (whether all are finite in bad), then scales and codes; the
        // second reading comes from L2
        float mx[R];
        uint32_t bad = 0;
#pragma unroll
        for (int t = 0; t < R; ++t) {
            mx[t] = 0.0f;
            if (t >= m) continue;
#pragma unroll 4
            for (int g = tid; g < groups; g += kConsumers) {
                float v[4];
                load4<DT>(x + t * p.a.x_stride, 4 * g, p.hidden, p.vec, v);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (isfinite(v[i])) mx[t] = fmaxf(mx[t], fabsf(v[i]));
                    else bad |= 1u << t;
                }
            }
        }
#pragma unroll
        for (int t = 0; t < R; ++t) {
            if (t >= m) continue;
            const uint32_t u = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(mx[t]));
            if (lane == 0) sm.part[warp][t] = __uint_as_float(u);
        }
        bad = __reduce_or_sync(0xFFFFFFFFu, bad);
        if (lane == 0) sm.bad[warp] = static_cast<int>(bad);
        named_bar_sync(1, kConsumers);
        for (int w = 0; w < kWarps; ++w) bad |= static_cast<uint32_t>(sm.bad[w]);
        if (tid == 0 && blockIdx.x == 0 && bad) set_err(p.err, LHS_ERRBIT_NONFINITE);
        for (int t = 0; t < R; ++t) {
            float top = 0.0f;
            if (t < m)
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm.part[w][t]);
            const float scale = (bad >> t) & 1u ? 0.0f : __fdiv_rn(top, 127.0f);
            const float rcp = __frcp_rn(scale);
            if (tid == 0) sm.scale[t] = scale;
#pragma unroll 4
            for (int g = tid; g < groups; g += kConsumers) {
                uint32_t w = 0;
                if (t < m) {
                    float v[4];
                    load4<DT>(x + t * p.a.x_stride, 4 * g, p.hidden, p.vec, v);
                    w = i8_code4(v, scale, rcp);
                }
                *reinterpret_cast<uint32_t *>(tok + t * pitch + 4 * g) = w ^ flip;
            }
        }
        named_bar_sync(1, kConsumers);
    }
}

template <int R>
__global__ void __launch_bounds__(kThreads, 1)
    i8_gemv_kernel(const __grid_constant__ CUtensorMap tm_tile, const __grid_constant__ CUtensorMap tm_unit,
                   const Params p) {
    extern __shared__ uint8_t dyn_smem[];
    uint8_t *ring = smem_align<1024>(dyn_smem);
    const int pitch = token_pitch(p.hidden);
    uint8_t *tok = ring + kGroups * p.nst * kTableStageBytes;
    Head &sm = *reinterpret_cast<Head *>(tok + R * pitch);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Share share(p.channels);
    const int nk = (p.hidden + kStageK - 1) / kStageK;

    if (tid == 0) {
        for (int s = 0; s < kGroups * p.nst; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], kGroupWarps);
        }
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_trigger();
    pdl_wait();  // the table may have been quantised, the tokens written, by the kernel before

    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*reinterpret_cast<volatile int *>(&sm.abort_flag)) return false;
        if (mbar_wait(bar, parity, kWaitTimeoutNs)) return true;
        set_err(p.err, LHS_ERRBIT_TIMEOUT);
        *reinterpret_cast<volatile int *>(&sm.abort_flag) = 1;
        return false;
    };

    if (warp == kWarps) {
        if (lane == 0) {
            tma_prefetch_map(&tm_tile);
            int s[kGroups] = {}, issued[kGroups] = {};
            uint32_t parity[kGroups];
#pragma unroll
            for (int w = 0; w < kGroups; ++w) parity[w] = 1;
            bool ok = true;
            // the groups' stages in turn
            for (int64_t i0 = 0; i0 < share.tiles() && ok; i0 += kGroups)
                for (int kc = 0; kc < nk && ok; ++kc)
#pragma unroll
                    for (int w = 0; w < kGroups; ++w) {
                        const int64_t i = i0 + w;
                        if (i >= share.tiles() || !ok) break;
                        const int slot = w * p.nst + s[w];
                        if (!wait(&sm.empty[slot], parity[w])) {
                            ok = false;
                            break;
                        }
                        const int32_t row = static_cast<int32_t>(share.row(i));
                        uint8_t *dst = ring + slot * kTableStageBytes;
                        if (i < share.rounds) {
                            mbar_arrive_expect_tx(&sm.full[slot], kTableStageBytes);
                            tma_load_2d(dst, &tm_tile, &sm.full[slot], kc * kStageK, row);
                        } else {
                            mbar_arrive_expect_tx(&sm.full[slot], share.units * kUnitBytes);
                            for (int u = 0; u < share.units; ++u)
                                tma_load_2d(dst + u * kUnitBytes, &tm_unit, &sm.full[slot], kc * kStageK,
                                            row + u * kUnitRows);
                        }
                        if (issued[w] < p.nst) ++issued[w];
                        if (++s[w] == p.nst) {
                            s[w] = 0;
                            parity[w] ^= 1u;
                        }
                    }
            // every copy that was issued has landed
#pragma unroll
            for (int w = 0; w < kGroups; ++w)
                for (int i = 0; i < issued[w]; ++i) {
                    if (--s[w] < 0) {
                        s[w] = p.nst - 1;
                        parity[w] ^= 1u;
                    }
                    mbar_wait(&sm.full[w * p.nst + s[w]], parity[w] ^ 1u, kWaitTimeoutNs);
                }
        }
        return;
    }

    if (!p.a.x) stage_tokens<-1, R>(p, tok, sm, tid);
    else if (p.a.x_dtype == LHS_F32) stage_tokens<LHS_F32, R>(p, tok, sm, tid);
    else if (p.a.x_dtype == LHS_F16) stage_tokens<LHS_F16, R>(p, tok, sm, tid);
    else stage_tokens<LHS_BF16, R>(p, tok, sm, tid);

    const int m = static_cast<int>(p.a.rows);
    const int g = lane >> 2, q = lane & 3;  // this thread's rows: g and g + 8 of the warp's 16
    // the dot products: quarter q of both rows' codes.  The f16 products: ldmatrix addresses, lanes
    // 8 i .. 8 i + 7 naming the rows of matrix i (A: rows 0-7 and 8-15 of the warp's, then the same
    // 16 bytes further on; B: eight tokens at four 16-byte steps)
    const int group = warp / kGroupWarps, wrow = warp % kGroupWarps * 16;  // the warp's rows of the group's tile
    const int arow = wrow + (lane & 15), apiece = lane >> 4;
    const uint32_t a_addr = smem_u32(ring) + arow * kStageK;
    const uint32_t b_addr = smem_u32(tok) + (lane & 7) * pitch + (lane >> 3) * 16;
    const int first = group * p.nst;  // the group's own ring
    int s = first;
    uint32_t parity = 0;
    for (int64_t i = group; i < share.tiles(); i += kGroups) {
        const bool mine = i < share.rounds || wrow < share.units * kUnitRows;  // the last tile may be short
        const int64_t ch = share.row(i) + wrow + g;
        float ws[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            ws[h] = mine && ch + 8 * h < p.channels
                        ? ld_dep(reinterpret_cast<const float *>(p.w_scales + (ch + 8 * h) * p.w_scale_stride))
                        : 0.0f;
        // sums of rows g and g + 8: of each token (dot products, a quarter of the codes each), or of
        // tokens 8 n + 2 q and 8 n + 2 q + 1
        constexpr int NT = R > 4 ? R / 8 : 1, NS = R > 4 ? 2 : R;
        int acc[2][NT][NS] = {};
        float c[NT][2][4] = {};
        for (int kc = 0; kc < nk; ++kc) {
            if (!__all_sync(0xFFFFFFFFu, wait(&sm.full[s], parity))) return;
            if (mine) {
                if constexpr (R <= 4) {
                    const uint8_t *w = ring + s * kTableStageBytes + (wrow + g) * kStageK;
                    const uint8_t *x = tok + kc * kStageK + q * 32;
                    uint4 u[2][2];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 2; ++e)  // rows 8 apart have the same swizzle
                            u[h][e] = *reinterpret_cast<const uint4 *>(w + h * 8 * kStageK + (((2 * q + e) ^ g) << 4));
#pragma unroll
                    for (int t = 0; t < R; ++t)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(x + t * pitch + e * 16);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                int &a = acc[h][0][t];
                                a = __dp4a(static_cast<int>(u[h][e].x), static_cast<int>(v.x), a);
                                a = __dp4a(static_cast<int>(u[h][e].y), static_cast<int>(v.y), a);
                                a = __dp4a(static_cast<int>(u[h][e].z), static_cast<int>(v.z), a);
                                a = __dp4a(static_cast<int>(u[h][e].w), static_cast<int>(v.w), a);
                            }
                        }
                } else {
                    const uint32_t base = a_addr + s * kTableStageBytes;
#pragma unroll
                    for (int o = 0; o < 2; ++o) {  // 64 codes at a time
                        uint32_t a[2][4], b[NT][4];
#pragma unroll
                        for (int e = 0; e < 2; ++e) ldmatrix_x4(base + (((4 * o + 2 * e + apiece) ^ (arow & 7)) << 4), a[e]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) ldmatrix_x4(b_addr + n * 8 * pitch + kc * kStageK + o * 64, b[n]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {  // 16 codes: words a[e / 2][2 (e % 2)] (row g) and the next (g + 8)
                            uint32_t a0, a1, a2, a3;
                            widen4(a[e >> 1][2 * (e & 1)] ^ 0x80808080u, a0, a2);
                            widen4(a[e >> 1][2 * (e & 1) + 1] ^ 0x80808080u, a1, a3);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                uint32_t b0, b1;
                                widen4(b[n][e], b0, b1);
                                mma_f16(c[n][e & 1], a0, a1, a2, a3, b0, b1);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.empty[s]);
            if (++s == first + p.nst) {
                s = first;
                parity ^= 1u;
            }
            if constexpr (R > 4) {
                if ((kc & 7) == 7 || kc + 1 == nk) {  // 1,024 codes: the two halves are exact
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            acc[e >> 1][n][e & 1] += __float2int_rn(c[n][0][e]) + __float2int_rn(c[n][1][e]);
                            c[n][0][e] = c[n][1][e] = 0.0f;
                        }
                }
            }
        }
        if (!mine) continue;
        if constexpr (R <= 4) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < R; ++t) {
                    acc[h][0][t] += __shfl_xor_sync(0xFFFFFFFFu, acc[h][0][t], 1);
                    acc[h][0][t] += __shfl_xor_sync(0xFFFFFFFFu, acc[h][0][t], 2);
                }
        }
        auto emit = [&](auto *out) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < NS; ++e) {
                        const int t = R > 4 ? 8 * n + 2 * q + e : e;
                        const float v = __fmul_rn(__fmul_rn(static_cast<float>(acc[h][n][e]), sm.scale[t]), ws[h]);
                        if ((R > 4 || q == e) && t < m && ch + 8 * h < p.channels)
                            put(out + t * p.out_stride + ch + 8 * h, v);
                    }
        };
        if (p.out_dtype == LHS_F32) emit(static_cast<float *>(p.out));
        else if (p.out_dtype == LHS_F16) emit(static_cast<__half *>(p.out));
        else emit(static_cast<__nv_bfloat16 *>(p.out));
    }
}

template <int R>
cudaError_t launch(const CUtensorMap &tm_tile, const CUtensorMap &tm_unit, Params &p, unsigned grid,
                   const DeviceInfo &dev, cudaStream_t stream) {
    const int fixed = 1024 + R * token_pitch(p.hidden) + static_cast<int>(sizeof(Head));
    p.nst = (kSmemBytes - fixed) / kTableStageBytes;
    p.nst = (p.nst < kMaxStages ? p.nst : kMaxStages) / kGroups;
    {
        static std::mutex mu;
        static bool done[64] = {};
        std::lock_guard<std::mutex> lock(mu);
        if (!done[dev.device]) {
            const cudaError_t e =
                cudaFuncSetAttribute(i8_gemv_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
            if (e != cudaSuccess) return e;
            done[dev.device] = true;
        }
    }
    return launch_pdl(i8_gemv_kernel<R>, dim3(grid), dim3(kThreads), fixed + kGroups * p.nst * kTableStageBytes, stream, tm_tile,
                      tm_unit, p);
}

}  // namespace

// The tokens' codes stay in shared memory, so hidden is bounded.
bool i8_gemv_serves(const lhs_i8 &table, int64_t tokens) {
    return tokens <= kMaxTokens &&
           static_cast<int64_t>(token_rows(tokens)) * token_pitch(table.hidden) <= kTokenBytes;
}

cudaError_t launch_i8_gemv(const I8Tokens &a, const lhs_i8 &table, void *out, int32_t out_dtype,
                           int64_t out_stride, int32_t *err, const DeviceInfo &dev, cudaStream_t stream) {
    Params p = {};
    p.a = a;
    if (a.x) {
        const int64_t size = a.x_dtype == LHS_F32 ? 4 : 2;
        p.vec = reinterpret_cast<uintptr_t>(a.x) % (4 * size) == 0 && a.x_stride % 4 == 0;
    } else {
        p.vec = reinterpret_cast<uintptr_t>(a.coded.codes) % 4 == 0 && a.coded.stride % 4 == 0;
    }
    p.w_scales = reinterpret_cast<const uint8_t *>(table.scales);
    p.w_scale_stride = table.scale_stride;
    p.channels = table.rows;
    p.hidden = table.hidden;
    p.out = out;
    p.out_stride = out_stride;
    p.out_dtype = out_dtype;
    p.err = err;
    CUtensorMap tm_tile, tm_unit;
    if (!make_map(&tm_tile, CU_TENSOR_MAP_DATA_TYPE_UINT8, table.codes, table.hidden, table.rows, table.stride, kStageK,
                  kCtaRows) ||
        !make_map(&tm_unit, CU_TENSOR_MAP_DATA_TYPE_UINT8, table.codes, table.hidden, table.rows, table.stride, kStageK,
                  kUnitRows))
        return cudaErrorInvalidValue;
    const int64_t units = (table.rows + kUnitRows - 1) / kUnitRows;
    const unsigned grid = static_cast<unsigned>(units < dev.num_sms ? units : dev.num_sms);
    switch (token_rows(a.rows)) {
    case 1: return launch<1>(tm_tile, tm_unit, p, grid, dev, stream);
    case 2: return launch<2>(tm_tile, tm_unit, p, grid, dev, stream);
    case 4: return launch<4>(tm_tile, tm_unit, p, grid, dev, stream);
    case 8: return launch<8>(tm_tile, tm_unit, p, grid, dev, stream);
    default: return launch<16>(tm_tile, tm_unit, p, grid, dev, stream);
    }
}

}  // namespace lhs
