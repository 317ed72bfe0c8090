// loss.cu — softmax cross entropy over the tied table, and its gradient: what
// stands before and after the products (loss_gemm.cu).
//
// ADR-0008 "Remote Embeddings and lm_head Service", POST /v1/logits, gives the
// softmax over the whole vocabulary for the largest logits; here it is asked
// for given tokens, and differentiated.
//
// The first kernel of a call numbers the positions that take part and copies
// their residuals, packed, into the workspace.  Positions without a target
// (prompts, padding) then cost nothing, whatever their residuals hold reaches
// nothing (0 * NaN would, in the sums over positions of the table's gradient),
// and rows of any stride and length become rows that TMA takes.
#include "train.cuh"

namespace lhs {
namespace {

constexpr int kPackThreads = 256;
constexpr int kPackWarps = kPackThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct PackParams {
    const uint16_t *x;
    int64_t x_stride, T;
    bool vec;                // rows of x start on 16-byte boundaries
    int32_t H, Hp, ignore;
    int64_t V;
    const int32_t *targets;
    float *loss, *lse;       // loss: zeroed where a position takes no part
    const float *lse_in, *dloss;
    float inv_temperature;
    bool f16;
    LossMeta *meta;
    int32_t *act, *tgt, *pos;
    const float *loss_in;    // or null
    float *lse_c, *gs, *em;  // packed
    const uint16_t *w;       // the table, where the targets' entries are kept apart
    bool w_vec;              // its rows start on 16-byte boundaries
    float *coef;
    int32_t *slot;           // set to -1
    int64_t n_slot;
    uint16_t *xc;
    uint32_t *sync;          // cleared
    int64_t n_sync;
    int32_t *err;
};

__device__ __forceinline__ bool takes_part(const PackParams &p, int32_t y) {
    return y >= 0 && static_cast<int64_t>(y) < p.V && y != p.ignore;
}

// Exclusive prefix of `flag` over the CTA's threads, and the total.
__device__ __forceinline__ int block_rank(bool flag, int &total, int *warp_n) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, flag);
    if (lane == 0) warp_n[warp] = __popc(m);
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < kPackWarps; ++w) {
        if (w < warp) before += warp_n[w];
        total += warp_n[w];
    }
    __syncthreads();
    return before + __popc(m & ((1u << lane) - 1u));
}

// Word c (8 values) of a row of H values; zeros past them.
__device__ __forceinline__ uint4 row_word(const uint16_t *row, int c, int H, bool vec) {
    if (vec && 8 * c + 8 <= H) return ld_dep(reinterpret_cast<const uint4 *>(row) + c);
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = 8 * c + i < H ? ld_dep(row + 8 * c + i) : 0u;
    return make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
}

// The sum of the products of two words' values.
__device__ __forceinline__ float word_dot(const uint4 &a, const uint4 &b, bool f16) {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (f16)
            s[i] = fmaf(f16_bits_to_f32(static_cast<uint16_t>(u[i])), f16_bits_to_f32(static_cast<uint16_t>(v[i])),
                        f16_bits_to_f32(static_cast<uint16_t>(u[i] >> 16)) * f16_bits_to_f32(static_cast<uint16_t>(v[i] >> 16)));
        else
            s[i] = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16),
                        __uint_as_float(u[i] & 0xFFFF0000u) * __uint_as_float(v[i] & 0xFFFF0000u));
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// Each CTA takes an equal range of positions.  It counts the ones before it
// (and all of them) itself: reading every target in every CTA is less than a
// launch that would count first (8,192 targets: 32 KB from L2).
template <bool GRAD>
__global__ void __launch_bounds__(kPackThreads) loss_pack_kernel(const PackParams p) {
    __shared__ int warp_n[kPackWarps];
    __shared__ int sum_before, sum_all;
    __shared__ int rank_of[kPackThreads];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t per = (p.T + gridDim.x - 1) / gridDim.x;
    const int64_t r0 = per * blockIdx.x < p.T ? per * blockIdx.x : p.T;
    const int64_t r1 = r0 + per < p.T ? r0 + per : p.T;
    if (tid == 0) sum_before = sum_all = 0;
    pdl_wait();
    pdl_trigger();  // after the wait, so that whoever follows has everything earlier behind it
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll 8
    for (int64_t i = tid; i < p.T; i += kPackThreads) {
        const int on = takes_part(p, ld_dep(p.targets + i)) ? 1 : 0;
        all += on;
        before += i < r0 ? on : 0;
    }
    before = __reduce_add_sync(0xFFFFFFFFu, before);
    all = __reduce_add_sync(0xFFFFFFFFu, all);
    if (lane == 0) {
        atomicAdd(&sum_before, before);
        atomicAdd(&sum_all, all);
    }
    __syncthreads();
    const int count = sum_all;
    const bool twin = GRAD && count <= kLossTwin;  // every residual twice (see kLossTwin)
    int base = sum_before;
    bool bad = false, nonfinite = false;
    for (int64_t b = r0; b < r1; b += kPackThreads) {
        const int64_t r = b + tid;
        const int32_t y = r < r1 ? ld_dep(p.targets + r) : p.ignore;
        const bool on = r < r1 && takes_part(p, y);
        if (r < r1 && !on && y != p.ignore) bad = true;
        int total;
        const int c = base + block_rank(on, total, warp_n);
        rank_of[tid] = on ? c : -1;
        if (on) {
            p.act[c] = static_cast<int32_t>(r);
            p.tgt[c] = y;
            if (twin) p.tgt[c + kLossTwin] = y;
        }
        if (r < r1) {
            if (GRAD) {
                p.pos[r] = on ? c : -1;
                if (on) {
                    const float l = ld_dep(p.lse_in + r), d = ld_dep(p.dloss + r);
                    const float e = p.loss_in ? expm1f(-ld_dep(p.loss_in + r)) : 0.0f;
                    if (!isfinite(l) || !isfinite(d) || !isfinite(e)) nonfinite = true;
                    p.lse_c[c] = l;
                    p.gs[c] = d * p.inv_temperature;
                    if (p.loss_in) p.em[c] = e;
                    if (twin) {
                        if (p.loss_in) p.em[c + kLossTwin] = e;
                        p.lse_c[c + kLossTwin] = l;
                        p.gs[c + kLossTwin] = d * p.inv_temperature;
                    }
                }
            } else if (!on) {
                p.loss[r] = 0.0f;
                p.lse[r] = 0.0f;
            }
        }
        __syncthreads();
        const int n = static_cast<int>(r1 - b < kPackThreads ? r1 - b : kPackThreads);
        const uint32_t words = p.Hp / 8;
#pragma unroll 4
        for (uint32_t i = tid; i < n * words; i += kPackThreads) {
            const uint32_t r = i / words, c = i - r * words;
            const int k = rank_of[r];
            if (k >= 0) {
                const uint4 v = row_word(p.x + (b + r) * p.x_stride, c, p.H, p.vec);
                reinterpret_cast<uint4 *>(p.xc + static_cast<int64_t>(k) * p.Hp)[c] = v;
                if (twin) reinterpret_cast<uint4 *>(p.xc + static_cast<int64_t>(k + kLossTwin) * p.Hp)[c] = v;
            }
        }
        if (GRAD && p.coef) {
            // the target's entry of g, from a logit of its own in f32 (the products' kernel adds to g what
            // its logit makes of it beyond this); a warp to a position, whose row has just been read
            for (int r = warp; r < n; r += kPackWarps) {
                const int k = rank_of[r];
                if (k < 0) continue;
                const uint16_t *x = p.x + (b + r) * p.x_stride;
                const uint16_t *w = p.w + static_cast<int64_t>(ld_dep(p.targets + b + r)) * p.H;
                float z = 0.0f;
#pragma unroll 2
                for (int c = lane; c < p.Hp / 8; c += 32)
                    z += word_dot(row_word(x, c, p.H, p.vec), row_word(w, c, p.H, p.w_vec), p.f16);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
                if (lane == 0) {
                    const float l = fmaf(z, p.inv_temperature, -ld_dep(p.lse_in + b + r));
                    const float e = p.loss_in ? expm1f(-ld_dep(p.loss_in + b + r)) : p_minus_1(l, exp2f(l * kLog2e));
                    const float coef = e * (ld_dep(p.dloss + b + r) * p.inv_temperature);
                    p.coef[k] = coef;
                    if (twin) p.coef[k + kLossTwin] = coef;
                }
            }
        }
        __syncthreads();
        base += total;
    }
    // rows past the last one, to the end of its tile: zeros, no target, no gradient
    const int64_t end = count > 0 ? (static_cast<int64_t>(count) + kLossTile - 1) / kLossTile * kLossTile : kLossTile;
    for (int64_t r = count + blockIdx.x * kPackWarps + warp; r < end; r += static_cast<int64_t>(gridDim.x) * kPackWarps) {
        if (twin && r >= kLossTwin && r < kLossTwin + count) continue;
        for (int c = lane; c < p.Hp / 8; c += 32)
            reinterpret_cast<uint4 *>(p.xc + r * p.Hp)[c] = make_uint4(0u, 0u, 0u, 0u);
        if (lane == 0) {
            p.act[r] = -1;
            p.tgt[r] = -1;
            if (GRAD) {
                p.lse_c[r] = INFINITY;
                p.gs[r] = 0.0f;
                if (p.coef) p.coef[r] = 0.0f;
            }
        }
    }
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPackThreads + tid; i < p.n_sync;
         i += static_cast<int64_t>(gridDim.x) * kPackThreads)
        p.sync[i] = 0u;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPackThreads + tid; i < p.n_slot;
         i += static_cast<int64_t>(gridDim.x) * kPackThreads)
        p.slot[i] = -1;
    if (bad) set_err(p.err, LHS_ERRBIT_BAD_TOKEN);
    if (nonfinite) set_err(p.err, LHS_ERRBIT_NONFINITE);
    if (blockIdx.x == 0) {
        // The power of two that brings the largest |g| into (1/4, 1] (bf16: its range needs no
        // more, and larger terms could overflow sums that fit) or up to 2^15 (f16: what lies
        // 2^-29 below it is still normal, 2^-39 below it the last subnormal).
        float top = 0.0f;
        if (GRAD) {
#pragma unroll 8
            for (int64_t i = tid; i < p.T; i += kPackThreads) {
                const float d = fabsf(ld_dep(p.dloss + i) * p.inv_temperature);
                if (takes_part(p, ld_dep(p.targets + i)) && isfinite(d)) top = fmaxf(top, d);
            }
            __shared__ float warp_top[kPackWarps];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            if (lane == 0) warp_top[warp] = top;
            __syncthreads();
            for (int w = 0; w < kPackWarps; ++w) top = fmaxf(top, warp_top[w]);
        }
        if (tid == 0) {
            int e = top > 0.0f ? ilogbf(top) + 1 : 0;  // top < 2^e
            e = e < -100 ? -100 : e > 100 ? 100 : e;
            e -= p.f16 ? 15 : 0;
            p.meta->count = count;
            p.meta->scale = exp2f(static_cast<float>(-e));
            p.meta->unscale = exp2f(static_cast<float>(e));
        }
    }
}

// The table in rows of whole 16-byte words, where its own are not.  A warp to a row; a
// word is cut out of the two aligned ones that it lies in, but at the table's end, where the
// second may reach past it.
__global__ void __launch_bounds__(256)
    loss_table_kernel(const uint16_t *w, int64_t V, int H, int Hp, uint16_t *out) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const int64_t end = V * H * 2;  // bytes; the table starts on a 16-byte boundary
    const uint8_t *bytes = reinterpret_cast<const uint8_t *>(w);
    for (int64_t r = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; r < V;
         r += (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5) {
#pragma unroll 2
        for (int c = lane; c < Hp / 8; c += 32) {
            const int64_t at = r * H * 2 + c * 16, a = at & ~int64_t(15);
            uint4 v;
            if (8 * c + 8 <= H && a + 32 <= end) {
                const uint4 lo = ld_dep(reinterpret_cast<const uint4 *>(bytes + a));
                const uint4 hi = ld_dep(reinterpret_cast<const uint4 *>(bytes + a + 16));
                const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                const int skip = static_cast<int>(at - a) / 4, bits = static_cast<int>(at - a) % 4 * 8;
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t x = 0, y = 0;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (skip == q) x = u[k + q], y = u[k + q + 1];
                    o[k] = __funnelshift_r(x, y, bits);
                }
                v = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
                v = row_word(w + r * H, c, H, false);
            }
            reinterpret_cast<uint4 *>(out + r * Hp)[c] = v;
        }
    }
}

// A pair (m, s) stands for (1 + s) exp(m): the 1 is the maximum's own term, kept
// out of the sums so that log1p sees a small rest unspoilt.
__device__ __forceinline__ void join_pair(float &m, float &s, float om, float os, float l2) {
    if (om == -INFINITY) {
        s += os;  // nothing, or NaN
    } else if (m == -INFINITY) {
        m = om;
        s += os;
    } else {
        const float lo = fminf(m, om), hi = fmaxf(m, om);
        s = (om > m ? os : s) + (1.0f + (om > m ? s : os)) * exp2f((lo - hi) * l2);
        m = hi;
    }
}

// Joins a token's parts of tiles: 8 tokens to a CTA, 128 threads to a token, which take the
// tiles in turn; their pairs are joined in a fixed order.  (32 tokens to a CTA with
// 32 threads each: 22 us for 256 tokens and 1,024 tiles.)
constexpr int kMergeTokens = 8, kMergeWarps = 32, kMergeThreads = 32 * kMergeWarps;
__global__ void __launch_bounds__(kMergeThreads)
    loss_merge_kernel(const LossMeta *meta, const int32_t *act, const float2 *stats, const float *zt, int64_t vt,
                      int64_t Tpad, float inv_temperature, float *loss, float *lse, int32_t *err) {
    constexpr int kShare = kMergeThreads / kMergeTokens, kBatch = 8;
    __shared__ float2 part[kMergeWarps][kMergeTokens];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kMergeTokens, i = i0 + threadIdx.x % kMergeTokens;
    const int count = ld_dep(&meta->count);
    if (i0 >= count) return;
    const float l2 = kLog2e * inv_temperature;
    float m = -INFINITY, s = 0.0f;
    for (int64_t v0 = threadIdx.x / kMergeTokens; v0 < vt; v0 += kShare * kBatch) {
        float2 t[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            t[k] = v0 + k * kShare < vt ? ld_dep(stats + (v0 + k * kShare) * Tpad + i) : make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) join_pair(m, s, t[k].x, t[k].y, l2);
    }
#pragma unroll
    for (int o = kMergeTokens; o < 32; o <<= 1)
        join_pair(m, s, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, s, o), l2);
    if (lane < kMergeTokens) part[warp][lane] = make_float2(m, s);
    __syncthreads();
    if (warp >= kMergeTokens) return;
    const float2 t = part[lane][warp];  // a warp to a token
    m = t.x, s = t.y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
        join_pair(m, s, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, s, o), l2);
    if (lane == 0 && i0 + warp < count) {
        const float ls = log1pf(s);
        float l = m * inv_temperature + ls;
        float c = (m - ld_dep(zt + i0 + warp)) * inv_temperature + ls;
        if (!isfinite(l)) {
            l = c = __int_as_float(0x7FC00000);
            set_err(err, LHS_ERRBIT_NONFINITE);
        }
        const int32_t r = ld_dep(act + i0 + warp);
        loss[r] = c;
        lse[r] = l;
    }
}

// dx of every position: its compact row's sums (and its twin's), joined in order,
// times the inverse of g's scale, and the target's row of the table by what is kept apart of
// its entry (w null: nothing is); or zeros.  A warp to 128 columns of a position.
template <typename T>
__global__ void __launch_bounds__(256)
    loss_dx_kernel(const LossMeta *meta, const int32_t *pos, const float *part, int splits, int64_t Tpad, int pitch,
                   int64_t n, int32_t H, T *dx, int64_t dx_stride, bool vec, const uint16_t *w, bool f16, int Hp,
                   const int32_t *tgt, const float *coef) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    const float u = ld_dep(&meta->unscale);
    const bool twin = ld_dep(&meta->count) <= kLossTwin;
    const uint32_t blocks = (H + 127) / 128;
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; i < n * blocks;
         i += (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5) {
        const int64_t r = i / blocks;
        const int32_t c = ld_dep(pos + r);
        T *d = dx + r * dx_stride;
        const int j = static_cast<int>(i - r * blocks) * 128 + lane * 4;
        if (j < H) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (c >= 0) {
                const float4 *src = reinterpret_cast<const float4 *>(part + static_cast<int64_t>(c) * pitch + j);
                const int64_t step = Tpad * pitch / 4;
                v = ld_dep(src);
#pragma unroll 4
                for (int k = 1; k < splits; ++k) {
                    const float4 a = ld_dep(src + k * step);
                    v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
                }
                if (twin) {
                    src += kLossTwin * pitch / 4;
                    for (int k = 0; k < splits; ++k) {
                        const float4 a = ld_dep(src + k * step);
                        v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
                    }
                }
                if (w) {  // (rows of whole 16-byte words)
                    const uint2 row = ld_dep(reinterpret_cast<const uint2 *>(w + static_cast<int64_t>(ld_dep(tgt + c)) * Hp + j));
                    const float e = ld_dep(coef + c);
                    const uint16_t b[4] = {static_cast<uint16_t>(row.x), static_cast<uint16_t>(row.x >> 16),
                                           static_cast<uint16_t>(row.y), static_cast<uint16_t>(row.y >> 16)};
                    float t[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) t[k] = e * (f16 ? f16_bits_to_f32(b[k]) : bf16_bits_to_f32(b[k]));
                    v.x = fmaf(v.x, u, t[0]), v.y = fmaf(v.y, u, t[1]), v.z = fmaf(v.z, u, t[2]), v.w = fmaf(v.w, u, t[3]);
                } else {
                    v.x *= u, v.y *= u, v.z *= u, v.w *= u;
                }
            }
            const float f[4] = {v.x, v.y, v.z, v.w};
            if (vec && j + 4 <= H) {
                alignas(16) T o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) put_rn(&o[k], f[k]);
                if (sizeof(T) == 4) *reinterpret_cast<float4 *>(d + j) = *reinterpret_cast<const float4 *>(o);
                else *reinterpret_cast<uint2 *>(d + j) = *reinterpret_cast<const uint2 *>(o);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (j + k < H) put_rn(d + j + k, f[k]);
            }
        }
    }
}

// The table in rows of whole 16-byte words.
const uint16_t *whole_rows(const LossArgs &a, const LossPlan &p) {
    return p.H % 8 ? reinterpret_cast<const uint16_t *>(a.ws + p.off_w) : static_cast<const uint16_t *>(a.t.data);
}

template <typename T>
cudaError_t launch_dx(const LossArgs &a, const LossPlan &p, const DeviceInfo &dev, cudaStream_t stream) {
    const int64_t want = (p.T * ((p.H + 127) / 128) + 7) / 8;
    const bool vec = reinterpret_cast<uintptr_t>(a.dx) % (4 * sizeof(T)) == 0 && a.dx_stride % 4 == 0;
    return launch_pdl(loss_dx_kernel<T>, dim3(static_cast<unsigned>(want < 8 * dev.num_sms ? want : 8 * dev.num_sms)),
                      dim3(256), 0, stream, reinterpret_cast<const LossMeta *>(a.ws + p.off_meta),
                      reinterpret_cast<const int32_t *>(a.ws + p.off_pos), reinterpret_cast<const float *>(a.ws + p.off_part),
                      p.splits, p.Tpad, p.part_pitch, p.T, p.H, static_cast<T *>(a.dx), a.dx_stride, vec,
                      p.apart ? whole_rows(a, p) : nullptr, !p.bf16, p.Hp,
                      reinterpret_cast<const int32_t *>(a.ws + p.off_tgt), reinterpret_cast<const float *>(a.ws + p.off_coef));
}

cudaError_t launch_pack(const LossArgs &a, const LossPlan &p, const DeviceInfo &dev, cudaStream_t stream) {
    PackParams k = {};
    k.x = static_cast<const uint16_t *>(a.x);
    k.x_stride = a.x_stride;
    k.T = p.T;
    k.vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.x_stride % 8 == 0;
    k.H = p.H;
    k.Hp = p.Hp;
    k.ignore = a.ignore;
    k.V = p.V;
    k.targets = a.targets;
    k.loss = a.loss;
    k.lse = a.lse;
    k.lse_in = a.lse_in;
    k.dloss = a.dloss;
    k.inv_temperature = a.inv_temperature;
    k.f16 = !p.bf16;
    k.meta = reinterpret_cast<LossMeta *>(a.ws + p.off_meta);
    k.act = reinterpret_cast<int32_t *>(a.ws + p.off_act);
    k.tgt = reinterpret_cast<int32_t *>(a.ws + p.off_tgt);
    k.pos = reinterpret_cast<int32_t *>(a.ws + p.off_pos);
    k.lse_c = reinterpret_cast<float *>(a.ws + p.off_lse);
    k.gs = reinterpret_cast<float *>(a.ws + p.off_gs);
    k.loss_in = a.loss_in;
    k.em = reinterpret_cast<float *>(a.ws + p.off_em);
    if (p.apart) {
        k.w = static_cast<const uint16_t *>(a.t.data);
        k.w_vec = p.H % 8 == 0;
        k.coef = reinterpret_cast<float *>(a.ws + p.off_coef);
        k.slot = reinterpret_cast<int32_t *>(a.ws + p.off_slot);
        k.n_slot = a.dtable ? p.V + p.vt : 0;
    }
    k.xc = reinterpret_cast<uint16_t *>(a.ws + p.off_x);
    k.sync = reinterpret_cast<uint32_t *>(a.ws + p.off_sync);
    k.n_sync = p.n_sync;
    k.err = a.err;
    cudaError_t e = cudaSuccess;
    if (p.H % 8) {
        const int64_t ctas = (p.V + 7) / 8;
        e = launch_pdl(loss_table_kernel, dim3(static_cast<unsigned>(ctas < 8 * dev.num_sms ? ctas : 8 * dev.num_sms)), dim3(256), 0,
                       stream, static_cast<const uint16_t *>(a.t.data), p.V, p.H, p.Hp,
                       reinterpret_cast<uint16_t *>(a.ws + p.off_w));
        if (e != cudaSuccess) return e;
    }
    // (by whole tiles of tokens: the rows that fill the last one up are written too)
    const int64_t want = p.Tpad;
    const unsigned grid = static_cast<unsigned>(want < 4 * dev.num_sms ? want : 4 * dev.num_sms);
    return launch_pdl(p.grad ? loss_pack_kernel<true> : loss_pack_kernel<false>, dim3(grid), dim3(kPackThreads), 0,
                      stream, k);
}

}  // namespace

LossPlan plan_loss(const lhs_table &t, int64_t tokens, bool grad) {
    LossPlan p = {};
    p.T = tokens;
    p.Tpad = tokens > 0 ? round_up(tokens, kLossTile) : kLossTile;
    p.V = t.vocab;
    p.vt = (t.vocab + kLossTile - 1) / kLossTile;
    p.H = t.hidden;
    p.Hp = static_cast<int32_t>(round_up(t.hidden, 8));
    p.bf16 = t.dtype == LHS_BF16;
    p.grad = grad;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += align256(bytes);
        return o;
    };
    p.off_meta = take(sizeof(LossMeta));
    p.off_act = take(p.Tpad * 4);
    p.off_tgt = take(p.Tpad * 4);
    p.off_x = take(p.Tpad * p.Hp * 2);
    p.off_w = take(p.H % 8 ? p.V * p.Hp * 2 : 0);
    if (!grad) {
        p.n_sync = 1;
        p.off_sync = take(4);
        p.off_stats = take(p.vt * kLossParts * p.Tpad * 8);
        p.off_zt = take(p.Tpad * 4);
    } else {
        choose_pieces(&p);
        p.part_pitch = static_cast<int32_t>(round_up(p.H, 4));
        p.off_sync = take(p.n_sync * 4);
        p.off_pos = take(p.T * 4);
        p.off_lse = take(p.Tpad * 4);
        p.off_gs = take(p.Tpad * 4);
        p.off_em = take(p.Tpad * 4);
        p.apart = p.T > kLossTwin;
        if (p.apart) {
            p.rows_pitch = round_up(p.H, 64);
            p.off_coef = take(p.Tpad * 4);
            p.off_slot = take((p.V + p.vt) * 4);
            p.off_rows = take((p.T < p.V ? p.T : p.V) * p.rows_pitch * 4);
            p.off_order = take(embed_grad_workspace(p.Hp, p.T));
        }
        p.off_g = take(p.slots * p.Tpad * p.piece * 2);
        p.off_part = take(p.splits * p.Tpad * p.part_pitch * 4);
    }
    p.bytes = at;
    return p;
}

cudaError_t launch_loss(const LossArgs &a, const LossPlan &p, cudaStream_t stream) {
    DeviceInfo dev;
    cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    if ((e = launch_pack(a, p, dev, stream)) != cudaSuccess) return e;
    if ((e = launch_loss_stats(a, p, stream)) != cudaSuccess) return e;
    return launch_pdl(loss_merge_kernel, dim3(static_cast<unsigned>(p.Tpad / kMergeTokens)), dim3(kMergeThreads), 0, stream,
                      reinterpret_cast<const LossMeta *>(a.ws + p.off_meta),
                      reinterpret_cast<const int32_t *>(a.ws + p.off_act),
                      reinterpret_cast<const float2 *>(a.ws + p.off_stats),
                      reinterpret_cast<const float *>(a.ws + p.off_zt), p.vt * kLossParts, p.Tpad, a.inv_temperature, a.loss, a.lse,
                      a.err);
}

cudaError_t launch_loss_grad(const LossArgs &a, const LossPlan &p, cudaStream_t stream) {
    if (p.T == 0) {
        const size_t es = a.dtable_dtype == LHS_F32 ? 4 : 2;
        return a.dtable && !a.accumulate ? launch_zero(a.dtable, static_cast<size_t>(p.V) * p.H * es, stream) : cudaSuccess;
    }
    DeviceInfo dev;
    cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    if ((e = launch_pack(a, p, dev, stream)) != cudaSuccess) return e;
    if (p.apart && a.dtable) {
        const TargetRowsArgs r = {a.targets, p.T, p.V, a.ignore, p.Hp, p.bf16,
                                  reinterpret_cast<const uint16_t *>(a.ws + p.off_x),
                                  reinterpret_cast<const int32_t *>(a.ws + p.off_pos),
                                  reinterpret_cast<const float *>(a.ws + p.off_coef),
                                  reinterpret_cast<float *>(a.ws + p.off_rows), p.rows_pitch,
                                  reinterpret_cast<int32_t *>(a.ws + p.off_slot), a.ws + p.off_order, a.err};
        if ((e = launch_target_rows(r, stream)) != cudaSuccess) return e;
    }
    if ((e = launch_loss_products(a, p, stream)) != cudaSuccess) return e;
    if (!a.dx) return cudaSuccess;
    if (a.dx_dtype == LHS_F32) return launch_dx<float>(a, p, dev, stream);
    return p.bf16 ? launch_dx<__nv_bfloat16>(a, p, dev, stream) : launch_dx<__half>(a, p, dev, stream);
}

}  // namespace lhs
