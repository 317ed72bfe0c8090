// loss_gemm.cu — the products of the cross entropy and of its gradient.
//
// First form: 64 x 64 tiles of f32 sums on the CUDA cores, one kernel a
// product, a piece of the vocabulary at a time.
#include "train.cuh"

namespace lhs {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int TS = 64, TK = 16;

// acc[a][b] = sum_k A(m0 + ty*4 + a, k) * B(n0 + tx*4 + b, k); element (i, k)
// of an operand lies i*si + k*sk further on; zeros from mm, nn, kk on.
template <typename T>
__device__ void tile_product(const T *A, int64_t sam, int64_t sak, int64_t mm, const T *B, int64_t sbn, int64_t sbk,
                             int64_t nn, int64_t kk, float (&acc)[4][4], float (*sa)[TS + 4], float (*sb)[TS + 4]) {
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = 0.0f;
    for (int64_t k0 = 0; k0 < kk; k0 += TK) {
        for (int i = tid; i < TS * TK; i += 256) {
            // consecutive threads along whichever index is contiguous
            const int ma = sak == 1 ? i / TK : i % TS, ka = sak == 1 ? i % TK : i / TS;
            sa[ka][ma] = ma < mm && k0 + ka < kk ? wide(A[ma * sam + (k0 + ka) * sak]) : 0.0f;
            const int nb = sbk == 1 ? i / TK : i % TS, kb = sbk == 1 ? i % TK : i / TS;
            sb[kb][nb] = nb < nn && k0 + kb < kk ? wide(B[nb * sbn + (k0 + kb) * sbk]) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < TK; ++k) {
            float va[4], vb[4];
#pragma unroll
            for (int a = 0; a < 4; ++a) va[a] = sa[k][ty * 4 + a];
#pragma unroll
            for (int b = 0; b < 4; ++b) vb[b] = sb[k][tx * 4 + b];
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(va[a], vb[b], acc[a][b]);
        }
        __syncthreads();
    }
}

// grid: vocabulary tiles of 256 x blocks of 64 tokens
template <typename T>
__global__ void __launch_bounds__(256)
    loss_stats_kernel(const LossMeta *meta, const int32_t *tgt, const T *x, int Hp, const T *w, int64_t V, int H,
                      float inv_temperature, int64_t Tpad, float2 *stats, float *zt) {
    __shared__ float sa[TK][TS + 4], sb[TK][TS + 4];
    pdl_wait();
    const int count = ld_dep(&meta->count);
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * TS;
    if (t0 >= count) return;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const float l2 = kLog2e * inv_temperature;
    float m[4], s[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        m[a] = -INFINITY;
        s[a] = 0.0f;
    }
    auto join = [&](int a, float om, float os) {
        const float n = fmaxf(m[a], om);
        s[a] = (m[a] == -INFINITY ? s[a] : s[a] * exp2f((m[a] - n) * l2)) +
               (om == -INFINITY ? os : os * exp2f((om - n) * l2));
        m[a] = n;
    };
    for (int sub = 0; sub < kLossTile / TS; ++sub) {
        const int64_t v0 = static_cast<int64_t>(blockIdx.x) * kLossTile + sub * TS;
        if (v0 >= V) break;
        float acc[4][4];
        tile_product(x + t0 * Hp, Hp, 1, Tpad - t0, w + v0 * H, H, 1, V - v0, H, acc, sa, sb);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const int y = ld_dep(tgt + t0 + ty * 4 + a);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int64_t v = v0 + tx * 4 + b;
                if (v < V) join(a, acc[a][b], acc[a][b] == -INFINITY ? 0.0f : acc[a][b] == INFINITY ? NAN : acc[a][b] == acc[a][b] ? 1.0f : NAN);
                if (v == y) zt[t0 + ty * 4 + a] = acc[a][b];
            }
        }
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            join(a, __shfl_xor_sync(0xFFFFFFFFu, m[a], o), __shfl_xor_sync(0xFFFFFFFFu, s[a], o));
        if (tx == 0) stats[blockIdx.x * Tpad + t0 + ty * 4 + a] = make_float2(m[a], s[a]);
    }
}

// grid: 64 vocabulary rows of the piece x blocks of 64 tokens
template <typename T>
__global__ void __launch_bounds__(256)
    loss_g_kernel(const LossMeta *meta, const int32_t *tgt, const float *lse2, const float *gs, const T *x, int Hp,
                  const T *w, int64_t V, int H, float inv_temperature, int64_t Tpad, int64_t v0, int64_t piece, T *g) {
    __shared__ float sa[TK][TS + 4], sb[TK][TS + 4];
    pdl_wait();
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * TS, c0 = static_cast<int64_t>(blockIdx.x) * TS;
    const int count = ld_dep(&meta->count);
    if (t0 >= (count > 0 ? (count + kLossTile - 1) / kLossTile * kLossTile : kLossTile)) return;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4];
    tile_product(x + t0 * Hp, Hp, 1, Tpad - t0, w + (v0 + c0) * H, H, 1, V - v0 - c0, H, acc, sa, sb);
    const float sc = ld_dep(&meta->scale);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const int64_t t = t0 + ty * 4 + a;
        const int y = ld_dep(tgt + t);
        const float l = ld_dep(lse2 + t), d = ld_dep(gs + t) * sc;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int64_t v = v0 + c0 + tx * 4 + b;
            const float p = exp2f(fmaf(acc[a][b], kLog2e * inv_temperature, -l)) - (v == y ? 1.0f : 0.0f);
            put_rn(g + t * piece + c0 + tx * 4 + b, v < V ? p * d : 0.0f);
        }
    }
}

// part (+)= g w over a piece; grid: 64 columns x 64 tokens
template <typename T>
__global__ void __launch_bounds__(256)
    loss_gw_kernel(const LossMeta *meta, const T *g, int64_t piece, const T *w, int64_t V, int H, int64_t v0, bool first,
                   int64_t Tpad, float *part) {
    __shared__ float sa[TK][TS + 4], sb[TK][TS + 4];
    pdl_wait();
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * TS, h0 = static_cast<int64_t>(blockIdx.x) * TS;
    if (t0 >= ld_dep(&meta->count)) return;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4];
    const int64_t kk = V - v0 < piece ? V - v0 : piece;
    tile_product(g + t0 * piece, piece, 1, Tpad - t0, w + v0 * H + h0, 1, static_cast<int64_t>(H), H - h0, kk, acc, sa, sb);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int64_t h = h0 + tx * 4 + b;
            if (h < H) {
                float *o = part + (t0 + ty * 4 + a) * H + h;
                *o = acc[a][b] + (first ? 0.0f : *o);
            }
        }
}

// dtable (+)= g^T x over a piece; grid: 64 columns x 64 vocabulary rows
template <typename T, typename O>
__global__ void __launch_bounds__(256)
    loss_gx_kernel(const LossMeta *meta, const T *g, int64_t piece, const T *x, int Hp, int64_t V, int H, int64_t v0,
                   bool accumulate, O *dtable) {
    __shared__ float sa[TK][TS + 4], sb[TK][TS + 4];
    pdl_wait();
    const int64_t c0 = static_cast<int64_t>(blockIdx.y) * TS, h0 = static_cast<int64_t>(blockIdx.x) * TS;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4];
    tile_product(g + c0, 1, piece, V - v0 - c0, x + h0, 1, static_cast<int64_t>(Hp), H - h0,
                 static_cast<int64_t>(ld_dep(&meta->count)), acc, sa, sb);
    const float u = ld_dep(&meta->unscale);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int64_t v = v0 + c0 + ty * 4 + a, h = h0 + tx * 4 + b;
            if (v < V && h < H) {
                O *o = dtable + v * H + h;
                put_rn(o, acc[a][b] * u + (accumulate ? wide(*o) : 0.0f));
            }
        }
}

template <typename T>
cudaError_t stats(const LossArgs &a, const LossPlan &p, cudaStream_t stream) {
    return launch_pdl(loss_stats_kernel<T>, dim3(static_cast<unsigned>(p.vt), static_cast<unsigned>(p.Tpad / TS)), dim3(256),
                      0, stream, reinterpret_cast<const LossMeta *>(a.ws + p.off_meta),
                      reinterpret_cast<const int32_t *>(a.ws + p.off_tgt), reinterpret_cast<const T *>(a.ws + p.off_x),
                      p.Hp, static_cast<const T *>(a.t.data), p.V, p.H, a.inv_temperature, p.Tpad,
                      reinterpret_cast<float2 *>(a.ws + p.off_stats), reinterpret_cast<float *>(a.ws + p.off_zt));
}

template <typename T>
cudaError_t products(const LossArgs &a, const LossPlan &p, cudaStream_t stream) {
    const LossMeta *meta = reinterpret_cast<const LossMeta *>(a.ws + p.off_meta);
    const T *x = reinterpret_cast<const T *>(a.ws + p.off_x), *w = static_cast<const T *>(a.t.data);
    T *g = reinterpret_cast<T *>(a.ws + p.off_g);
    float *part = reinterpret_cast<float *>(a.ws + p.off_part);
    const unsigned ht = static_cast<unsigned>((p.H + TS - 1) / TS), tt = static_cast<unsigned>(p.Tpad / TS);
    for (int64_t v0 = 0; v0 < p.V; v0 += p.piece) {
        const unsigned vt = static_cast<unsigned>(((p.V - v0 < p.piece ? p.V - v0 : p.piece) + TS - 1) / TS);
        cudaError_t e = launch_pdl(loss_g_kernel<T>, dim3(vt, tt), dim3(256), 0, stream, meta,
                                   reinterpret_cast<const int32_t *>(a.ws + p.off_tgt),
                                   reinterpret_cast<const float *>(a.ws + p.off_lse2),
                                   reinterpret_cast<const float *>(a.ws + p.off_gs), x, p.Hp, w, p.V, p.H,
                                   a.inv_temperature, p.Tpad, v0, p.piece, g);
        if (e == cudaSuccess && a.dx)
            e = launch_pdl(loss_gw_kernel<T>, dim3(ht, tt), dim3(256), 0, stream, meta, static_cast<const T *>(g), p.piece,
                           w, p.V, p.H, v0, v0 == 0, p.Tpad, part);
        if (e == cudaSuccess && a.dtable) {
            if (a.dtable_dtype == LHS_F32)
                e = launch_pdl(loss_gx_kernel<T, float>, dim3(ht, vt), dim3(256), 0, stream, meta,
                               static_cast<const T *>(g), p.piece, x, p.Hp, p.V, p.H, v0, a.accumulate,
                               static_cast<float *>(a.dtable));
            else
                e = launch_pdl(loss_gx_kernel<T, T>, dim3(ht, vt), dim3(256), 0, stream, meta, static_cast<const T *>(g),
                               p.piece, x, p.Hp, p.V, p.H, v0, a.accumulate, static_cast<T *>(a.dtable));
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_loss_stats(const LossArgs &a, const LossPlan &p, cudaStream_t stream) {
    return p.bf16 ? stats<__nv_bfloat16>(a, p, stream) : stats<__half>(a, p, stream);
}
cudaError_t launch_loss_products(const LossArgs &a, const LossPlan &p, cudaStream_t stream) {
    return p.bf16 ? products<__nv_bfloat16>(a, p, stream) : products<__half>(a, p, stream);
}

}  // namespace lhs
