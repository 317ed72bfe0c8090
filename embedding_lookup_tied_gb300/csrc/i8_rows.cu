// i8_rows.cu — rows quantised to int8 codes with one scale each
// (lhs_i8_quantize), by the i8 wire format's rule (ADR-0009 "Wire Format
// Evolution", Wire Layout): scale = f32(max|x| / 127), code = clamp(rne(f32(x
// / scale)), -127, 127).
//
// A value is read once (2 or 4 bytes) and its code written (1), so HBM is the
// floor.  A row belongs to a warp (up to 1,024 values) or to a CTA of eight, whose
// lanes take four values at a time and keep them in registers between the
// maximum and the codes: up to eight fours a lane; what is beyond, in rows of more
// than 8,192 values, is read again from L2.
//
// What bounds it: issue slots.  151,936 x 896, a warp to a row: 133 us from f32
// (76% of the HBM rate) and 128 us from bf16 (48%), where 28.6 instructions a value
// take 79% of the slots (about 11 of them the quotient, the tests for its borders
// and the packing; the rest is widening, the maximum, predicates and the loop in
// fours).  A CTA to a row adds two barriers without a load under way: 262,144 x
// 5,376 from f16 1.53 ms (41%), 65,536 x 5,376 from f32 445 us, for which the wire
// format's bulk encoder, the same rule in eights out of a ring of rows, takes 285.
#include "i8_common.cuh"

namespace lhs {
namespace {

constexpr int kThreads = 256;
constexpr int kSteps = 8;  // fours a lane keeps

struct Out {
    int8_t *codes;
    int64_t stride;
    uint8_t *scales;
    int64_t scale_stride;
    bool words;  // four codes may be stored at once
};

// Four values as they are stored (zeros past hidden), and widened.
template <int DT>
struct Four {
    using E = Elem<DT>;
    using T = typename E::T;
    uint32_t w[sizeof(T)];  // 16 or 8 bytes
    __device__ __forceinline__ void load(const T *row, int j, int hidden, bool vec) {
        if (vec && j + 4 <= hidden) {
            if (DT == LHS_F32) {
                const uint4 u = ld_dep(reinterpret_cast<const uint4 *>(row + j));
                w[0] = u.x; w[1] = u.y; w[sizeof(T) - 2] = u.z; w[sizeof(T) - 1] = u.w;
            } else {
                const uint2 u = ld_dep(reinterpret_cast<const uint2 *>(row + j));
                w[0] = u.x; w[1] = u.y;
            }
        } else {
            uint32_t e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e[i] = 0;
                if (j + i < hidden) {
                    const T x = ld_dep(row + j + i);
                    if constexpr (DT == LHS_F32) e[i] = __float_as_uint(x);
                    else e[i] = x;
                }
            }
            if (DT == LHS_F32) {
                w[0] = e[0]; w[1] = e[1]; w[sizeof(T) - 2] = e[2]; w[sizeof(T) - 1] = e[3];
            } else {
                w[0] = e[0] | e[1] << 16; w[1] = e[2] | e[3] << 16;
            }
        }
    }
    __device__ __forceinline__ void widen(float (&v)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == LHS_F32) v[i] = __uint_as_float(w[i]);
            else v[i] = E::widen(static_cast<T>(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu));
        }
    }
};

__device__ __forceinline__ void store4(const Out &o, int8_t *row, int j, int hidden, uint32_t w) {
    if (o.words && j + 4 <= hidden) {
        *reinterpret_cast<uint32_t *>(row + j) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (j + i < hidden) row[j + i] = static_cast<int8_t>(w >> (8 * i));
    }
}

// LANES: threads to a row, 32 or kThreads.
template <int DT, int LANES>
__global__ void __launch_bounds__(kThreads, DT == LHS_F32 ? 3 : 4)
    i8_quantize_kernel(const Out out, const typename Elem<DT>::T *x, int64_t x_stride, bool vec, int64_t rows,
                       int hidden, int32_t *err) {
    __shared__ float sm_m[kThreads / 32];
    __shared__ int sm_f[kThreads / 32];
    constexpr int kRows = kThreads / LANES;
    const int lane = threadIdx.x % LANES;
    pdl_trigger();
    pdl_wait();
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < rows; r0 += static_cast<int64_t>(gridDim.x) * kRows) {
        const int64_t r = r0 + threadIdx.x / LANES;
        if (LANES == 32 && r >= rows) continue;
        const typename Elem<DT>::T *row = x + r * x_stride;
        Four<DT> keep[kSteps];
        float m = 0.0f, z = 0.0f;  // max|x|, and NaN where a value is not finite (0 x is)
        auto scan = [&](const Four<DT> &f) {
            float w[4];
            f.widen(w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m = fmaxf(m, fabsf(w[i]));
                z = __fmaf_rn(w[i], 0.0f, z);
            }
        };
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int j = 4 * (lane + s * LANES);
            if (j < hidden) keep[s].load(row, j, hidden, vec);
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            if (4 * (lane + s * LANES) < hidden) scan(keep[s]);
        for (int j = 4 * (lane + kSteps * LANES); j < hidden; j += 4 * LANES) {
            Four<DT> f;
            f.load(row, j, hidden, vec);
            scan(f);
        }
        int bad = z != z ? 1 : 0;
        if (LANES == 32) {
            m = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m)));
            bad = __any_sync(0xFFFFFFFFu, bad);
        } else {
            block_max_or(m, bad, sm_m, sm_f);
        }
        const float scale = bad ? 0.0f : __fdiv_rn(m, 127.0f);
        const float rcp = __frcp_rn(scale);
        int8_t *codes = out.codes + r * out.stride;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int j = 4 * (lane + s * LANES);
            if (j >= hidden) break;
            float w[4];
            keep[s].widen(w);
            store4(out, codes, j, hidden, i8_code4(w, scale, rcp));
        }
        for (int j = 4 * (lane + kSteps * LANES); j < hidden; j += 4 * LANES) {
            Four<DT> f;
            f.load(row, j, hidden, vec);
            float w[4];
            f.widen(w);
            store4(out, codes, j, hidden, i8_code4(w, scale, rcp));
        }
        if (lane == 0) {
            *reinterpret_cast<float *>(out.scales + r * out.scale_stride) = scale;
            if (bad) set_err(err, LHS_ERRBIT_NONFINITE);
        }
    }
}

template <int DT>
cudaError_t launch(const lhs_i8 &t, const void *x, int64_t x_stride, int32_t *err, cudaStream_t stream) {
    using T = typename Elem<DT>::T;
    const bool vec = reinterpret_cast<uintptr_t>(x) % (4 * sizeof(T)) == 0 && x_stride % 4 == 0;
    const Out out = {const_cast<int8_t *>(t.codes), t.stride,
                     reinterpret_cast<uint8_t *>(const_cast<float *>(t.scales)), t.scale_stride,
                     reinterpret_cast<uintptr_t>(t.codes) % 4 == 0 && t.stride % 4 == 0};
    const bool warp = t.hidden <= 4 * 32 * kSteps;
    const int64_t ctas = warp ? (t.rows + kThreads / 32 - 1) / (kThreads / 32) : t.rows;
    const dim3 grid(static_cast<unsigned>(ctas < (1 << 20) ? ctas : (1 << 20)));
    if (warp)
        return launch_pdl(i8_quantize_kernel<DT, 32>, grid, dim3(kThreads), 0, stream, out, static_cast<const T *>(x),
                          x_stride, vec, t.rows, t.hidden, err);
    return launch_pdl(i8_quantize_kernel<DT, kThreads>, grid, dim3(kThreads), 0, stream, out,
                      static_cast<const T *>(x), x_stride, vec, t.rows, t.hidden, err);
}

}  // namespace

cudaError_t launch_i8_quantize(const lhs_i8 &t, const void *x, int32_t x_dtype, int64_t x_stride, int32_t *err,
                               cudaStream_t stream) {
    switch (x_dtype) {
    case LHS_F32: return launch<LHS_F32>(t, x, x_stride, err, stream);
    case LHS_F16: return launch<LHS_F16>(t, x, x_stride, err, stream);
    default: return launch<LHS_BF16>(t, x, x_stride, err, stream);
    }
}

}  // namespace lhs
