// i8_rows.cu — rows quantised to int8 codes with one scale each
// (lhs_i8_quantize), by the i8 wire format's rule (ADR-0009 "Wire Format
// Evolution", Wire Layout): scale = f32(max|x| / 127), code = clamp(rne(f32(x
// / scale)), -127, 127).
#include "decode.cuh"

namespace lhs {
namespace {

constexpr int kThreads = 256;

// One CTA per row: max|x| and whether all values are finite, then the codes.
template <int DT>
__global__ void __launch_bounds__(kThreads)
    i8_quantize_kernel(const lhs_i8 t, const typename Elem<DT>::T *x, int64_t x_stride, int32_t *err) {
    using E = Elem<DT>;
    __shared__ float sm_m[kThreads / 32];
    __shared__ int sm_f[kThreads / 32];
    pdl_trigger();
    pdl_wait();
    for (int64_t r = blockIdx.x; r < t.rows; r += gridDim.x) {
        const typename E::T *row = x + r * x_stride;
        float m = 0.0f;
        int bad = 0;
        for (int j = threadIdx.x; j < t.hidden; j += kThreads) {
            const float v = E::widen(ld_dep(row + j));
            if (isfinite(v)) m = fmaxf(m, fabsf(v));
            else bad = 1;
        }
        block_max_or(m, bad, sm_m, sm_f);
        const float scale = bad ? 0.0f : __fdiv_rn(m, 127.0f);
        const float rcp = __frcp_rn(scale);
        int8_t *out = const_cast<int8_t *>(t.codes) + r * t.stride;
        for (int j = threadIdx.x; j < t.hidden; j += kThreads)
            out[j] = static_cast<int8_t>(i8_code(E::widen(ld_dep(row + j)), scale, rcp));
        if (threadIdx.x == 0) {
            *reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(const_cast<float *>(t.scales)) +
                                       r * t.scale_stride) = scale;
            if (bad) set_err(err, LHS_ERRBIT_NONFINITE);
        }
    }
}

template <int DT>
cudaError_t launch(const lhs_i8 &t, const void *x, int64_t x_stride, int32_t *err, cudaStream_t stream) {
    const int64_t grid = t.rows < (1 << 20) ? t.rows : (1 << 20);
    return launch_pdl(i8_quantize_kernel<DT>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, t,
                      static_cast<const typename Elem<DT>::T *>(x), x_stride, err);
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
