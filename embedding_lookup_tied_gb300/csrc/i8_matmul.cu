// i8_matmul.cu — the lm_head as a product in 8 bits: logits[t][c] =
// (sum_j a[t][j] w[c][j]) * a_scale[t] * w_scale[c], integers summed exactly
// (ADR-0008 "Remote Embeddings and lm_head Service", POST /v1/logits, over a
// table and residuals in the i8 form of ADR-0009 "Wire Format Evolution").
#include <cuda_bf16.h>

#include "decode.cuh"

namespace lhs {
namespace {

constexpr int kPrepThreads = 256;

__host__ __device__ constexpr int64_t align_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// Workspace: the tokens' codes [tokens][kpad] (zeros past hidden), then their
// scales.
int64_t kpad_of(int hidden) { return align_up(hidden, 64); }
int64_t scales_offset(int hidden, int64_t tokens) { return align_up(tokens * kpad_of(hidden), 256); }

// Where a coded token set is a message, whether its header names another
// seq_len (the words lie before the first position).
__device__ __forceinline__ bool message_mismatch(const lhs_i8 &a) {
    if (!a.header) return false;
    const uint8_t *buf = reinterpret_cast<const uint8_t *>(a.scales) - a.header;
    return ld_dep(reinterpret_cast<const uint32_t *>(buf) + 1) != static_cast<uint32_t>(a.rows);
}
// The scale of coded token r; NaN (and MALFORMED) where its message is not
// one the product can take.  Called by one thread.
__device__ __forceinline__ float coded_scale(const lhs_i8 &a, int64_t r, int32_t *err) {
    const uint8_t *p = reinterpret_cast<const uint8_t *>(a.scales) + r * a.scale_stride;
    float s = ld_dep(reinterpret_cast<const float *>(p));
    if (a.header && (message_mismatch(a) || ld_dep(reinterpret_cast<const float *>(p) + 1) != 0.0f)) {
        set_err(err, LHS_ERRBIT_MALFORMED);
        s = __int_as_float(0x7FC00000);
    }
    return s;
}

// One CTA per token: its codes and its scale into the workspace.
template <int DT>
__global__ void __launch_bounds__(kPrepThreads)
    i8_prep_wide_kernel(const typename Elem<DT>::T *x, int64_t x_stride, int64_t tokens, int hidden, int kpad,
                        int8_t *codes, float *scales, int32_t *err) {
    using E = Elem<DT>;
    __shared__ float sm_m[kPrepThreads / 32];
    __shared__ int sm_f[kPrepThreads / 32];
    pdl_trigger();
    pdl_wait();
    for (int64_t r = blockIdx.x; r < tokens; r += gridDim.x) {
        const typename E::T *row = x + r * x_stride;
        float m = 0.0f;
        int bad = 0;
        for (int j = threadIdx.x; j < hidden; j += kPrepThreads) {
            const float v = E::widen(ld_dep(row + j));
            if (isfinite(v)) m = fmaxf(m, fabsf(v));
            else bad = 1;
        }
        block_max_or(m, bad, sm_m, sm_f);
        const float scale = bad ? 0.0f : __fdiv_rn(m, 127.0f);
        const float rcp = __frcp_rn(scale);
        for (int j = threadIdx.x; j < kpad; j += kPrepThreads)
            codes[r * kpad + j] =
                j < hidden ? static_cast<int8_t>(i8_code(E::widen(ld_dep(row + j)), scale, rcp)) : int8_t(0);
        if (threadIdx.x == 0) {
            scales[r] = scale;
            if (bad) set_err(err, LHS_ERRBIT_NONFINITE);
        }
    }
}

__global__ void __launch_bounds__(kPrepThreads)
    i8_prep_coded_kernel(const lhs_i8 a, int kpad, int8_t *codes, float *scales, int32_t *err) {
    pdl_trigger();
    pdl_wait();
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int8_t *row = a.codes + r * a.stride;
        for (int j = threadIdx.x; j < kpad; j += kPrepThreads)
            codes[r * kpad + j] = j < a.hidden ? ld_dep(row + j) : int8_t(0);
        if (threadIdx.x == 0) scales[r] = coded_scale(a, r, err);
    }
}

template <int OD>
__device__ __forceinline__ void store_out(void *out, int64_t i, float v) {
    if (OD == LHS_F32) reinterpret_cast<float *>(out)[i] = v;
    else if (OD == LHS_F16) reinterpret_cast<__half *>(out)[i] = __float2half_rn(v);
    else reinterpret_cast<__nv_bfloat16 *>(out)[i] = __float2bfloat16_rn(v);
}

// Tiles of 64 channels x 32 tokens, 64 codes at a time in shared memory; a
// thread sums one channel against eight tokens with four-way dot products.
constexpr int kTC = 64, kTT = 32, kTK = 64;
template <int OD>
__global__ void __launch_bounds__(256)
    i8_matmul_kernel(const lhs_i8 w, const int8_t *codes, const float *scales, int64_t tokens, int kpad, void *out,
                     int64_t out_stride) {
    __shared__ int ws[kTC][kTK / 4 + 1];
    __shared__ int as[kTT][kTK / 4];
    const int c = threadIdx.x & (kTC - 1), g = threadIdx.x / kTC;
    pdl_trigger();
    pdl_wait();
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kTC;
    for (int64_t t0 = static_cast<int64_t>(blockIdx.y) * kTT; t0 < tokens;
         t0 += static_cast<int64_t>(gridDim.y) * kTT) {
        int acc[8] = {};
        for (int k0 = 0; k0 < kpad; k0 += kTK) {
            __syncthreads();
            for (int i = threadIdx.x; i < kTC * kTK / 4; i += 256) {
                const int r = i / (kTK / 4), q = i % (kTK / 4);
                uint32_t v = 0;
                const int k = k0 + q * 4;
                if (c0 + r < w.rows && k < w.hidden) {  // rows are 16-byte aligned, so the word lies inside the row's stride
                    v = __ldg(reinterpret_cast<const uint32_t *>(w.codes + (c0 + r) * w.stride + k));
                    if (w.hidden - k < 4) v &= (1u << (8 * (w.hidden - k))) - 1u;
                }
                ws[r][q] = static_cast<int>(v);
            }
            for (int i = threadIdx.x; i < kTT * kTK / 4; i += 256) {
                const int r = i / (kTK / 4), q = i % (kTK / 4);
                as[r][q] = t0 + r < tokens
                               ? __ldcg(reinterpret_cast<const int *>(codes + (t0 + r) * kpad + k0) + q)
                               : 0;
            }
            __syncthreads();
#pragma unroll
            for (int q = 0; q < kTK / 4; ++q) {
                const int wv = ws[c][q];
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = __dp4a(wv, as[g * 8 + i][q], acc[i]);
            }
        }
        if (c0 + c < w.rows) {
            const float wsc = __ldg(reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(w.scales) +
                                                                    (c0 + c) * w.scale_stride));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t t = t0 + g * 8 + i;
                if (t < tokens)
                    store_out<OD>(out, t * out_stride + c0 + c,
                                  __fmul_rn(__fmul_rn(static_cast<float>(acc[i]), __ldcg(scales + t)), wsc));
            }
        }
    }
}

template <int DT>
cudaError_t prep_wide(const I8Tokens &a, int hidden, int kpad, int8_t *codes, float *scales, int32_t *err,
                      unsigned grid, cudaStream_t stream) {
    return launch_pdl(i8_prep_wide_kernel<DT>, dim3(grid), dim3(kPrepThreads), 0, stream,
                      static_cast<const typename Elem<DT>::T *>(a.x), a.x_stride, a.rows, hidden, kpad, codes,
                      scales, err);
}

}  // namespace

size_t i8_matmul_workspace(const lhs_i8 &table, int64_t tokens) {
    return static_cast<size_t>(scales_offset(table.hidden, tokens) + align_up(tokens * 4, 256));
}

cudaError_t launch_i8_matmul(const I8Tokens &a, const lhs_i8 &table, void *out, int32_t out_dtype,
                             int64_t out_stride, void *ws, int32_t *err, cudaStream_t stream) {
    const int kpad = static_cast<int>(kpad_of(table.hidden));
    int8_t *codes = static_cast<int8_t *>(ws);
    float *scales = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + scales_offset(table.hidden, a.rows));
    const unsigned pg = static_cast<unsigned>(a.rows < (1 << 20) ? a.rows : (1 << 20));
    cudaError_t e;
    if (!a.x) e = launch_pdl(i8_prep_coded_kernel, dim3(pg), dim3(kPrepThreads), 0, stream, a.coded, kpad, codes,
                             scales, err);
    else if (a.x_dtype == LHS_F32) e = prep_wide<LHS_F32>(a, table.hidden, kpad, codes, scales, err, pg, stream);
    else if (a.x_dtype == LHS_F16) e = prep_wide<LHS_F16>(a, table.hidden, kpad, codes, scales, err, pg, stream);
    else e = prep_wide<LHS_BF16>(a, table.hidden, kpad, codes, scales, err, pg, stream);
    if (e != cudaSuccess) return e;
    const int64_t ty = (a.rows + kTT - 1) / kTT;
    const dim3 grid(static_cast<unsigned>((table.rows + kTC - 1) / kTC), static_cast<unsigned>(ty < 65535 ? ty : 65535));
    if (out_dtype == LHS_F32)
        return launch_pdl(i8_matmul_kernel<LHS_F32>, grid, dim3(256), 0, stream, table, codes, scales, a.rows, kpad,
                          out, out_stride);
    if (out_dtype == LHS_F16)
        return launch_pdl(i8_matmul_kernel<LHS_F16>, grid, dim3(256), 0, stream, table, codes, scales, a.rows, kpad,
                          out, out_stride);
    return launch_pdl(i8_matmul_kernel<LHS_BF16>, grid, dim3(256), 0, stream, table, codes, scales, a.rows, kpad,
                      out, out_stride);
}

}  // namespace lhs
