// decode.cuh — launcher prototypes of the 8-bit lm_head product and of token
// sampling (i8_rows.cu, i8_gemv.cu, i8_matmul.cu, sample.cu; checked in
// decode_abi.cu).
#pragma once

#include "lhs_internal.cuh"

namespace lhs {

// Element j of a row of an activation or logits type.
template <int DT>
struct Elem;
template <>
struct Elem<LHS_F32> {
    using T = float;
    static __device__ __forceinline__ float widen(T v) { return v; }
};
template <>
struct Elem<LHS_F16> {
    using T = uint16_t;
    static __device__ __forceinline__ float widen(T v) { return f16_bits_to_f32(v); }
};
template <>
struct Elem<LHS_BF16> {
    using T = uint16_t;
    static __device__ __forceinline__ float widen(T v) { return bf16_bits_to_f32(v); }
};

// Wide tokens of a product (codes == null) or coded ones.
struct I8Tokens {
    const void *x;          // wide rows
    int32_t x_dtype;
    int64_t x_stride;       // elements
    lhs_i8 coded;           // coded rows, where x is null
    int64_t rows;
};

cudaError_t launch_i8_quantize(const lhs_i8 &t, const void *x, int32_t x_dtype, int64_t x_stride, int32_t *err,
                               cudaStream_t stream);
size_t i8_matmul_workspace(const lhs_i8 &table, int64_t tokens);
cudaError_t launch_i8_matmul(const I8Tokens &a, const lhs_i8 &table, void *out, int32_t out_dtype,
                             int64_t out_stride, void *ws, int32_t *err, cudaStream_t stream);

struct SampleParams {
    const void *logits;
    int64_t stride;
    int64_t rows;
    int32_t vocab;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *ids;
    float *probs;
    int32_t *err;
};
cudaError_t launch_sample(const SampleParams &p, int32_t dtype, cudaStream_t stream);

}  // namespace lhs
