// i8_common.cuh — what the two kernels of the 8-bit product share: how tokens
// are read, how the table is staged and how results are written.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "decode.cuh"

namespace lhs {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // lm_head.cu

// A stage of the table's ring: 128 rows x 128 codes, 128-byte swizzle (the
// 16-byte piece i of row r lies at piece i ^ (r & 7)).
constexpr int kStageK = 128;
constexpr int kCtaRows = 128;
constexpr int kTableStageBytes = kCtaRows * kStageK;

// Where a coded token set is a message, whether its header names another
// seq_len (the words lie before the first position).
__device__ __forceinline__ bool message_mismatch(const lhs_i8 &a) {
    const uint8_t *buf = reinterpret_cast<const uint8_t *>(a.scales) - a.header;
    return ld_dep(reinterpret_cast<const uint32_t *>(buf) + 1) != static_cast<uint32_t>(a.rows);
}
// The scale of coded token r; NaN (and MALFORMED) where its message is not
// one the product can take.  Called by one thread; err may be null.
__device__ __forceinline__ float coded_scale(const lhs_i8 &a, int64_t r, int32_t *err) {
    const uint8_t *p = reinterpret_cast<const uint8_t *>(a.scales) + r * a.scale_stride;
    float s = ld_dep(reinterpret_cast<const float *>(p));
    if (a.header && (message_mismatch(a) || ld_dep(reinterpret_cast<const float *>(p) + 1) != 0.0f)) {
        if (err) set_err(err, LHS_ERRBIT_MALFORMED);
        s = __int_as_float(0x7FC00000);
    }
    return s;
}

// Values j .. j+3 of a row (zeros past hidden).
template <int DT>
__device__ __forceinline__ void load4(const typename Elem<DT>::T *row, int j, int hidden, bool vec,
                                      float (&v)[4]) {
    using E = Elem<DT>;
    if (vec && j + 4 <= hidden) {
        if (DT == LHS_F32) {
            const float4 w = ld_dep(reinterpret_cast<const float4 *>(row + j));
            v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
        } else {
            const ushort4 w = ld_dep(reinterpret_cast<const ushort4 *>(row + j));
            v[0] = E::widen(static_cast<typename E::T>(w.x)); v[1] = E::widen(static_cast<typename E::T>(w.y));
            v[2] = E::widen(static_cast<typename E::T>(w.z)); v[3] = E::widen(static_cast<typename E::T>(w.w));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = j + i < hidden ? E::widen(ld_dep(row + j + i)) : 0.0f;
    }
}

// Four codes, their sign bits flipped (code + 128), as f16 in order: under the
// exponent byte 0x64 code + 128 is 1024 + code + 128; less 1152 it is the code,
// exactly.
__device__ __forceinline__ void widen4(uint32_t x, uint32_t &lo, uint32_t &hi) {
    const uint32_t bias = 0x64806480u;  // 1152, 1152
    const uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
    const __half2 c = *reinterpret_cast<const __half2 *>(&bias);
    const __half2 p = __hsub2(*reinterpret_cast<const __half2 *>(&a), c);
    const __half2 q = __hsub2(*reinterpret_cast<const __half2 *>(&b), c);
    lo = *reinterpret_cast<const uint32_t *>(&p);
    hi = *reinterpret_cast<const uint32_t *>(&q);
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__half *p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

inline bool make_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, uint64_t cols, uint64_t rows,
              uint64_t pitch, uint32_t box_cols, uint32_t box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {pitch};
    const cuuint32_t box[2] = {box_cols, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, type, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The streaming kernel of few tokens (i8_gemv.cu): whether it takes this
// product, and its launch.
bool i8_gemv_serves(const lhs_i8 &table, int64_t tokens);
cudaError_t launch_i8_gemv(const I8Tokens &a, const lhs_i8 &table, void *out, int32_t out_dtype,
                           int64_t out_stride, int32_t *err, const DeviceInfo &dev, cudaStream_t stream);

}  // namespace lhs
