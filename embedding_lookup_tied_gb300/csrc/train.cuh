// train.cuh — plans and launcher prototypes of the cross entropy over the tied
// table, its gradient, and the gradient of the lookup (loss.cu, loss_gemm.cu,
// embed_grad.cu; checked in train_abi.cu).
#pragma once

#include <cuda_bf16.h>

#include "decode.cuh"
#include "loss_queue.cuh"

namespace lhs {

// What one call needs to know on the device, written by its first kernel.
struct LossMeta {
    int32_t count;    // positions that take part
    float scale;      // g is multiplied by this power of two before it is rounded
    float unscale;    // its inverse
};

// Workspace of one call.  The positions that take part are numbered 0 .. count
// in their order ("compact"); rows of x that do not are never read again.
struct LossPlan : LossQueue {
    int64_t T;              // positions
    int32_t Hp;             // hidden rounded up to 8 (rows of whole 16-byte words)
    bool bf16, grad;
    size_t off_meta;        // LossMeta
    size_t off_act;         // int32 [Tpad]: position of a compact row, -1 past count
    size_t off_tgt;         // int32 [Tpad]: its target, -1 past count
    size_t off_x;           // [Tpad x Hp]: its residual, zeros past hidden and count
    size_t off_w;           // [V x Hp]: the table, where its rows are not whole 16-byte words
    size_t off_sync;        // uint32 [n_sync]: what CTAs tell one another; 0 at the start
    // loss
    size_t off_stats;       // float2 [vt x kLossParts x Tpad]: maximum of a part, sum of its other exponentials
    size_t off_zt;          // f32 [Tpad]: the target's logit
    // gradient
    size_t off_pos;         // int32 [T]: compact row of a position, -1
    size_t off_lse;         // f32 [Tpad]: lse, +inf past count
    size_t off_gs;          // f32 [Tpad]: dloss / temperature, 0 past count
    bool apart;             // the targets' entries are kept apart
    size_t off_em;          // f32 [Tpad]: exp(-loss) - 1, where the losses are given
    size_t off_coef;        // f32 [Tpad]: the part of a target's entry that is, 0 past count
    size_t off_slot;        // int32 [V + vt]: the row's sum in off_rows, or -1; whether a row of a tile has one, or -1
    size_t off_rows;        // f32 [min(T, V) x rows_pitch]: sums of coef x over a target's positions
    size_t off_order;       // workspace of their order
    int64_t rows_pitch;     // hidden rounded up to a block of a tile's columns
    size_t off_g;           // [slots x Tpad x piece]: g of a piece of the vocabulary
    size_t off_part;        // f32 [splits x Tpad x part_pitch]: dx so far
    int32_t part_pitch;     // hidden rounded up to 4
    size_t bytes;
};
LossPlan plan_loss(const lhs_table &t, int64_t tokens, bool grad);

struct LossArgs {
    lhs_table t;
    const void *x;
    int64_t x_stride;
    const int32_t *targets;
    int32_t ignore;
    float inv_temperature;
    float *loss, *lse;              // loss
    const float *lse_in, *dloss;    // gradient
    const float *loss_in;           // or null
    void *dx;
    int32_t dx_dtype;
    int64_t dx_stride;
    void *dtable;
    int32_t dtable_dtype;
    bool accumulate;
    uint8_t *ws;
    int32_t *err;
};
cudaError_t launch_loss(const LossArgs &a, const LossPlan &p, cudaStream_t stream);
cudaError_t launch_loss_grad(const LossArgs &a, const LossPlan &p, cudaStream_t stream);

// The products between the first and the last kernel of a call (loss_gemm.cu).
cudaError_t launch_loss_stats(const LossArgs &a, const LossPlan &p, cudaStream_t stream);
cudaError_t launch_loss_products(const LossArgs &a, const LossPlan &p, cudaStream_t stream);

struct EmbedGradArgs {
    int64_t vocab;
    int32_t hidden;
    const int32_t *ids;
    int64_t n;
    int32_t ignore;
    float scale;
    const void *dout;
    int32_t dout_dtype;
    int64_t dout_stride;
    void *dtable;
    int32_t dtable_dtype;
    bool accumulate;
    uint8_t *ws;
    int32_t *err;
};
size_t embed_grad_workspace(int32_t hidden, int64_t n);

// rows[slot_of[v]] = sum of coef x over the positions whose target is v, in a fixed order; for the loss's
// gradient.  slot_of holds -1 beforehand, for V rows and their tiles.
struct TargetRowsArgs {
    const int32_t *targets;
    int64_t T, V;
    int32_t ignore, Hp;
    bool bf16;
    const uint16_t *x;      // packed
    const int32_t *pos;     // packed row of a position
    const float *coef;      // of a packed row
    float *rows;
    int64_t pitch;
    int32_t *slot_of;
    uint8_t *ws;            // embed_grad_workspace(Hp, T)
    int32_t *err;
};
cudaError_t launch_target_rows(const TargetRowsArgs &a, cudaStream_t stream);
cudaError_t launch_embed_grad(const EmbedGradArgs &a, cudaStream_t stream);
// Zeroes `bytes` at a 16-byte aligned address.
cudaError_t launch_zero(void *p, size_t bytes, cudaStream_t stream);

// p - 1 for the logarithm l of a probability p.  Above 1/2 the difference would lose what p
// was rounded by.
__device__ __forceinline__ float p_minus_1(float l, float p) { return p <= 0.5f ? p - 1.0f : expm1f(l); }

// A value rounded to an output type (beyond the f16 range +-inf).
__device__ __forceinline__ void put_rn(float *p, float v) { *p = v; }
__device__ __forceinline__ void put_rn(__half *p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put_rn(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ float wide(float v) { return v; }
__device__ __forceinline__ float wide(__half v) { return __half2float(v); }
__device__ __forceinline__ float wide(__nv_bfloat16 v) { return __bfloat162float(v); }

}  // namespace lhs
