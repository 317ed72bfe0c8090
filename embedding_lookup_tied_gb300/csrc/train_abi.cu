// train_abi.cu — the C-ABI boundary of the cross entropy over the tied table,
// its gradient and the lookup's gradient: argument checks, then the launchers.
#include <cmath>
#include <initializer_list>

#include "train.cuh"

namespace lhs {
namespace {

constexpr int64_t kMaxLossTokens = 1ll << 24;
constexpr int64_t kMaxLookups = 1ll << 30;
constexpr int32_t kMaxTrainHidden = 65536;
constexpr int64_t kMaxStride = 1ll << 40;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int elem_size(int32_t dtype) {
    return dtype == LHS_F32 ? 4 : (dtype == LHS_F16 || dtype == LHS_BF16) ? 2 : 0;
}

// Memory of an argument: rows of row_bytes, stride bytes apart.
struct Rows {
    uintptr_t at;
    uint64_t rows, stride, row_bytes;
};
Rows bytes_of(const void *p, uint64_t n) { return {reinterpret_cast<uintptr_t>(p), p && n ? 1u : 0u, n, n}; }
Rows rows_of(const void *p, int64_t rows, int64_t stride, int64_t row, int size) {
    return {reinterpret_cast<uintptr_t>(p), p ? static_cast<uint64_t>(rows) : 0u, static_cast<uint64_t>(stride) * size,
            static_cast<uint64_t>(row) * size};
}
// Whether a row of r lies in the bytes of one that is contiguous.
bool meet(const Rows &one, const Rows &r) {
    const uintptr_t end = one.at + one.row_bytes;
    if (!one.rows || !r.rows || end <= r.at) return false;
    const uint64_t from = one.at > r.at ? one.at - r.at : 0;
    const uint64_t k = from < r.row_bytes ? 0 : (from - r.row_bytes) / r.stride + 1;  // the first row that ends behind it
    return k < r.rows && k * r.stride < end - r.at;
}
bool meet(const Rows &one, std::initializer_list<Rows> others) {
    for (const Rows &r : others)
        if (meet(one, r)) return true;
    return false;
}
Rows table_rows(const lhs_table &t) { return bytes_of(t.data, static_cast<uint64_t>(t.vocab) * t.row_bytes); }

int check_loss_table(const lhs_table *t, int64_t tokens) {
    if (!t) return LHS_ERR_INVALID_ARG;
    lhs_table again;
    const int rc = lhs_table_init(&again, t->data, t->vocab, t->hidden, t->dtype);
    if (rc) return rc;
    if (t->row_bytes != again.row_bytes) return LHS_ERR_INVALID_ARG;
    if (tokens < 0 || tokens > kMaxLossTokens || t->hidden > kMaxTrainHidden) return LHS_ERR_INVALID_ARG;
    if (t->dtype != LHS_F16 && t->dtype != LHS_BF16) return LHS_ERR_UNSUPPORTED;
    // tiles are numbered in 31 bits
    if (plan_loss(*t, tokens, true).items > 0x7FFFFFFFll - (1 << 20)) return LHS_ERR_UNSUPPORTED;
    return LHS_OK;
}

// What both calls take.
int check_loss_args(const lhs_table *t, const void *d_x, int32_t x_dtype, int64_t x_stride, int64_t tokens,
                    const int32_t *d_targets, float temperature, const void *d_ws, const int32_t *d_err) {
    const int rc = check_loss_table(t, tokens);
    if (rc) return rc;
    if (x_dtype != t->dtype || x_stride < t->hidden || x_stride > kMaxStride) return LHS_ERR_INVALID_ARG;
    if (!(std::isfinite(temperature) && temperature > 0.0f) || !std::isfinite(1.0f / temperature)) return LHS_ERR_INVALID_ARG;
    if (tokens == 0) return LHS_OK;
    if (!d_x || !aligned(d_x, 2) || !d_targets || !aligned(d_targets, 4) || !d_ws || !aligned(d_ws, 256) || !d_err ||
        !aligned(d_err, 4))
        return LHS_ERR_INVALID_ARG;
    return LHS_OK;
}

}  // namespace
}  // namespace lhs

using namespace lhs;

extern "C" {

int lhs_loss_workspace(const lhs_table *t, int64_t tokens, size_t *bytes) {
    const int rc = check_loss_table(t, tokens);
    if (rc) return rc;
    if (!bytes) return LHS_ERR_INVALID_ARG;
    *bytes = plan_loss(*t, tokens, false).bytes;
    return LHS_OK;
}

int lhs_loss_grad_workspace(const lhs_table *t, int64_t tokens, size_t *bytes) {
    const int rc = check_loss_table(t, tokens);
    if (rc) return rc;
    if (!bytes) return LHS_ERR_INVALID_ARG;
    *bytes = plan_loss(*t, tokens, true).bytes;
    return LHS_OK;
}

int lhs_loss(const lhs_table *t, const void *d_x, int32_t x_dtype, int64_t x_stride, int64_t tokens,
             const int32_t *d_targets, int32_t ignore, float temperature, float *d_loss, float *d_lse, void *d_ws,
             size_t ws_bytes, int32_t *d_err, void *stream) {
    const int rc = check_loss_args(t, d_x, x_dtype, x_stride, tokens, d_targets, temperature, d_ws, d_err);
    if (rc) return rc;
    if (tokens == 0) return LHS_OK;
    if (!d_loss || !aligned(d_loss, 4) || !d_lse || !aligned(d_lse, 4)) return LHS_ERR_INVALID_ARG;
    const LossPlan p = plan_loss(*t, tokens, false);
    if (ws_bytes < p.bytes) return LHS_ERR_BUFFER_TOO_SMALL;
    const Rows table = table_rows(*t), x = rows_of(d_x, tokens, x_stride, t->hidden, elem_size(x_dtype)),
               y = bytes_of(d_targets, 4 * tokens), loss = bytes_of(d_loss, 4 * tokens),
               lse = bytes_of(d_lse, 4 * tokens), ws = bytes_of(d_ws, p.bytes), err = bytes_of(d_err, 4);
    if (meet(loss, {table, x, y, lse, ws, err}) || meet(lse, {table, x, y, ws, err}) || meet(ws, {table, x, y, err}) ||
        meet(err, {table, x, y}))
        return LHS_ERR_INVALID_ARG;
    LossArgs a = {};
    a.t = *t;
    a.x = d_x;
    a.x_stride = x_stride;
    a.targets = d_targets;
    a.ignore = ignore;
    a.inv_temperature = 1.0f / temperature;
    a.loss = d_loss;
    a.lse = d_lse;
    a.ws = static_cast<uint8_t *>(d_ws);
    a.err = d_err;
    return cuda_status(launch_loss(a, p, static_cast<cudaStream_t>(stream)));
}

int lhs_loss_grad(const lhs_table *t, const void *d_x, int32_t x_dtype, int64_t x_stride, int64_t tokens,
                  const int32_t *d_targets, int32_t ignore, float temperature, const float *d_lse,
                  const float *d_dloss, void *d_dx, int32_t dx_dtype, int64_t dx_stride, void *d_dtable,
                  int32_t dtable_dtype, int32_t accumulate, void *d_ws, size_t ws_bytes, int32_t *d_err,
                  void *stream) {
    return lhs_loss_grad_of(t, d_x, x_dtype, x_stride, tokens, d_targets, ignore, temperature, nullptr, d_lse, d_dloss,
                            d_dx, dx_dtype, dx_stride, d_dtable, dtable_dtype, accumulate, d_ws, ws_bytes, d_err, stream);
}

int lhs_loss_grad_of(const lhs_table *t, const void *d_x, int32_t x_dtype, int64_t x_stride, int64_t tokens,
                     const int32_t *d_targets, int32_t ignore, float temperature, const float *d_loss,
                     const float *d_lse, const float *d_dloss, void *d_dx, int32_t dx_dtype, int64_t dx_stride,
                     void *d_dtable, int32_t dtable_dtype, int32_t accumulate, void *d_ws, size_t ws_bytes,
                     int32_t *d_err, void *stream) {
    const int rc = check_loss_args(t, d_x, x_dtype, x_stride, tokens, d_targets, temperature, d_ws, d_err);
    if (rc) return rc;
    if (accumulate != 0 && accumulate != 1) return LHS_ERR_INVALID_ARG;
    if (d_dtable && ((dtable_dtype != t->dtype && dtable_dtype != LHS_F32) || !aligned(d_dtable, 16)))
        return LHS_ERR_INVALID_ARG;
    if (d_dx && ((dx_dtype != t->dtype && dx_dtype != LHS_F32) || dx_stride < t->hidden || dx_stride > kMaxStride ||
                 !aligned(d_dx, elem_size(dx_dtype))))
        return LHS_ERR_INVALID_ARG;
    if (tokens > 0) {
        if (!d_dx && !d_dtable) return LHS_ERR_INVALID_ARG;
        if (!d_lse || !aligned(d_lse, 4) || !d_dloss || !aligned(d_dloss, 4) || !aligned(d_loss, 4)) return LHS_ERR_INVALID_ARG;
    }
    const LossPlan p = plan_loss(*t, tokens, true);
    const Rows table = table_rows(*t),
               dtable = bytes_of(d_dtable, static_cast<uint64_t>(t->vocab) * t->hidden * elem_size(dtable_dtype));
    if (meet(dtable, table)) return LHS_ERR_INVALID_ARG;  // also of no positions
    if (tokens > 0) {
        if (ws_bytes < p.bytes) return LHS_ERR_BUFFER_TOO_SMALL;
        const Rows x = rows_of(d_x, tokens, x_stride, t->hidden, elem_size(x_dtype)), y = bytes_of(d_targets, 4 * tokens),
                   lse = bytes_of(d_lse, 4 * tokens), dloss = bytes_of(d_dloss, 4 * tokens), loss = bytes_of(d_loss, 4 * tokens),
                   dx = rows_of(d_dx, tokens, dx_stride, t->hidden, elem_size(dx_dtype)), ws = bytes_of(d_ws, p.bytes),
                   err = bytes_of(d_err, 4);
        // (dx may lie over x, which the first kernel has read)
        if (meet(dtable, {x, y, loss, lse, dloss, dx, ws, err}) || meet(ws, {table, x, y, loss, lse, dloss, dx, err}) ||
            meet(err, {table, x, y, loss, lse, dloss, dx}) || meet(table, dx) || meet(y, dx) || meet(loss, dx) ||
            meet(lse, dx) || meet(dloss, dx))
            return LHS_ERR_INVALID_ARG;
    }
    LossArgs a = {};
    a.t = *t;
    a.x = d_x;
    a.x_stride = x_stride;
    a.targets = d_targets;
    a.ignore = ignore;
    a.inv_temperature = 1.0f / temperature;
    a.lse_in = d_lse;
    a.loss_in = d_loss;
    a.dloss = d_dloss;
    a.dx = d_dx;
    a.dx_dtype = dx_dtype;
    a.dx_stride = dx_stride;
    a.dtable = d_dtable;
    a.dtable_dtype = dtable_dtype;
    a.accumulate = accumulate != 0;
    a.ws = static_cast<uint8_t *>(d_ws);
    a.err = d_err;
    return cuda_status(launch_loss_grad(a, p, static_cast<cudaStream_t>(stream)));
}

int64_t lhs_embed_grad_workspace(int64_t vocab, int32_t hidden, int64_t n) {
    if (vocab < 1 || vocab > 0x7FFFFFFFll || hidden < 1 || hidden > kMaxTrainHidden || n < 0 || n > kMaxLookups) return -1;
    return static_cast<int64_t>(embed_grad_workspace(hidden, n));
}

int lhs_embed_grad(int64_t vocab, int32_t hidden, const int32_t *d_ids, int64_t n, int32_t ignore, float scale,
                   const void *d_dout, int32_t dout_dtype, int64_t dout_stride, void *d_dtable, int32_t dtable_dtype,
                   int32_t accumulate, void *d_ws, size_t ws_bytes, int32_t *d_err, void *stream) {
    const int64_t need = lhs_embed_grad_workspace(vocab, hidden, n);
    if (need < 0 || !std::isfinite(scale) || (accumulate != 0 && accumulate != 1)) return LHS_ERR_INVALID_ARG;
    const int es = elem_size(dout_dtype);
    if (!es || dout_stride < hidden || dout_stride > kMaxStride || !elem_size(dtable_dtype)) return LHS_ERR_INVALID_ARG;
    if (!d_dtable || !aligned(d_dtable, 16)) return LHS_ERR_INVALID_ARG;
    if (n > 0) {
        if (!d_ids || !aligned(d_ids, 4) || !d_dout || !aligned(d_dout, es) || !d_ws || !aligned(d_ws, 256) || !d_err ||
            !aligned(d_err, 4))
            return LHS_ERR_INVALID_ARG;
        if (ws_bytes < static_cast<size_t>(need)) return LHS_ERR_BUFFER_TOO_SMALL;
        // ids that change while they are sorted would be moved to places that were not counted
        const Rows dout = rows_of(d_dout, n, dout_stride, hidden, es), ids = bytes_of(d_ids, 4 * n),
                   dtable = bytes_of(d_dtable, static_cast<uint64_t>(vocab) * hidden * elem_size(dtable_dtype)),
                   ws = bytes_of(d_ws, need), err = bytes_of(d_err, 4);
        if (meet(dtable, {dout, ids, ws, err}) || meet(ws, {dout, ids, err}) || meet(err, {dout, ids}))
            return LHS_ERR_INVALID_ARG;
    }
    if (n == 0 && accumulate) return LHS_OK;
    EmbedGradArgs a = {vocab, hidden, d_ids, n, ignore, scale, d_dout, dout_dtype, dout_stride, d_dtable, dtable_dtype,
                       accumulate != 0, static_cast<uint8_t *>(d_ws), d_err};
    return cuda_status(launch_embed_grad(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
