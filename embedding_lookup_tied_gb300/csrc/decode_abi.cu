// decode_abi.cu — the C-ABI boundary of the 8-bit lm_head product and of token
// sampling: argument checks, then the launchers.
#include "decode.cuh"

namespace lhs {
namespace {

constexpr int64_t kMaxRows = 0x7FFFFFFFll;
constexpr int32_t kMaxI8Hidden = 1 << 24;
// |sum| <= hidden * 128 * 128 < 2^31 (a code may be -128)
constexpr int32_t kMaxMatmulHidden = 131071;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int elem_size(int32_t dtype) {
    return dtype == LHS_F32 ? 4 : (dtype == LHS_F16 || dtype == LHS_BF16) ? 2 : 0;
}

int check_i8(const lhs_i8 *t) {
    if (!t) return LHS_ERR_INVALID_ARG;
    if (t->rows < 0 || t->rows > kMaxRows || t->hidden < 1 || t->hidden > kMaxI8Hidden) return LHS_ERR_INVALID_ARG;
    if (t->stride < t->hidden || t->stride > (1ll << 40)) return LHS_ERR_INVALID_ARG;
    if (t->scale_stride < 4 || t->scale_stride % 4 || t->scale_stride > (1ll << 40)) return LHS_ERR_INVALID_ARG;
    if (t->header != 0 && t->header != 16 && t->header != 12) return LHS_ERR_INVALID_ARG;
    if (t->rows > 0 && (!t->codes || !t->scales || !aligned(t->scales, 4))) return LHS_ERR_INVALID_ARG;
    if (t->header && (t->stride != t->hidden + 8 || t->scale_stride != t->stride || t->hidden % 4 ||
                      (t->rows > 0 && reinterpret_cast<const uint8_t *>(t->codes) !=
                                          reinterpret_cast<const uint8_t *>(t->scales) + 8)))
        return LHS_ERR_INVALID_ARG;
    return LHS_OK;
}

int check_matmul_table(const lhs_i8 *t) {
    const int rc = check_i8(t);
    if (rc) return rc;
    if (t->header || t->hidden > kMaxMatmulHidden || t->stride % 16 || !aligned(t->codes, 16))
        return LHS_ERR_INVALID_ARG;
    return LHS_OK;
}

// The rest of both product calls, once the tokens are described.
int run_matmul(const I8Tokens &a, const lhs_i8 *table, void *d_out, int32_t out_dtype, int64_t out_stride,
               void *d_ws, size_t ws_bytes, int32_t *d_err, void *stream) {
    const int es = elem_size(out_dtype);
    if (!es || out_stride < table->rows || out_stride > (1ll << 40)) return LHS_ERR_INVALID_ARG;
    if (a.rows == 0 || table->rows == 0) return LHS_OK;
    if (!d_out || !aligned(d_out, es) || !d_ws || !aligned(d_ws, 256) || !d_err || !aligned(d_err, 4))
        return LHS_ERR_INVALID_ARG;
    if (ws_bytes < i8_matmul_workspace(*table, a.rows)) return LHS_ERR_BUFFER_TOO_SMALL;
    return cuda_status(launch_i8_matmul(a, *table, d_out, out_dtype, out_stride, d_ws, d_err,
                                        static_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace lhs

using namespace lhs;

extern "C" {

int lhs_i8_init(lhs_i8 *t, const int8_t *d_codes, int64_t stride, const float *d_scales, int64_t scale_stride,
                int64_t rows, int32_t hidden) {
    if (!t) return LHS_ERR_INVALID_ARG;
    lhs_i8 tmp = {d_codes, d_scales, rows, stride, scale_stride, hidden, 0};
    const int rc = check_i8(&tmp);
    if (rc) return rc;
    *t = tmp;
    return LHS_OK;
}

int lhs_i8_message(lhs_i8 *t, const void *d_buf, size_t buf_bytes, int32_t header, int32_t seq_len,
                   int32_t hidden) {
    if (!t || !d_buf || !aligned(d_buf, 4) || (header != 16 && header != 12)) return LHS_ERR_INVALID_ARG;
    if (hidden < 1 || hidden > kMaxI8Hidden || hidden % 4) return LHS_ERR_INVALID_ARG;
    const int64_t need = header == 16 ? lhs_wire_bytes(LHS_WIRE_I8, seq_len, hidden)
                                      : lhs_wire_response_bytes(LHS_WIRE_I8, seq_len, hidden);
    if (need < 0) return LHS_ERR_INVALID_ARG;
    if (buf_bytes < static_cast<size_t>(need)) return LHS_ERR_BUFFER_TOO_SMALL;
    const uint8_t *pos = static_cast<const uint8_t *>(d_buf) + header;
    lhs_i8 tmp = {reinterpret_cast<const int8_t *>(pos + 8), reinterpret_cast<const float *>(pos), seq_len,
                  static_cast<int64_t>(hidden) + 8, static_cast<int64_t>(hidden) + 8, hidden, header};
    const int rc = check_i8(&tmp);
    if (rc) return rc;
    *t = tmp;
    return LHS_OK;
}

int lhs_i8_quantize(const lhs_i8 *t, const void *d_x, int32_t x_dtype, int64_t x_stride, int32_t *d_err,
                    void *stream) {
    const int rc = check_i8(t);
    if (rc) return rc;
    const int es = elem_size(x_dtype);
    if (t->header || !es || x_stride < t->hidden || x_stride > (1ll << 40)) return LHS_ERR_INVALID_ARG;
    if (t->rows == 0) return LHS_OK;
    if (!d_x || !aligned(d_x, es) || !d_err || !aligned(d_err, 4)) return LHS_ERR_INVALID_ARG;
    return cuda_status(launch_i8_quantize(*t, d_x, x_dtype, x_stride, d_err, static_cast<cudaStream_t>(stream)));
}

int lhs_i8_workspace(const lhs_i8 *table, int64_t tokens, size_t *bytes) {
    const int rc = check_matmul_table(table);
    if (rc) return rc;
    if (tokens < 0 || tokens > kMaxRows || !bytes) return LHS_ERR_INVALID_ARG;
    *bytes = i8_matmul_workspace(*table, tokens);
    return LHS_OK;
}

int lhs_i8_matmul(const lhs_i8 *a, const lhs_i8 *table, void *d_out, int32_t out_dtype, int64_t out_stride,
                  void *d_ws, size_t ws_bytes, int32_t *d_err, void *stream) {
    int rc = check_matmul_table(table);
    if (rc) return rc;
    rc = check_i8(a);
    if (rc) return rc;
    if (a->hidden != table->hidden) return LHS_ERR_INVALID_ARG;
    I8Tokens tok = {};
    tok.coded = *a;
    tok.rows = a->rows;
    return run_matmul(tok, table, d_out, out_dtype, out_stride, d_ws, ws_bytes, d_err, stream);
}

int lhs_i8_logits(const lhs_i8 *table, const void *d_x, int32_t x_dtype, int64_t x_stride, int64_t tokens,
                  void *d_out, int32_t out_dtype, int64_t out_stride, void *d_ws, size_t ws_bytes, int32_t *d_err,
                  void *stream) {
    const int rc = check_matmul_table(table);
    if (rc) return rc;
    const int es = elem_size(x_dtype);
    if (!es || tokens < 0 || tokens > kMaxRows || x_stride < table->hidden || x_stride > (1ll << 40))
        return LHS_ERR_INVALID_ARG;
    if (tokens > 0 && table->rows > 0 && (!d_x || !aligned(d_x, es))) return LHS_ERR_INVALID_ARG;
    I8Tokens tok = {};
    tok.x = d_x;
    tok.x_dtype = x_dtype;
    tok.x_stride = x_stride;
    tok.rows = tokens;
    return run_matmul(tok, table, d_out, out_dtype, out_stride, d_ws, ws_bytes, d_err, stream);
}

int lhs_sample(const void *d_logits, int32_t dtype, int64_t stride, int64_t rows, int64_t vocab, const float *d_u,
               const float *d_temperature, const int32_t *d_top_k, const float *d_top_p, const float *d_min_p,
               int32_t *d_ids, float *d_probs, int32_t *d_err, void *stream) {
    const int es = elem_size(dtype);
    if (!es || rows < 0 || rows > kMaxRows || vocab < 1 || vocab > kMaxRows || stride < vocab ||
        stride > (1ll << 40))
        return LHS_ERR_INVALID_ARG;
    if (rows == 0) return LHS_OK;
    if (!d_logits || !aligned(d_logits, es) || !d_u || !d_ids || !d_err) return LHS_ERR_INVALID_ARG;
    for (const void *q : {static_cast<const void *>(d_u), static_cast<const void *>(d_temperature),
                          static_cast<const void *>(d_top_k), static_cast<const void *>(d_top_p),
                          static_cast<const void *>(d_min_p), static_cast<const void *>(d_ids),
                          static_cast<const void *>(d_probs), static_cast<const void *>(d_err)})
        if (!aligned(q, 4)) return LHS_ERR_INVALID_ARG;
    SampleParams p = {d_logits, stride, rows, static_cast<int32_t>(vocab), d_u, d_temperature, d_top_p, d_min_p,
                      d_top_k, d_ids, d_probs, d_err};
    return cuda_status(launch_sample(p, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
