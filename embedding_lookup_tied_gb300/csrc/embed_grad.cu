// embed_grad.cu — the gradient of the scaled embedding lookup: dtable[v] =
// scale * sum of dout over the positions that name row v.
//
// Counterpart of the lookup of ADR-0008 "Remote Embeddings and lm_head Service"
// (POST /v1/embed) with the scale of "embedding-inference — Port
// Specification" (Forward graph).
//
// First form: positions ordered by (id, position) by counting, for each, the
// ones before it; then a CTA to a distinct id, which adds its positions up in
// order.
#include "train.cuh"

namespace lhs {
namespace {

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

__device__ __forceinline__ uint32_t key_of(int32_t id, int64_t vocab, int32_t ignore) {
    return id >= 0 && id < vocab && id != ignore ? static_cast<uint32_t>(id) : 0xFFFFFFFFu;
}

__global__ void __launch_bounds__(256) zero_kernel(uint4 *p, size_t n16, uint8_t *tail, int ntail) {
    pdl_wait();
    for (size_t i = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n16;
         i += static_cast<size_t>(gridDim.x) * blockDim.x)
        p[i] = make_uint4(0u, 0u, 0u, 0u);
    if (blockIdx.x == 0 && static_cast<int>(threadIdx.x) < ntail) tail[threadIdx.x] = 0;
}

__global__ void __launch_bounds__(256)
    rank_ids_kernel(const int32_t *ids, int n, int64_t vocab, int32_t ignore, uint32_t *keys, int32_t *order,
                    int32_t *err) {
    __shared__ uint32_t tile[256];
    pdl_wait();
    const int i = blockIdx.x * 256 + threadIdx.x;
    const int32_t id = i < n ? ld_dep(ids + i) : ignore;
    const uint32_t k = key_of(id, vocab, ignore);
    if (k == 0xFFFFFFFFu && id != ignore) set_err(err, LHS_ERRBIT_BAD_TOKEN);
    int rank = 0;
    for (int b = 0; b < n; b += 256) {
        tile[threadIdx.x] = b + static_cast<int>(threadIdx.x) < n ? key_of(ld_dep(ids + b + threadIdx.x), vocab, ignore) : 0;
        __syncthreads();
        const int m = n - b < 256 ? n - b : 256;
        for (int j = 0; j < m; ++j) rank += tile[j] < k || (tile[j] == k && b + j < i) ? 1 : 0;
        __syncthreads();
    }
    if (i < n) {
        keys[rank] = k;
        order[rank] = i;
    }
}

template <int DT, typename O>
__global__ void __launch_bounds__(128)
    sum_rows_kernel(const uint32_t *keys, const int32_t *order, int n, int hidden, float scale,
                    const typename Elem<DT>::T *dout, int64_t dout_stride, bool accumulate, O *dtable) {
    pdl_wait();
    const int i0 = blockIdx.x;
    const uint32_t k = ld_dep(keys + i0);
    if (k == 0xFFFFFFFFu || (i0 > 0 && ld_dep(keys + i0 - 1) == k)) return;
    for (int j = threadIdx.x; j < hidden; j += 128) {
        float s = 0.0f;
        for (int i = i0; i < n && ld_dep(keys + i) == k; ++i)
            s += Elem<DT>::widen(ld_dep(dout + ld_dep(order + i) * dout_stride + j));
        O *o = dtable + static_cast<int64_t>(k) * hidden + j;
        put_rn(o, fmaf(s, scale, accumulate ? wide(*o) : 0.0f));
    }
}

template <int DT>
cudaError_t sum_rows(const EmbedGradArgs &a, const uint32_t *keys, const int32_t *order, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(a.n)), block(128);
    const auto *d = static_cast<const typename Elem<DT>::T *>(a.dout);
    const int n = static_cast<int>(a.n);
    if (a.dtable_dtype == LHS_F32)
        return launch_pdl(sum_rows_kernel<DT, float>, grid, block, 0, stream, keys, order, n, a.hidden, a.scale, d,
                          a.dout_stride, a.accumulate, static_cast<float *>(a.dtable));
    if (a.dtable_dtype == LHS_F16)
        return launch_pdl(sum_rows_kernel<DT, __half>, grid, block, 0, stream, keys, order, n, a.hidden, a.scale, d,
                          a.dout_stride, a.accumulate, static_cast<__half *>(a.dtable));
    return launch_pdl(sum_rows_kernel<DT, __nv_bfloat16>, grid, block, 0, stream, keys, order, n, a.hidden, a.scale, d,
                      a.dout_stride, a.accumulate, static_cast<__nv_bfloat16 *>(a.dtable));
}

}  // namespace

cudaError_t launch_zero(void *p, size_t bytes, cudaStream_t stream) {
    DeviceInfo dev;
    const cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return e;
    const size_t n16 = bytes / 16, want = (n16 + 255) / 256, cap = static_cast<size_t>(dev.num_sms) * 8;
    return launch_pdl(zero_kernel, dim3(static_cast<unsigned>(want < 1 ? 1 : want < cap ? want : cap)), dim3(256), 0, stream,
                      static_cast<uint4 *>(p), n16, static_cast<uint8_t *>(p) + n16 * 16, static_cast<int>(bytes % 16));
}

size_t embed_grad_workspace(int64_t, int32_t, int64_t n) { return 2 * align256(static_cast<size_t>(n) * 4); }

cudaError_t launch_embed_grad(const EmbedGradArgs &a, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    if (!a.accumulate) {
        const size_t es = a.dtable_dtype == LHS_F32 ? 4 : 2;
        e = launch_zero(a.dtable, static_cast<size_t>(a.vocab) * a.hidden * es, stream);
        if (e != cudaSuccess) return e;
    }
    if (a.n == 0) return cudaSuccess;
    uint32_t *keys = reinterpret_cast<uint32_t *>(a.ws);
    int32_t *order = reinterpret_cast<int32_t *>(a.ws + align256(static_cast<size_t>(a.n) * 4));
    e = launch_pdl(rank_ids_kernel, dim3(static_cast<unsigned>((a.n + 255) / 256)), dim3(256), 0, stream, a.ids,
                   static_cast<int>(a.n), a.vocab, a.ignore, keys, order, a.err);
    if (e != cudaSuccess) return e;
    switch (a.dout_dtype) {
    case LHS_F32: return sum_rows<LHS_F32>(a, keys, order, stream);
    case LHS_F16: return sum_rows<LHS_F16>(a, keys, order, stream);
    default: return sum_rows<LHS_BF16>(a, keys, order, stream);
    }
}

}  // namespace lhs
