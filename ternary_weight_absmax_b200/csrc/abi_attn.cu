// abi_attn.cu -- the entry points of the cache and attention calls: host-side
// validation, then one launch.  Declarations: include/bitnet_w2a8.h.
#include <atomic>

#include "attn.cuh"

namespace bitnet {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encode() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 f = fn.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        fn.store(f, std::memory_order_release);
    }
    return f;
}

namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

bitnet_status cuda_fail(cudaError_t e, const char *what) {
    return set_error_detail(BITNET_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool dtype_ok(int32_t d) { return d == BITNET_F32 || d == BITNET_BF16 || d == BITNET_F16; }
size_t row_align(int32_t d) { return d == BITNET_F32 ? 16 : 8; }  // four elements

constexpr int32_t kMaxHeads = 1024;
constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int32_t kMaxSeqs = 1 << 24;

bitnet_status check_cache(const bitnet_kv_cache *c) {
    if (!c) return set_error_detail(BITNET_ERR_NULL, "cache is NULL");
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return set_error_detail(BITNET_ERR_NULL, "cache buffer is NULL");
    if (c->head_dim != 64 && c->head_dim != 128)
        return set_error_detail(BITNET_ERR_SHAPE, "head_dim %d: 64 or 128", c->head_dim);
    if (c->kv_heads < 1 || c->kv_heads > kMaxHeads)
        return set_error_detail(BITNET_ERR_SHAPE, "kv_heads %d outside 1..%d", c->kv_heads, kMaxHeads);
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
        return set_error_detail(BITNET_ERR_SHAPE, "page_size %d: a power of two, 16..1024", c->page_size);
    if (c->num_pages < 1 || c->num_pages >= (int64_t(1) << 31) / (c->kv_heads * c->page_size))
        return set_error_detail(BITNET_ERR_SHAPE, "num_pages %lld: from 1, and below 2^31 rows in all", (long long)c->num_pages);
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return set_error_detail(BITNET_ERR_ALIGN, "codes need 16-byte, scales 4-byte alignment");
    return BITNET_OK;
}

bitnet_status check_index(int32_t seqs, int32_t max_pages) {
    if (seqs < 1 || seqs > kMaxSeqs) return set_error_detail(BITNET_ERR_SHAPE, "seqs %d outside 1..%d", seqs, kMaxSeqs);
    if (max_pages < 1) return set_error_detail(BITNET_ERR_SHAPE, "max_pages %d < 1", max_pages);
    return BITNET_OK;
}

bitnet_status check_heads(int32_t q_heads, int32_t kv_heads) {
    if (q_heads < 1 || q_heads > kMaxHeads || q_heads % kv_heads)
        return set_error_detail(BITNET_ERR_SHAPE, "q_heads %d: a multiple of kv_heads %d, at most %d", q_heads, kv_heads,
                                kMaxHeads);
    return BITNET_OK;
}

// Rows of `heads` vectors of head_dim elements, `stride` elements apart.
bitnet_status check_rows(const void *p, int64_t stride, int32_t heads, int32_t head_dim, size_t align, int64_t tokens,
                         int64_t multiple, const char *what) {
    if (!p) return set_error_detail(BITNET_ERR_NULL, "%s is NULL", what);
    if (!aligned(p, align) || stride % multiple)
        return set_error_detail(BITNET_ERR_ALIGN, "%s: %zu-byte alignment and a stride in multiples of %lld elements", what,
                                align, (long long)multiple);
    if (stride < (int64_t)heads * head_dim && tokens > 1)
        return set_error_detail(BITNET_ERR_SHAPE, "%s: stride %lld below a row's %d elements", what, (long long)stride,
                                heads * head_dim);
    if (stride < 0 || stride > (int64_t(1) << 32))
        return set_error_detail(BITNET_ERR_SHAPE, "%s: stride %lld invalid", what, (long long)stride);
    return BITNET_OK;
}

}  // namespace
}  // namespace bitnet

using namespace bitnet;

extern "C" {

bitnet_status bitnet_kv_append(const bitnet_kv_cache *cache, const bitnet_kv_append_args *a, bitnet_stream_t stream) {
    set_error_detail(BITNET_OK, "%s", "");
    bitnet_status s = check_cache(cache);
    if (s != BITNET_OK) return s;
    if (!a) return set_error_detail(BITNET_ERR_NULL, "args is NULL");
    if (a->tokens < 0 || a->tokens > kMaxTokens)
        return set_error_detail(BITNET_ERR_SHAPE, "tokens %lld invalid", (long long)a->tokens);
    if ((s = check_index(a->seqs, a->max_pages)) != BITNET_OK) return s;
    if (!dtype_ok(a->in_dtype) || !dtype_ok(a->out_dtype))
        return set_error_detail(BITNET_ERR_VALUE, "unknown dtype %d / %d", a->in_dtype, a->out_dtype);
    if ((a->q == nullptr) != (a->q_out == nullptr) || (a->q == nullptr) != (a->q_heads == 0))
        return set_error_detail(BITNET_ERR_NULL, "q, q_out and q_heads go together");
    if (a->q && (s = check_heads(a->q_heads, cache->kv_heads)) != BITNET_OK) return s;
    if ((a->rope == nullptr) != (a->rot_dim == 0) || (a->rope && (a->rot_dim < 8 || a->rot_dim > cache->head_dim ||
                                                                  a->rot_dim % 8 || a->rope_rows < 1)))
        return set_error_detail(BITNET_ERR_SHAPE, "rot_dim %d: a multiple of 8 up to head_dim with rope (%lld rows), 0 without",
                                a->rot_dim, (long long)a->rope_rows);
    if ((a->q_norm || a->k_norm) && !(a->eps >= 0.0f && a->eps < 1e30f))
        return set_error_detail(BITNET_ERR_VALUE, "eps is negative or not finite");
    if (a->tokens == 0) return BITNET_OK;
    const size_t al = row_align(a->in_dtype);
    if (a->q && (s = check_rows(a->q, a->q_stride, a->q_heads, cache->head_dim, al, a->tokens, 4, "q")) != BITNET_OK) return s;
    if ((s = check_rows(a->k, a->k_stride, cache->kv_heads, cache->head_dim, al, a->tokens, 4, "k")) != BITNET_OK) return s;
    if ((s = check_rows(a->v, a->v_stride, cache->kv_heads, cache->head_dim, al, a->tokens, 4, "v")) != BITNET_OK) return s;
    if (!a->cu_tokens || !a->cache_len || !a->block_table)
        return set_error_detail(BITNET_ERR_NULL, "cu_tokens, cache_len or block_table is NULL");
    if (!aligned(a->cu_tokens, 4) || !aligned(a->cache_len, 4) || !aligned(a->block_table, 4) || !aligned(a->rope, 16) ||
        !aligned(a->q_norm, 16) || !aligned(a->k_norm, 16) || !aligned(a->q_out, 16) || !aligned(a->k_out, 16) ||
        !aligned(a->v_out, 16))
        return set_error_detail(BITNET_ERR_ALIGN, "index arrays need 4-byte, rope, norms and outputs 16-byte alignment");
    DeviceGlobals g;
    cudaError_t e = device_globals(&g);
    if (e != cudaSuccess) return cuda_fail(e, "device globals");
    e = launch_kv_append(*cache, *a, g, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BITNET_OK : cuda_fail(e, "kv_append launch");
}

bitnet_status bitnet_kv_gather(const bitnet_kv_cache *cache, const int32_t *cu_tokens, const int32_t *block_table,
                               int32_t seqs, int32_t max_pages, int64_t tokens, void *k_out, void *v_out, int32_t dtype,
                               bitnet_stream_t stream) {
    set_error_detail(BITNET_OK, "%s", "");
    bitnet_status s = check_cache(cache);
    if (s != BITNET_OK) return s;
    if (tokens < 0 || tokens > kMaxTokens) return set_error_detail(BITNET_ERR_SHAPE, "tokens %lld invalid", (long long)tokens);
    if ((s = check_index(seqs, max_pages)) != BITNET_OK) return s;
    if (!dtype_ok(dtype)) return set_error_detail(BITNET_ERR_VALUE, "unknown dtype %d", dtype);
    if (tokens == 0) return BITNET_OK;
    if (!cu_tokens || !block_table || !k_out || !v_out) return set_error_detail(BITNET_ERR_NULL, "NULL pointer");
    if (!aligned(cu_tokens, 4) || !aligned(block_table, 4) || !aligned(k_out, 16) || !aligned(v_out, 16))
        return set_error_detail(BITNET_ERR_ALIGN, "index arrays need 4-byte, outputs 16-byte alignment");
    DeviceGlobals g;
    cudaError_t e = device_globals(&g);
    if (e != cudaSuccess) return cuda_fail(e, "device globals");
    e = launch_kv_gather(*cache, cu_tokens, block_table, seqs, max_pages, tokens, k_out, v_out, dtype, g,
                         reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BITNET_OK : cuda_fail(e, "kv_gather launch");
}

size_t bitnet_attn_decode_workspace_bytes(int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    if (seqs < 1 || seqs > kMaxSeqs || kv_heads < 1 || kv_heads > kMaxHeads || q_heads < 1 || q_heads > kMaxHeads ||
        q_heads % kv_heads || (head_dim != 64 && head_dim != 128))
        return 0;
    return attn_decode_workspace_bytes(seqs, q_heads, kv_heads, head_dim);
}

bitnet_status bitnet_attn_decode(const bitnet_kv_cache *cache, const void *q, int64_t q_stride, int32_t q_heads,
                                 const int32_t *seq_len, const int32_t *block_table, int32_t seqs, int32_t max_pages,
                                 float scale, void *out, float *lse, int32_t dtype, void *workspace_dev,
                                 size_t workspace_bytes, bitnet_stream_t stream) {
    set_error_detail(BITNET_OK, "%s", "");
    bitnet_status s = check_cache(cache);
    if (s != BITNET_OK) return s;
    if ((s = check_index(seqs, max_pages)) != BITNET_OK) return s;
    if ((s = check_heads(q_heads, cache->kv_heads)) != BITNET_OK) return s;
    if (!dtype_ok(dtype)) return set_error_detail(BITNET_ERR_VALUE, "unknown dtype %d", dtype);
    if (!(scale > -1e30f && scale < 1e30f)) return set_error_detail(BITNET_ERR_VALUE, "scale is not finite");
    if ((s = check_rows(q, q_stride, q_heads, cache->head_dim, row_align(dtype), seqs, 4, "q")) != BITNET_OK) return s;
    if (!seq_len || !block_table || !out || !workspace_dev) return set_error_detail(BITNET_ERR_NULL, "NULL pointer");
    if (!aligned(seq_len, 4) || !aligned(block_table, 4) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(workspace_dev, 16))
        return set_error_detail(BITNET_ERR_ALIGN, "index arrays and lse need 4-byte, out and workspace 16-byte alignment");
    const size_t need = attn_decode_workspace_bytes(seqs, q_heads, cache->kv_heads, cache->head_dim);
    if (workspace_bytes < need) return set_error_detail(BITNET_ERR_BUFSIZE, "workspace %zu < %zu bytes", workspace_bytes, need);
    DeviceGlobals g;
    cudaError_t e = device_globals(&g);
    if (e != cudaSuccess) return cuda_fail(e, "device globals");
    DecodeCall d{*cache, q, q_stride, q_heads, seq_len, block_table, seqs, max_pages, scale, out, lse, dtype, workspace_dev};
    e = launch_attn_decode(d, g, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BITNET_OK : cuda_fail(e, "attn_decode launch");
}

bitnet_status bitnet_attn_prompt(const bitnet_attn_prompt_args *a, bitnet_stream_t stream) {
    set_error_detail(BITNET_OK, "%s", "");
    if (!a) return set_error_detail(BITNET_ERR_NULL, "args is NULL");
    if (a->head_dim != 64 && a->head_dim != 128)
        return set_error_detail(BITNET_ERR_SHAPE, "head_dim %d: 64 or 128", a->head_dim);
    if (a->kv_heads < 1 || a->kv_heads > kMaxHeads)
        return set_error_detail(BITNET_ERR_SHAPE, "kv_heads %d outside 1..%d", a->kv_heads, kMaxHeads);
    bitnet_status s = check_heads(a->q_heads, a->kv_heads);
    if (s != BITNET_OK) return s;
    if (a->seqs < 1 || a->seqs > kMaxSeqs)
        return set_error_detail(BITNET_ERR_SHAPE, "seqs %d outside 1..%d", a->seqs, kMaxSeqs);
    if (a->q_tokens < 0 || a->q_tokens > kMaxTokens || a->k_tokens < 0 || a->k_tokens > kMaxTokens)
        return set_error_detail(BITNET_ERR_SHAPE, "tokens %lld / %lld invalid", (long long)a->q_tokens,
                                (long long)a->k_tokens);
    if ((a->dtype != BITNET_BF16 && a->dtype != BITNET_F16) || (a->out_dtype != a->dtype && a->out_dtype != BITNET_F32))
        return set_error_detail(BITNET_ERR_VALUE, "dtype %d / out_dtype %d: a 16-bit type, out in it or in fp32", a->dtype,
                                a->out_dtype);
    if (!(a->scale > -1e30f && a->scale < 1e30f)) return set_error_detail(BITNET_ERR_VALUE, "scale is not finite");
    if (a->q_tokens == 0) return BITNET_OK;
    if ((s = check_rows(a->q, a->q_stride, a->q_heads, a->head_dim, 16, a->q_tokens, 8, "q")) != BITNET_OK) return s;
    if (a->k_tokens > 0) {
        if ((s = check_rows(a->k, a->k_stride, a->kv_heads, a->head_dim, 16, a->k_tokens, 8, "k")) != BITNET_OK) return s;
        if ((s = check_rows(a->v, a->v_stride, a->kv_heads, a->head_dim, 16, a->k_tokens, 8, "v")) != BITNET_OK) return s;
    }
    const int64_t pairs = (a->q_heads / a->kv_heads + 1) / 2 * (int64_t)a->kv_heads;
    if ((a->q_tokens / 128 + a->seqs) * pairs > 0x7fffffff)
        return set_error_detail(BITNET_ERR_SHAPE, "%lld tokens of %d heads: more than 2^31 tiles", (long long)a->q_tokens, a->q_heads);
    if (!a->cu_q || !a->cu_k || !a->out) return set_error_detail(BITNET_ERR_NULL, "NULL pointer");
    if (!aligned(a->cu_q, 4) || !aligned(a->cu_k, 4) || !aligned(a->out, 16) || !aligned(a->lse, 4))
        return set_error_detail(BITNET_ERR_ALIGN, "index arrays and lse need 4-byte, out 16-byte alignment");
    int dev = 0, major = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e != cudaSuccess) return cuda_fail(e, "device query");
    if (major != 10)
        return set_error_detail(BITNET_ERR_UNSUPPORTED, "attn_prompt needs an sm_100 device (found sm_%d)", major * 10);
    DeviceGlobals g;
    e = device_globals(&g);
    if (e != cudaSuccess) return cuda_fail(e, "device globals");
    e = launch_attn_prompt(*a, g, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BITNET_OK : cuda_fail(e, "attn_prompt launch");
}

}  // extern "C"
