// attn.cuh -- what the cache and attention kernels share: launchers, the
// element types, and how a work unit finds its sequence.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include "common.cuh"

namespace bitnet {

constexpr int kKvBlock = BITNET_KV_BLOCK;

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encode();  // NULL if the driver has none

cudaError_t launch_kv_append(const bitnet_kv_cache &c, const bitnet_kv_append_args &a, const DeviceGlobals &g,
                             cudaStream_t st);
cudaError_t launch_kv_gather(const bitnet_kv_cache &c, const int32_t *cu, const int32_t *table, int32_t seqs,
                             int32_t max_pages, int64_t tokens, void *k_out, void *v_out, int32_t dtype,
                             const DeviceGlobals &g, cudaStream_t st);
size_t attn_decode_workspace_bytes(int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim);
struct DecodeCall {
    bitnet_kv_cache c;
    const void *q;
    int64_t q_stride;
    int32_t q_heads;
    const int32_t *seq_len, *table;
    int32_t seqs, max_pages;
    float scale;
    void *out;
    float *lse;
    int32_t dtype;
    void *workspace;
};
cudaError_t launch_attn_decode(const DecodeCall &d, const DeviceGlobals &g, cudaStream_t st);
cudaError_t launch_attn_prompt(const bitnet_attn_prompt_args &a, const DeviceGlobals &g, cudaStream_t st);

#ifdef __CUDACC__
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The larger; NaN where an operand is (fmaxf gives the other operand).
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// N consecutive elements as fp32 (one vector load), and back with one rounding each.
template <int N>
__device__ __forceinline__ void load_f32(const float *p, float (&v)[N]) {
    if constexpr (N == 4) {
        const float4 t = *reinterpret_cast<const float4 *>(p);
        v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
    } else {
        const float2 t = *reinterpret_cast<const float2 *>(p);
        v[0] = t.x, v[1] = t.y;
    }
}
__device__ __forceinline__ float2 up2(__nv_bfloat162 h) { return __bfloat1622float2(h); }
__device__ __forceinline__ float2 up2(__half2 h) { return __half22float2(h); }
template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
    using type = __nv_bfloat162;
    static __device__ __forceinline__ type down(float a, float b) { return __floats2bfloat162_rn(a, b); }
};
template <>
struct Pair<__half> {
    using type = __half2;
    static __device__ __forceinline__ type down(float a, float b) { return __floats2half2_rn(a, b); }
};
template <int N, typename T>
__device__ __forceinline__ void load_f32(const T *p, float (&v)[N]) {
    using P2 = typename Pair<T>::type;
    P2 h[N / 2];
    if constexpr (N == 4)
        *reinterpret_cast<uint2 *>(h) = *reinterpret_cast<const uint2 *>(p);
    else
        *reinterpret_cast<uint32_t *>(h) = *reinterpret_cast<const uint32_t *>(p);
#pragma unroll
    for (int i = 0; i < N / 2; i++) {
        const float2 f = up2(h[i]);
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}
template <int N>
__device__ __forceinline__ void store_from_f32(float *p, const float (&v)[N]) {
    if constexpr (N == 2) {
        *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) reinterpret_cast<float4 *>(p)[i / 4] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}
template <int N, typename T>
__device__ __forceinline__ void store_from_f32(T *p, const float (&v)[N]) {
    using P2 = typename Pair<T>::type;
    P2 h[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; i++) h[i] = Pair<T>::down(v[2 * i], v[2 * i + 1]);
    const uint32_t *w = reinterpret_cast<const uint32_t *>(h);
    if constexpr (N == 2) {
        *reinterpret_cast<uint32_t *>(p) = w[0];
    } else if constexpr (N == 4) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 8)
            reinterpret_cast<uint4 *>(p)[i / 8] = make_uint4(w[i / 2], w[i / 2 + 1], w[i / 2 + 2], w[i / 2 + 3]);
    }
}

// Latches BOUNDS if sequence i's rows go backwards, begin before row 0 or pass
// `rows`, or its length in the cache (`len`, if given) is negative.  Done for every
// sequence apart from the work units below: one behind the last row, or one that
// goes backwards, may own no unit.
__device__ __forceinline__ void check_sequence(const int32_t *cu, int64_t rows, const int32_t *len, int64_t i, unsigned *err) {
    const int lo = cu[i], hi = cu[i + 1];
    if (lo < 0 || hi < lo || hi > rows || (len && len[i] < 0)) atomicOr(err, kErrBounds);
}

// Sequences of a packed batch own consecutive work units: sequence i those from
// base(i) = cu[i] / per + slack * i on (per: tokens of a unit; slack: units that
// a sequence may need beyond tokens / per).  The bases need no pass over the
// lengths, and their last value bounds the grid on the host.  Returns the last
// sequence whose base is not above `unit`, by a search that a warp makes 32
// ways at a time (all lanes call it; any cu gives an index in 0 .. seqs-1).
__device__ __forceinline__ int64_t unit_base(const int32_t *cu, int i, int per, int slack) {
    return (int64_t)cu[i] / per + (int64_t)slack * i;
}
__device__ __forceinline__ int find_seq(const int32_t *cu, int seqs, int64_t unit, int per, int slack) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = seqs;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int64_t at = lo + (int64_t)lane * step;
        const bool below = at < hi && unit_base(cu, (int)at, per, slack) <= unit;
        int n = __popc(__ballot_sync(0xffffffffu, below));
        if (n < 1) n = 1;
        lo += (n - 1) * step;
        if (lo > seqs - 1) lo = seqs - 1;
        if (hi > lo + step) hi = lo + step;
    }
    return lo;
}
#endif

}  // namespace bitnet
