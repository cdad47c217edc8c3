// kv_cache.cu -- the paged int8 key / value cache: append (per-head norm,
// rotation, quantisation) and gather.
//
// Append.  A CTA owns one 16-token block of one sequence and one or more kv
// heads: the new tokens of the block, their keys and values, and the query heads
// of the groups.  A warp holds a head vector in registers (D / 32 elements a
// lane), so the norm is one warp reduction, a rotation partner is in the same
// lane (interleaved) or one shuffle away (half layout), and q, k, v are read
// once, several vectors of a warp in flight.  The block's scale needs the absmax
// of all its new tokens: each warp leaves those of its vectors in shared memory,
// and after one barrier the warps quantise what they still hold.  A block with
// one new token (a decode step) needs no barrier: each warp has all it needs.
// Older codes of the block are rewritten only if the scale falls.
// Blocks are found without a pass over the lengths: with few tokens a sequence
// (below 32/15) by a unit for each token, otherwise by a unit for each 16 and two
// for each sequence, whichever makes the smaller grid.  Bound: HBM at prompt
// sizes (8k tokens of 32 + 2 x 8 heads of 128 from fp32, k and v in bf16 as well: 90
// us, 4.3 TB/s; what is missing is latency: a block is looked up before its vectors are
// asked for, and waits at its barrier),
// latency at one token a sequence (1: 3.0 us, 256: 6.0 us; 4.9 and 11.4 where the
// scales fall and the older codes of the blocks are rewritten, which is done by
// one warp a head and not begun before the new scale is known).
//
// Gather.  64 tokens of one head per CTA, 16 codes a thread and load; bound: HBM
// (64k tokens of 8 heads of 128 to bf16: 78.2 us, 5.5 TB/s).
#include <algorithm>

#include "attn.cuh"

namespace bitnet {
namespace {

constexpr int kGatherTokens = 64;
constexpr int kGatherThreads = 256;

struct CacheView {
    int8_t *codes[2];
    float *scale[2];
    int64_t num_pages;
    int kv_heads, page_shift;  // page_size = 1 << page_shift
};

struct AppendArgs {
    CacheView c;
    const void *in[3];    // q, k, v
    int64_t stride[3];
    void *out[3];
    const int32_t *cu, *cache_len, *table;
    const float *rope;
    const float *norm[2];  // q, k
    int64_t tokens, rope_rows;
    int seqs, max_pages, q_heads, group, rot_dim, interleaved;
    int heads_per_cta, per, slack;  // kv heads of a CTA; units as in find_seq
    float eps;
    unsigned *err;
};

CacheView view_of(const bitnet_kv_cache &c) {
    CacheView v;
    v.codes[0] = c.k, v.codes[1] = c.v;
    v.scale[0] = c.k_scale, v.scale[1] = c.v_scale;
    v.num_pages = c.num_pages;
    v.kv_heads = c.kv_heads;
    v.page_shift = 0;
    while ((1 << v.page_shift) < c.page_size) v.page_shift++;
    return v;
}

// x <- (x * r) * w, r = 1 / sqrt(mean(x^2) + eps).  The squares and their sum
// are fp64 (a fp32 square is exact there), so r does not depend on the order
// of the sum, or on rsqrt's last bit, but for a chance of about 2^-28 a vector,
// and codes are reproducible by any implementation of the definition.
template <int D>
__device__ __forceinline__ void norm_vec(float (&x)[D / 32], const float *w, float eps) {
    constexpr int V = D / 32;
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < V; i++) ss = fma((double)x[i], (double)x[i], ss);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = (float)rsqrt(ss / D + (double)eps);
    float wv[V];
    load_f32<V>(w + (threadIdx.x & 31) * V, wv);
#pragma unroll
    for (int i = 0; i < V; i++) x[i] = __fmul_rn(__fmul_rn(x[i], r), wv[i]);
}

// What a position does to a lane's V elements: x <- x * c + y * s with y the
// partner, s negated for the first of a pair (a * c - b * s is the same sum).
// Held for all vectors of a token.
template <int D>
struct Turn {
    static constexpr int V = D / 32;
    float c[V], s[V];
    int from;        // lane of the partners (half layout)
    bool on, mine;   // there is a rotation; it reaches this lane's elements

    __device__ __forceinline__ void load(const float *row, int rot, bool interleaved) {
        const int lane = threadIdx.x & 31, e0 = lane * V;
        on = rot > 0, mine = e0 < rot, from = lane;
        if (!on) return;
        if (interleaved) {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                c[i] = c[i + 1] = mine ? row[(e0 + i) / 2] : 0.0f;
                s[i + 1] = mine ? row[rot / 2 + (e0 + i) / 2] : 0.0f;
                s[i] = -s[i + 1];
            }
        } else {
            // rot is a multiple of 8 and V at most 4: the partners of a lane's
            // elements are all in one lane, rot / 2 elements away.
            const bool first = e0 < rot / 2;
            if (mine) {
                const int j = first ? e0 : e0 - rot / 2;
                load_f32<V>(row + j, c);
                load_f32<V>(row + rot / 2 + j, s);
                from = first ? lane + rot / (2 * V) : lane - rot / (2 * V);
            }
#pragma unroll
            for (int i = 0; i < V; i++) s[i] = first ? -s[i] : s[i];
        }
    }
    __device__ __forceinline__ void apply(float (&x)[V], bool interleaved) const {
        if (!on) return;
        float y[V];
        if (interleaved) {
#pragma unroll
            for (int i = 0; i < V; i++) y[i] = x[i ^ 1];
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) y[i] = __shfl_sync(0xffffffffu, x[i], from);
        }
        if (mine) {
#pragma unroll
            for (int i = 0; i < V; i++) x[i] = __fadd_rn(__fmul_rn(x[i], c[i]), __fmul_rn(y[i], s[i]));
        }
    }
};

// rint(x * s), |x * s| at most 127 and a rounding (s is 127 over an absmax of at
// least |x|, or smaller, so the definition's clamp changes nothing): the low byte
// of the sum with 1.5 2^23.  (Where s is NaN any byte will do.)
__device__ __forceinline__ uint32_t quant(float x, float s) {
    return __float_as_uint(__fadd_rn(__fmul_rn(x, s), 12582912.0f));
}
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// A new scale for a block that holds older tokens: the smaller one, and by how
// much its old codes have to shrink.
// NaN, once there, stays (1e-5 bounds a real scale, so the sum is finite).
__device__ __forceinline__ float joint_scale(float s, float was, float &fall) {
    const float both = s + was;
    s = both == both ? fminf(s, was) : both;
    fall = s < was ? __fdiv_rn(s, was) : 1.0f;
    return s;
}
// NaN for a block that holds a NaN or an infinity: codes have no such values, and
// those that they would turn into are not told from real ones.
__device__ __forceinline__ float block_scale(float amax) {
    return amax < INFINITY ? __fmul_rn(127.0f, __frcp_rn(amax > kEps ? amax : kEps)) : NAN;
}
// codes <- rint(codes * fall): `rows` rows from p on, by `threads` threads.
template <int D>
__device__ __forceinline__ void shrink(int8_t *codes, int rows, float fall, int me, int threads) {
    char4 *p = reinterpret_cast<char4 *>(codes);
    for (int i = me; i < rows * D / 4; i += threads) {
        const char4 c = p[i];
        reinterpret_cast<uint32_t *>(p)[i] =
            bytes4(quant((float)c.x, fall), quant((float)c.y, fall), quant((float)c.z, fall), quant((float)c.w, fall));
    }
}
template <int V>
__device__ __forceinline__ void store_codes(int8_t *dst, const float (&x)[V], float s) {
    if constexpr (V == 4)
        *reinterpret_cast<uint32_t *>(dst) = bytes4(quant(x[0], s), quant(x[1], s), quant(x[2], s), quant(x[3], s));
    else
        *reinterpret_cast<uint16_t *>(dst) = (uint16_t)__byte_perm(quant(x[0], s), quant(x[1], s), 0x0040);
}
template <int V>
__device__ __forceinline__ float absmax(const float (&x)[V]) {
    unsigned m = 0;  // not negative: ordered as integers, NaN above all others
#pragma unroll
    for (int k = 0; k < V; k++) m = max(m, __float_as_uint(fabsf(x[k])));
    return __uint_as_float(__reduce_max_sync(0xffffffffu, m));
}

template <int D, typename In, typename Out, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 32 / kWarps)
kv_append_kernel(const AppendArgs a) {
    constexpr int V = D / 32;
    constexpr int kHeld = kKvBlock / kWarps;  // tokens of a warp
    constexpr int kFlight = 4;                      // query vectors that a warp reads at once
    __shared__ float amax[2][kKvBlock];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == kWarps - 1 && blockIdx.y == 0) {
#pragma unroll 1
        for (int64_t i = (int64_t)blockIdx.x * 32 + lane; i < a.seqs; i += (int64_t)gridDim.x * 32)
            check_sequence(a.cu, a.tokens, a.cache_len, i, a.err);
    }
    // Warp 0 finds the block: its positions, their rows, and its page.
    __shared__ struct {
        int64_t first, tok;  // position and row of the first new token
        int n, slot, page;   // new tokens (0: nothing to do); the first one's place in the block; -1: no page
    } b;
    if (warp == 0) {
        const int64_t unit = blockIdx.x;
        int seq = -1;
        if (a.per == 1 && unit < a.seqs) {  // one token a sequence, mostly: unit i is sequence i
            const int64_t lo = a.cu[unit], hi = a.cu[unit + 1];
            if (lo == unit && hi > unit) seq = (int)unit;
        }
        if (seq < 0) seq = find_seq(a.cu, a.seqs, unit, a.per, a.slack);
        const int64_t t0 = a.cu[seq], t1 = a.cu[seq + 1];
        const int64_t old = a.cache_len[seq];
        const bool bad = t0 < 0 || t1 < t0 || t1 > a.tokens || old < 0;  // latched by check_sequence
        const int64_t blk = old / kKvBlock + (unit - unit_base(a.cu, seq, a.per, a.slack));  // block of the sequence
        const int64_t first = max(old, blk * kKvBlock);
        const int64_t last = min(old + (t1 - t0), (blk + 1) * kKvBlock);
        const int n = bad || first >= last ? 0 : (int)(last - first);
        const int64_t pg = blk * kKvBlock >> a.c.page_shift;
        int64_t page = -1;
        if (n > 0 && pg < a.max_pages) page = a.table[(int64_t)seq * a.max_pages + pg];
        if (page >= a.c.num_pages) page = -1;
        if (lane == 0) {
            if (n > 0 && (page < 0 || (a.rope && last > a.rope_rows))) atomicOr(a.err, kErrBounds);
            b.first = first, b.tok = t0 + (first - old);
            b.n = n, b.slot = (int)(first - blk * kKvBlock), b.page = page < 0 ? -1 : (int)page;
        }
    }
    __syncthreads();
    const int n = b.n, slot = b.slot, page = b.page;
    const int64_t first = b.first, tok = b.tok;
    if (n == 0) return;
    const bool here = page >= 0;  // a bad page leaves the cache alone
    const int in_page = (int)((first - slot) & ((1 << a.c.page_shift) - 1));
    auto row_of = [&](int head) { return (((int64_t)page * a.c.kv_heads + head) << a.c.page_shift) + in_page; };  // block's first row

    const bool inter = a.interleaved != 0;
    auto turn_of = [&](int i, Turn<D> &t) {
        const int64_t p = min(first + i, a.rope_rows - 1);
        t.load(a.rope + p * a.rot_dim, a.rot_dim, inter);
    };
    // Token i's vector of `head` in q (0), k (1) or v (2), and in its output.
    auto from = [&](int which, int i, int head) {
        return static_cast<const In *>(a.in[which]) + (tok + i) * a.stride[which] + (int64_t)head * D + lane * V;
    };
    auto to = [&](int which, int i, int head, int heads) {
        return static_cast<Out *>(a.out[which]) + ((tok + i) * heads + head) * D + lane * V;
    };
    const int h0 = blockIdx.y * a.heads_per_cta, h1 = min(h0 + a.heads_per_cta, a.c.kv_heads);

    if (n == 1) {
        // Vectors: for each head the key and the value, then all query heads.
        const int kv = 2 * (h1 - h0), vecs = kv + (a.in[0] ? (h1 - h0) * a.group : 0);
        Turn<D> t;
        turn_of(0, t);
        for (int e0 = warp; e0 < vecs; e0 += kFlight * kWarps) {
            float x[kFlight][V];
#pragma unroll
            for (int u = 0; u < kFlight; u++) {
                const int e = e0 + u * kWarps;
                if (e < kv)
                    load_f32<V>(from(1 + (e & 1), 0, h0 + (e >> 1)), x[u]);
                else if (e < vecs)
                    load_f32<V>(from(0, 0, h0 * a.group + e - kv), x[u]);
            }
#pragma unroll
            for (int u = 0; u < kFlight; u++) {
                const int e = e0 + u * kWarps;
                if (e >= vecs) continue;
                if (e >= kv) {
                    if (a.norm[0]) norm_vec<D>(x[u], a.norm[0], a.eps);
                    t.apply(x[u], inter);
                    store_from_f32<V>(to(0, 0, h0 * a.group + e - kv, a.q_heads), x[u]);
                    continue;
                }
                const int head = h0 + (e >> 1), side = e & 1;
                if (side == 0) {
                    if (a.norm[1]) norm_vec<D>(x[u], a.norm[1], a.eps);
                    t.apply(x[u], inter);
                }
                if (a.out[1 + side]) store_from_f32<V>(to(1 + side, 0, head, a.c.kv_heads), x[u]);
                float s = block_scale(absmax(x[u]));
                if (!here) continue;
                const int64_t row0 = row_of(head);
                float *at = (side ? a.c.scale[1] : a.c.scale[0]) + row0 / kKvBlock;
                int8_t *codes = (side ? a.c.codes[1] : a.c.codes[0]) + row0 * D;
                if (slot > 0) {
                    float fall;
                    s = joint_scale(s, *at, fall);
                    __syncwarp();  // every lane has the old scale
                    if (fall < 1.0f) shrink<D>(codes, slot, fall, lane, 32);
                }
                if (lane == 0) *at = s;
                store_codes<V>(codes + slot * D + lane * V, x[u], s);
            }
        }
        return;
    }

    // A warp has one token of every kWarps: its key and value stay in registers,
    // and the cosines and sines serve all the vectors of the token.
    for (int head = h0; head < h1; head++) {
        float k[kHeld][V], v[kHeld][V];
        Turn<D> t[kHeld];
#pragma unroll
        for (int u = 0; u < kHeld; u++) {
            const int i = warp + u * kWarps;
            if (i >= n) continue;
            load_f32<V>(from(1, i, head), k[u]);
            load_f32<V>(from(2, i, head), v[u]);
            turn_of(i, t[u]);
        }
        if (head > h0) __syncthreads();  // the maxima of the head before have been read
#pragma unroll
        for (int u = 0; u < kHeld; u++) {
            const int i = warp + u * kWarps;
            if (i >= n) continue;
            // The group's queries, kFlight heads at once; the key and value while the first are under way.
            const In *src = a.in[0] ? from(0, i, head * a.group) : nullptr;
            Out *dst = a.in[0] ? to(0, i, head * a.group, a.q_heads) : nullptr;
            float q[kFlight][V];
            auto load_q = [&](int g0) {
#pragma unroll
                for (int j = 0; j < kFlight; j++)
                    if (g0 + j < a.group) load_f32<V>(src + (g0 + j) * D, q[j]);
            };
            if (a.in[0]) load_q(0);
            if (a.norm[1]) norm_vec<D>(k[u], a.norm[1], a.eps);
            t[u].apply(k[u], inter);
            if (a.out[1]) store_from_f32<V>(to(1, i, head, a.c.kv_heads), k[u]);
            if (a.out[2]) store_from_f32<V>(to(2, i, head, a.c.kv_heads), v[u]);
            const float mk = absmax(k[u]), mv = absmax(v[u]);
            if (lane == 0) amax[0][i] = mk, amax[1][i] = mv;
            for (int g0 = 0; g0 < (a.in[0] ? a.group : 0); g0 += kFlight) {
                if (g0 > 0) load_q(g0);
#pragma unroll
                for (int j = 0; j < kFlight; j++) {
                    if (g0 + j >= a.group) continue;
                    if (a.norm[0]) norm_vec<D>(q[j], a.norm[0], a.eps);
                    t[u].apply(q[j], inter);
                    store_from_f32<V>(dst + (g0 + j) * D, q[j]);
                }
            }
        }
        __syncthreads();
        if (!here) continue;
        // Half a warp for each side: the scale, and by how much older codes shrink.
        const int64_t row0 = row_of(head);
        const int side = lane >> 4, at = lane & 15;
        float *scale = (side ? a.c.scale[1] : a.c.scale[0]) + row0 / kKvBlock;
        const unsigned half = side ? 0xffff0000u : 0x0000ffffu;
        float s = block_scale(__uint_as_float(__reduce_max_sync(half, at < n ? __float_as_uint(amax[side][at]) : 0u)));
        float fall = 1.0f;
        if (slot > 0) {
            s = joint_scale(s, *scale, fall);
            __syncthreads();  // every thread has read the old scales before they are replaced
        }
        if (warp == 0 && at == 0) *scale = s;
        const float sk = __shfl_sync(0xffffffffu, s, 0), sv = __shfl_sync(0xffffffffu, s, 16);
#pragma unroll
        for (int u = 0; u < kHeld; u++) {
            const int i = warp + u * kWarps;
            if (i >= n) continue;
            const int64_t to_code = (row0 + slot + i) * D + lane * V;
            store_codes<V>(a.c.codes[0] + to_code, k[u], sk);
            store_codes<V>(a.c.codes[1] + to_code, v[u], sv);
        }
        if (slot > 0) {
            const float fk = __shfl_sync(0xffffffffu, fall, 0), fv = __shfl_sync(0xffffffffu, fall, 16);
            if (fk < 1.0f) shrink<D>(a.c.codes[0] + row0 * D, slot, fk, threadIdx.x, 32 * kWarps);
            if (fv < 1.0f) shrink<D>(a.c.codes[1] + row0 * D, slot, fv, threadIdx.x, 32 * kWarps);
        }
    }
}

struct GatherArgs {
    CacheView c;
    const int32_t *cu, *table;
    int64_t tokens;
    int seqs, max_pages;
    void *out[2];
    unsigned *err;
};

template <int D, typename Out>
__global__ void __launch_bounds__(kGatherThreads)
kv_gather_kernel(const GatherArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int head = blockIdx.y;
    const int64_t unit = blockIdx.x;
    if (head == 0 && threadIdx.x >= kGatherThreads - 32) {  // 32 sequences a unit: there are more units than sequences
        const int64_t i = unit * 32 + (threadIdx.x & 31);
        if (i < a.seqs) check_sequence(a.cu, a.tokens, nullptr, i, a.err);
    }
    const int seq = find_seq(a.cu, a.seqs, unit, kGatherTokens, 1);
    const int64_t t0 = a.cu[seq], t1 = a.cu[seq + 1];
    if (t0 < 0 || t1 < t0 || t1 > a.tokens) return;  // latched by check_sequence
    const int64_t first = (unit - unit_base(a.cu, seq, kGatherTokens, 1)) * kGatherTokens;
    const int n = (int)min((int64_t)kGatherTokens, t1 - t0 - first);
    if (first < 0 || n <= 0) return;  // a unit before the first sequence, or that no sequence uses
    constexpr int kPer = D / 16;  // 16-code pieces of a row
#pragma unroll
    for (int side = 0; side < 2; side++) {
#pragma unroll
        for (int e0 = 0; e0 < kGatherTokens * kPer; e0 += kGatherThreads) {
            const int e = e0 + threadIdx.x, i = e / kPer, part = e % kPer;
            if (i >= n) continue;
            const int64_t p = first + i, pg = p >> a.c.page_shift;
            int64_t page = -1;
            if (pg < a.max_pages) page = a.table[(int64_t)seq * a.max_pages + pg];
            if (page < 0 || page >= a.c.num_pages) {
                atomicOr(a.err, kErrBounds);
                continue;
            }
            const int64_t row = ((page * a.c.kv_heads + head) << a.c.page_shift) + (p & ((1 << a.c.page_shift) - 1));
            const int4 w = __ldcs(reinterpret_cast<const int4 *>(a.c.codes[side] + row * D) + part);
            const float inv = __fdiv_rn(1.0f, a.c.scale[side][row / kKvBlock]);
            float v[16];
            const int ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 16; k++) v[k] = __fmul_rn((float)(int8_t)(ws[k / 4] >> (8 * (k % 4))), inv);
            store_from_f32<16>(static_cast<Out *>(a.out[side]) + ((t0 + p) * a.c.kv_heads + head) * D + part * 16, v);
        }
    }
}

cudaLaunchConfig_t config(dim3 grid, int threads, cudaStream_t st, cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

template <int D, typename In, typename Out>
cudaError_t append_warps(const cudaLaunchConfig_t &cfg, const AppendArgs &a) {
    if (cfg.blockDim.x == 256) return cudaLaunchKernelEx(&cfg, kv_append_kernel<D, In, Out, 8>, a);
    return cudaLaunchKernelEx(&cfg, kv_append_kernel<D, In, Out, 16>, a);
}
template <int D, typename In>
cudaError_t append_out(const cudaLaunchConfig_t &cfg, const AppendArgs &a, int out) {
    switch (out) {
        case BITNET_F32: return append_warps<D, In, float>(cfg, a);
        case BITNET_BF16: return append_warps<D, In, __nv_bfloat16>(cfg, a);
        default: return append_warps<D, In, __half>(cfg, a);
    }
}
template <int D>
cudaError_t append_in(const cudaLaunchConfig_t &cfg, const AppendArgs &a, int in, int out) {
    switch (in) {
        case BITNET_F32: return append_out<D, float>(cfg, a, out);
        case BITNET_BF16: return append_out<D, __nv_bfloat16>(cfg, a, out);
        default: return append_out<D, __half>(cfg, a, out);
    }
}
template <int D>
cudaError_t gather_out(const cudaLaunchConfig_t &cfg, const GatherArgs &a, int out) {
    switch (out) {
        case BITNET_F32: return cudaLaunchKernelEx(&cfg, kv_gather_kernel<D, float>, a);
        case BITNET_BF16: return cudaLaunchKernelEx(&cfg, kv_gather_kernel<D, __nv_bfloat16>, a);
        default: return cudaLaunchKernelEx(&cfg, kv_gather_kernel<D, __half>, a);
    }
}

}  // namespace

cudaError_t launch_kv_append(const bitnet_kv_cache &c, const bitnet_kv_append_args &p, const DeviceGlobals &g,
                             cudaStream_t st) {
    AppendArgs a;
    a.c = view_of(c);
    a.in[0] = p.q, a.in[1] = p.k, a.in[2] = p.v;
    a.stride[0] = p.q_stride, a.stride[1] = p.k_stride, a.stride[2] = p.v_stride;
    a.out[0] = p.q_out, a.out[1] = p.k_out, a.out[2] = p.v_out;
    a.cu = p.cu_tokens, a.cache_len = p.cache_len, a.table = p.block_table;
    a.rope = p.rope;
    a.norm[0] = p.q_norm, a.norm[1] = p.k_norm;
    a.tokens = p.tokens, a.rope_rows = p.rope_rows;
    a.seqs = p.seqs, a.max_pages = p.max_pages, a.q_heads = p.q_heads, a.group = p.q_heads / c.kv_heads;
    a.rot_dim = p.rot_dim, a.interleaved = p.interleaved;
    a.eps = p.eps;
    a.err = g.err;
    cudaLaunchAttribute attr[1];
    const int64_t blocks = p.tokens / kKvBlock + 2 * (int64_t)p.seqs;
    const bool by_token = p.tokens < blocks;
    a.per = by_token ? 1 : kKvBlock, a.slack = by_token ? 0 : 2;
    const int64_t units = by_token ? p.tokens : blocks;
    // A decode batch has little to do for each head: as many heads to a CTA as
    // leave no more CTAs than four for each SM, which run at once (256 sequences of 8
    // kv heads and 32 query heads, with norms, no scale falling: 4 heads a CTA 5.7 us, 3 heads and a
    // second wave 8.2, 8 heads 6.7; one head a CTA and units of 16 tokens 22).
    const int per_unit = by_token ? (int)std::max((int64_t)1, std::min((int64_t)c.kv_heads, 4 * (int64_t)num_sms() / units))
                                  : (c.kv_heads + 1) / 2;  // CTAs
    a.heads_per_cta = (c.kv_heads + per_unit - 1) / per_unit;
    const dim3 grid((unsigned)units, (unsigned)((c.kv_heads + a.heads_per_cta - 1) / a.heads_per_cta));
    const cudaLaunchConfig_t cfg = config(grid, by_token ? 256 : 512, st, attr);
    return c.head_dim == 128 ? append_in<128>(cfg, a, p.in_dtype, p.out_dtype)
                             : append_in<64>(cfg, a, p.in_dtype, p.out_dtype);
}

cudaError_t launch_kv_gather(const bitnet_kv_cache &c, const int32_t *cu, const int32_t *table, int32_t seqs,
                             int32_t max_pages, int64_t tokens, void *k_out, void *v_out, int32_t dtype,
                             const DeviceGlobals &g, cudaStream_t st) {
    GatherArgs a;
    a.c = view_of(c);
    a.cu = cu, a.table = table;
    a.tokens = tokens;
    a.seqs = seqs, a.max_pages = max_pages;
    a.out[0] = k_out, a.out[1] = v_out;
    a.err = g.err;
    cudaLaunchAttribute attr[1];
    const dim3 grid((unsigned)(tokens / kGatherTokens + seqs), (unsigned)c.kv_heads);
    const cudaLaunchConfig_t cfg = config(grid, kGatherThreads, st, attr);
    return c.head_dim == 128 ? gather_out<128>(cfg, a, dtype) : gather_out<64>(cfg, a, dtype);
}

}  // namespace bitnet
