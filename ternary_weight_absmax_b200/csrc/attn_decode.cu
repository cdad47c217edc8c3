// attn_decode.cu -- attention of one token per sequence over the paged int8
// cache:  out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q.k_t - max).
//
// Bound: the cache is read from HBM (2 D bytes a token and kv head), once for up to
// 8 query heads of a kv head; larger groups go through it once for each 8 (the
// second time mostly from L2: 64 x 4k, 16 query heads on each of 2 kv heads, 58 us).
// Measured, heads of 128: 64 x 4k, 32 on 8 heads, fp32 104 us (4.6 TB/s), bf16 96;
// 8 x 32k, bf16 96 us (5.5 TB/s); 1 x 131071, 5 kv heads, bf16 40 us, 9 of them start
// and join; 1 x 700 8.6 us.  Short sequences are bound by latency (256 x 500, 2 kv
// heads of 64: 25 us, 1.3 TB/s).
//
// Products, on the warp-level MMAs, transposed so that tokens (scores) and
// elements (output) are the 16 rows and up to 8 query heads the 8 columns: the
// output of a head takes half the registers that heads as rows would.  At 8 heads a
// kv head no row or column idles; at 4 half of the columns do.
//   Scores (m16n8k32, int8, exact int32 sums): codes are operands as they are.
//   A query is v m / 8355000 with m its head's largest element and v a 24-bit
//   integer, split into three signed bytes (bf16 calls: 16 bits, two bytes), an
//   MMA each; the three sums become one fp32 score.  The rounding of v, 2^-24 of
//   m, is fp32's own on the largest element.
//   Output (m16n8k16, fp16, fp32 sums): codes are exact in fp16 (byte | 0x6400
//   is 1024 + code + 128, one subtraction gives the code); a softmax weight
//   enters as two fp16 parts, hi = rn(w), lo = rn(w - hi), two MMAs into the same
//   sums.  bf16 calls take one part: an fp16 weight's half step is an eighth of
//   the output's.  (fp16 calls take two: one would double the error.)
//
// Memory.  One lane of each warp copies 16- or 32-token tiles of K and V rows
// by TMA into the warp's own ring of kStages tiles (plain asynchronous copies of
// the same bytes stalled in the load unit, at 3.6 TB/s).  The TMA's swizzle puts
// the 16-byte chunks of 8 consecutive rows in 8 different bank groups, so that
// ldmatrix reads them without conflicts: K rows as the first product's operand
// as they are, V transposed in pairs of elements, which are an m-tile's rows g
// and g + 8.  The weights, a column of which a lane has after the first product
// and a row of which it needs for the second, are transposed by movmatrix.
// Nothing but the two products' operands passes through registers.
//
// Split.  All tiles (32 tokens of one sequence and kv head, up to 8 query
// heads) lie on one line, sequence by sequence; each warp takes an equal run of
// it, by itself: no barrier between warps after the lengths are summed.  The
// lengths are read on the device, so the same launch (and captured graph) serves
// any lengths.  A unit (a sequence's kv head) that lies in one run is finished
// there; else each warp leaves its maximum, sum and weighted values in the
// workspace, and a second kernel, started by programmatic dependent launch, joins
// them in the order of the line.  (Runs of CTAs, whose warps were joined in
// shared memory at the end of each unit, lost 10 to 40 % of a batch in those
// joins; joining the parts in the last CTA to arrive at a counter cost 6.7 us of a
// 13.7 us call, fences and the atomic being dearer than a dependent launch.)

#include <atomic>
#include <type_traits>

#include "attn.cuh"
#include "tcgen05.cuh"

namespace bitnet {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;       // tokens of a warp's step
constexpr int kStages = 3;      // tiles of a warp's ring: the present one and the next two
constexpr int kLens = 512;      // lengths kept in shared memory (those of more sequences are read again)
constexpr int kHeads = 8;       // query heads of a unit
constexpr int kMaxCtas = 1024;  // bound of the grid, for the workspace's size
constexpr long long kDrainCycles = 2000000;  // ~1 ms
constexpr float kWeightScale = 16384.0f;  // softmax weights enter the MMA as w 2^14: far above fp16's smallest step

// How a unit lies on the line: in one run (parts 1: finished there), or in the
// runs of warps first, first + 1, ...; the part of the first is its second one if
// the unit begins inside its run.
struct __align__(16) Split {
    int parts, first, inside, pad;
};

struct Args {
    const float *ks, *vs;
    int64_t num_pages;
    int kv_heads, page_shift;
    const void *q;
    int64_t q_stride;
    const int32_t *seq_len, *table;
    int seqs, max_pages;
    int q_heads, group, chunks, per_chunk;  // group split into chunks of per_chunk <= 8 heads
    float scale_log2;                       // scale * log2(e)
    void *out;
    float *lse;
    Split *splits;  // [units], by the warp whose run the unit begins in
    float *parts;   // [warps][2]: the part of the unit that began before the run, of that which goes on behind
    unsigned *err;
    const unsigned *wait_limit;
};

// CTAs an SM: at D = 128 two leave the registers that the kernel wants (three of
// 168 registers, with a tile less each, took 106 us against 104 on 64 x 4k).
// At D = 64 four of 128 registers took 23.7 us against 24.9 on 256 x 500, but 12.6
// against 11.5 on 40 x 250 with 8 kv heads and 16.1 against 15.1 on 20 x 750.
constexpr int ctas_per_sm(int head_dim) { return head_dim == 64 ? 3 : 2; }

template <int D>
struct Cfg {
    static constexpr int kSide = kTile * D;         // bytes of K or V of a tile
    static constexpr int kStageBytes = 2 * kSide;
    static constexpr int kPart = kHeads * (D + 2);  // floats of a part: max, sum, values
    static constexpr size_t kRing = (size_t)kWarps * kStages * kStageBytes;
    static constexpr size_t kSmem = 1024 + kRing + kWarps * kStages * 8;
    // Byte offset of 16-byte chunk `chunk` of row r, as the TMA's swizzle (128 or 64 bytes) leaves it.
    static __device__ __forceinline__ uint32_t at(int r, int chunk) {
        return (uint32_t)(r * D + ((chunk ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4));
    }
};

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
// Bytes `sel` picks from w (codes + 128) as two fp16 codes.
template <uint32_t kSel>
__device__ __forceinline__ uint32_t codes2(uint32_t w) {
    const uint32_t h = prmt(w, 0x64646464u, kSel);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&h), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An integer below 2^22 in magnitude as fp32, by an addition to 1.5 2^23.
__device__ __forceinline__ float small_int(int x) { return __int_as_float(0x4b400000 + x) - 12582912.0f; }
// x as fp16 parts, two values at a time: hi, and what is left where kTwo.
template <bool kTwo>
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x, y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    if constexpr (kTwo) {
        const float2 f = __half22float2(h);
        const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    }
}
// An 8 x 8 matrix of fp16, two of a row a lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// 2^e and the exponent of x, for normal numbers.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int exponent(float x) { return ((__float_as_int(x) >> 23) & 255) - 127; }

// N output elements from their weighted sum, and the row's lse where it is asked for.
template <int N, typename T>
__device__ __forceinline__ void finish(T *out, float *lse, float m, float l, float (&s)[N]) {
    const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);  // no tokens: 0; a score that is NaN: NaN
#pragma unroll
    for (int k = 0; k < N; k++) s[k] *= inv;
    store_from_f32<N>(out, s);
    if (lse) *lse = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D))
attn_decode_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const Args a) {
    using C = Cfg<D>;
    constexpr bool kTwo = !std::is_same<T, __nv_bfloat16>::value;  // weights in two fp16 parts
    constexpr int kBytes = kTwo ? 3 : 2;                           // of a query's integer
    constexpr float kLargest = kTwo ? 8355000.0f : 32600.0f;       // below 127 (65536 + 256 + 1), 127 (256 + 1)
    constexpr int kM = D / 16;             // m-tiles of the second product
    constexpr int kK = D / 32;             // k-steps of the first
    extern __shared__ unsigned char smem_raw[];
    __shared__ int64_t scan_total[kWarps];
    __shared__ int lens[kLens];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t ring = base + (uint32_t)(warp * kStages * C::kStageBytes);
    const uint32_t bars = base + (uint32_t)C::kRing + (uint32_t)(warp * kStages * 8);
    if (lane == 0) {
        for (int i = 0; i < kStages; i++) ptx::mbar_init(bars + 8 * i, 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&map_k);
        ptx::prefetch_tmap(&map_v);
    }
    __syncwarp();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // A try may be suspended for as long as a copy takes: at a cap of one a wait has
    // none, and runs out for certain.
    const uint32_t limit = *a.wait_limit - 1;
    uint32_t tile_no = 0;  // tiles that this warp has asked for: the stage and its phase
    bool ok = true;        // no wait has run out

    const int units = a.kv_heads * a.chunks;  // units of a sequence: kv head by kv head, chunk by chunk
    const int64_t limit_len = (int64_t)a.max_pages << a.page_shift;
    auto tiles_of = [&](int len) -> int {
        if (len < 0 || len > limit_len) len = 0;
        return len ? (len - 1) / kTile + 1 : 1;  // an empty sequence has one tile without tokens
    };
    const bool kept = a.seqs <= kLens;

    // Tiles of all sequences, and the run of the line that is this warp's.
    int64_t total = 0;
    for (int i = tid; i < a.seqs; i += kThreads) {
        const int len = a.seq_len[i];
        if (kept) lens[i] = len;
        total += tiles_of(len);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) scan_total[warp] = total;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kWarps; w++) total += scan_total[w];
    auto len_of = [&](int i) -> int { return kept ? lens[i] : a.seq_len[i]; };
    total *= units;
    if (total > 0x7fff0000) {  // positions on the line are 32-bit
        if (tid == 0) atomicOr(a.err, kErrBounds);
        for (int64_t u = (int64_t)blockIdx.x * kThreads + tid; u < (int64_t)a.seqs * units; u += (int64_t)gridDim.x * kThreads)
            a.splits[u].parts = 0;
        return;
    }
    const int all = (int)total, workers = (int)gridDim.x * kWarps, me = (int)blockIdx.x * kWarps + warp;
    const int per = max(1, (all + workers - 1) / workers);
    const int begin = me * per, end = min(begin + per, all);
    if (begin >= end) return;

    // The sequence that `begin` lies in, and its first tile: every warp walks the lengths 32 at a time.
    int seq = a.seqs - 1;
    int seq_base = 0;
    for (int i0 = 0; i0 < a.seqs; i0 += 32) {
        const int i = i0 + lane;
        const int t = i < a.seqs ? tiles_of(len_of(i)) * units : 0;
        int incl = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        const unsigned past = __ballot_sync(0xffffffffu, seq_base + incl > begin);
        if (past) {
            const int w = __ffs(past) - 1;
            seq = i0 + w;
            seq_base += __shfl_sync(0xffffffffu, incl - t, w);
            break;
        }
        seq_base += __shfl_sync(0xffffffffu, incl, 31);
    }

    // The present unit, and this warp's tiles of it: my0, my0 + 1, ...
    const bool paired = a.page_shift > 4;  // a tile's two blocks lie in one page
    int at = begin, len = 0, count = 1, first = 0, stop = 0, kvh = 0, head0 = 0, heads = 0, my0 = 0, steps = 0, unit = 0;
    const int32_t *table = nullptr;
    int page0 = 0, page1 = 0;  // pages of the tile to ask for next
    float sc[kStages - 1];     // lanes 0-3: scales of the tiles asked for, the oldest first
#pragma unroll
    for (int i = 0; i < kStages - 1; i++) sc[i] = 1.0f;

    // The page of a block: read a tile before it is used, so that no check
    // waits for it here.  (An ordinary load, as that of the scales: the non-coherent path
    // is for memory that no one writes while the kernel runs, and this one starts
    // beside the append.)
    auto page_of = [&](int blk) -> int {
        return (int64_t)blk * kKvBlock < len ? table[blk << 4 >> a.page_shift] : 0;
    };
    auto pages_of = [&](int t) {
        page0 = page_of(2 * t);
        if (!paired) page1 = page_of(2 * t + 1);
    };
    // A block's first row in the cache, or -1 (no tokens, bad page).
    auto row_of = [&](int blk, int page) -> int {
        if ((int64_t)blk * kKvBlock >= len) return -1;
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) atomicOr(a.err, kErrBounds);
            return -1;
        }
        return ((page * a.kv_heads + kvh) << a.page_shift) + (blk << 4 & ((1 << a.page_shift) - 1));  // below 2^31
    };
    // Asks for tile t: its rows by TMA into the next stage, its scales into
    // `scale` of lanes 0-3 (K and V of the first block, of the second).  A block that is
    // not there leaves what the stage held (finite codes, masked later).
    auto fetch = [&](int t, float &scale) {
        const int r0 = row_of(2 * t, page0);
        const int r1 = paired && r0 >= 0 ? r0 + kKvBlock : row_of(2 * t + 1, page1);
        if (lane == 0) {
            const uint32_t stage = tile_no % kStages, dst = ring + stage * C::kStageBytes, bar = bars + 8 * stage;
            ptx::mbar_arrive_expect_tx(bar, (uint32_t)((r0 >= 0) + (r1 >= 0)) * (2 * kKvBlock * D));
            if (r0 >= 0) {
                ptx::tma_load_2d(dst, &map_k, bar, 0, r0);
                ptx::tma_load_2d(dst + C::kSide, &map_v, bar, 0, r0);
            }
            if (r1 >= 0 && !paired) {
                ptx::tma_load_2d(dst + kKvBlock * D, &map_k, bar, 0, r1);
                ptx::tma_load_2d(dst + C::kSide + kKvBlock * D, &map_v, bar, 0, r1);
            }
        }
        tile_no++;
        const int r = lane & 2 ? r1 : r0;
        const bool have = r >= 0 && (2 * t + (lane >> 1 & 1)) * kKvBlock < len;
        if (lane < 4 && have) scale = (lane & 1 ? a.vs : a.ks)[r >> 4];
    };
    // Moves on to the unit that `at` lies in, and asks for its first tiles.
    auto begin_unit = [&]() {
        len = len_of(seq);
        count = tiles_of(len);
        while (at >= seq_base + count * units) {
            seq_base += count * units;
            seq++;
            len = len_of(seq);
            count = tiles_of(len);
        }
        unit = (at - seq_base) / count;  // tiles [first, first + count) of the line
        first = seq_base + unit * count;
        stop = min(end, first + count);
        kvh = unit / a.chunks;
        const int chunk = unit - kvh * a.chunks;
        head0 = kvh * a.group + chunk * a.per_chunk;
        heads = min(a.per_chunk, a.group - chunk * a.per_chunk);
        if (len < 0 || len > limit_len) {
            if (lane == 0) atomicOr(a.err, kErrBounds);
            len = 0;
        }
        table = a.table + (int64_t)seq * a.max_pages;
        my0 = at - first;
        steps = stop - at;
        if (ok) {
            pages_of(my0);
            const int p0 = page0, p1 = page1;
            if (steps > 1) pages_of(my0 + 1);
            const int q0 = page0, q1 = page1;
            if (steps > 2) pages_of(my0 + 2);
            const int r0 = page0, r1 = page1;
            page0 = p0, page1 = p1;
            fetch(my0, sc[0]);
            page0 = q0, page1 = q1;
            if (steps > 1) fetch(my0 + 1, sc[1]);
            page0 = r0, page1 = r1;
        }
    };
    // Queries: lane (g, c) has elements 16 e + 4c .. +3 of head g.
    float qv[2 * kK][4];
    auto load_q = [&]() {
        const T *q = static_cast<const T *>(a.q) + (int64_t)seq * a.q_stride + (int64_t)(head0 + g) * D;
#pragma unroll
        for (int e = 0; e < 2 * kK; e++) {
#pragma unroll
            for (int i = 0; i < 4; i++) qv[e][i] = 0.0f;
            if (g < heads) load_f32<4>(q + e * 16 + c * 4, qv[e]);
        }
    };

    begin_unit();
    load_q();
    while (true) {
        // The queries as bytes of integers, four elements to a register.
        uint32_t qb[kBytes][2 * kK];
        float factor[2];  // of the scores of heads 2c, 2c + 1
        {
            // A query that is not finite makes m NaN or infinite, its integers 0 and,
            // by 0 times the factor, every score NaN.
            float m = 1e-30f;
#pragma unroll
            for (int e = 0; e < 2 * kK; e++)
#pragma unroll
                for (int i = 0; i < 4; i++) m = max_nan(m, fabsf(qv[e][i]));
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const float up = __fdiv_rn(kLargest, m), row = a.scale_log2 * __fdiv_rn(m, kLargest);
            factor[0] = __shfl_sync(0xffffffffu, row, 8 * c);
            factor[1] = __shfl_sync(0xffffffffu, row, 8 * c + 4);
#pragma unroll
            for (int e = 0; e < 2 * kK; e++) {
#pragma unroll
                for (int x = 0; x < kBytes; x++) qb[x][e] = 0;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    int v = __float2int_rn(qv[e][i] * up);
#pragma unroll
                    for (int x = 0; x < kBytes; x++) {  // lowest byte first, each signed
                        const int byte = x + 1 < kBytes ? (int)(int8_t)v : v;
                        qb[x][e] |= (uint32_t)(byte & 255) << (8 * i);
                        v = (v - byte) >> 8;
                    }
                }
            }
        }

        float o[kM][4];
#pragma unroll
        for (int j = 0; j < kM; j++)
#pragma unroll
            for (int i = 0; i < 4; i++) o[j][i] = 0.0f;
        float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.0f, 0.0f};  // heads 2c, 2c + 1
        // The output's sums are in units of 2^e_run / 2^14, 2^e_run the power of
        // two in the largest value step (1 / scale) so far.
        int e_run = -100;

        for (int s = 0; s < steps && ok; s++) {
            const uint32_t now = tile_no - min(kStages - 1, steps - s);  // this tile's number
            ok = ptx::mbar_wait(bars + 8 * (now % kStages), now / kStages & 1, limit, nullptr);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                if (lane == 0) atomicOr(a.err, kErrTimeout);
                break;
            }
            const float scales = sc[0];
            sc[0] = sc[1];
            if (s + kStages - 1 < steps) fetch(my0 + s + kStages - 1, sc[1]);
            if (s + kStages < steps) pages_of(my0 + s + kStages);
            const uint32_t src = ring + now % kStages * C::kStageBytes;
            const int left = len - (my0 + s) * kTile;  // tokens from this tile on

            // Scores: d[0], d[1] token g of the block, heads 2c and 2c + 1; d[2], d[3]
            // token g + 8.
            float sv[2][4], vinv[2];
            float m_new[2] = {m_run[0], m_run[1]};
#pragma unroll
            for (int b = 0; b < 2; b++) {
                int di[kBytes][4];
#pragma unroll
                for (int x = 0; x < kBytes; x++)
#pragma unroll
                    for (int i = 0; i < 4; i++) di[x][i] = 0;
#pragma unroll
                for (int t = 0; t < kK; t++) {
                    // matrices: rows 0-7 and 8-15 of chunk 2t, then of chunk 2t + 1
                    uint32_t x[4];
                    ldsm(x, src + C::at(b * kKvBlock + (lane & 15), 2 * t + (lane >> 4)));
#pragma unroll
                    for (int k = 0; k < kBytes; k++) mma(di[k], x[0], x[1], x[2], x[3], qb[k][2 * t], qb[k][2 * t + 1]);
                }
                float d[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    d[i] = small_int(di[kBytes - 1][i]);
#pragma unroll
                    for (int k = kBytes - 2; k >= 0; k--) d[i] = fmaf(d[i], 256.0f, small_int(di[k][i]));
                }
                const int have = left - b * kKvBlock;  // tokens of this block
                const float ks = __frcp_rn(__shfl_sync(0xffffffffu, scales, 2 * b));
                const float vs = __frcp_rn(__shfl_sync(0xffffffffu, scales, 2 * b + 1));
                vinv[b] = have > 0 ? vs : 0.0f;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    sv[b][i] = g + 4 * (i & 2) < have ? d[i] * (ks * factor[i & 1]) : -INFINITY;
                    m_new[i & 1] = fmaxf(m_new[i & 1], sv[b][i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; i++) {
                m_new[i] = fmaxf(m_new[i], __shfl_xor_sync(0xffffffffu, m_new[i], 4));
                m_new[i] = fmaxf(m_new[i], __shfl_xor_sync(0xffffffffu, m_new[i], 8));
                m_new[i] = fmaxf(m_new[i], __shfl_xor_sync(0xffffffffu, m_new[i], 16));
            }
            // What the sums so far are multiplied by, as this tile's are added.
            const int e_new = max(e_run, exponent(fmaxf(vinv[0], vinv[1])));
            const float fe = pow2(max(-126, e_run - e_new));
            float f[2], m_use[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                m_use[i] = m_new[i] == -INFINITY ? 0.0f : m_new[i];
                f[i] = ex2(m_run[i] - m_use[i]);
                l_run[i] *= f[i];
                f[i] *= fe;
                m_run[i] = m_new[i];
            }
            e_run = e_new;
            const float to_unit = pow2(max(-126, -e_run)) * kWeightScale;
            uint32_t ph[2][2], pl[2][2];
#pragma unroll
            for (int b = 0; b < 2; b++) {
                float p[4];
                const float vf = vinv[b] * to_unit;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    p[i] = ex2(sv[b][i] - m_use[i & 1]);
                    l_run[i & 1] += p[i];
                    p[i] *= vf;
                }
                split2<kTwo>(p[0], p[1], ph[b][0], pl[b][0]);
                split2<kTwo>(p[2], p[3], ph[b][1], pl[b][1]);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    ph[b][i] = transposed(ph[b][i]);
                    if constexpr (kTwo) pl[b][i] = transposed(pl[b][i]);
                }
            }
            // The MMA cuts its fp32 sums off; a tile's products are summed on their
            // own and join the running sums by an fma, which rounds (one MMA after
            // the other into the running sums left 4000 tokens 2e-6 off).
#pragma unroll
            for (int j = 0; j < kM; j += 2) {
                float t[2][4];
#pragma unroll
                for (int i = 0; i < 4; i++) t[0][i] = t[1][i] = 0.0f;
#pragma unroll
                for (int b = 0; b < 2; b++) {
                    // matrices: tokens 0-7 and 8-15 of chunk j, then of chunk j + 1,
                    // transposed: (t0 e0, t0 e1, t1 e0, t1 e1) with tokens 2c, 2c + 1
                    // and elements 2g, 2g + 1 of the chunk
                    uint32_t w[4];
                    ldsm_t(w, src + C::kSide + C::at(b * kKvBlock + (lane & 15), j + (lane >> 4)));
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const uint32_t x = w[2 * i] ^ 0x80808080u, y = w[2 * i + 1] ^ 0x80808080u;
                        const uint32_t va[4] = {codes2<0x4240>(x), codes2<0x4341>(x), codes2<0x4240>(y), codes2<0x4341>(y)};
                        mma(t[i], va, ph[b][0], ph[b][1]);
                        if constexpr (kTwo) mma(t[i], va, pl[b][0], pl[b][1]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; i++)
#pragma unroll
                    for (int x = 0; x < 4; x++) o[j + i][x] = fmaf(o[j + i][x], f[x & 1], t[i][x]);
            }
            __syncwarp();  // every lane has read the stage before it is asked for again
        }
        if (!ok) {  // no copy may be in flight when the CTA ends or reuses the ring
            const long long t0 = clock64();
            for (uint32_t n = tile_no - min(tile_no, (uint32_t)kStages); n < tile_no; n++)
                while (!ptx::mbar_try_wait(bars + 8 * (n % kStages), n / kStages & 1) && clock64() - t0 < kDrainCycles) {
                }
            __syncwarp();
        }

        // The next unit's first tiles are under way while this one is finished.
        const int heads_c = heads;
        const bool inside = first > begin;  // this warp's part is its first one, but for a unit that begins inside its run
        if (lane == 0 && first >= begin)
            a.splits[(int64_t)seq * units + unit] = {(first + count - 1) / per - me + 1, me, inside, 0};
        const int64_t row = (int64_t)seq * a.q_heads + head0;
        const bool whole = at == first && stop == first + count;
        at = stop;
        const bool more = at < end;
        if (more) {
            begin_unit();
            load_q();
        }
        float *part = a.parts + (2 * (int64_t)me + (inside ? 1 : 0)) * C::kPart;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 4);
            l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 8);
            l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 16);
            // lane (g, c) has elements 16 j + 2g, + 1 of heads 2c, 2c + 1
            const int h = 2 * c + i;
            if (h >= heads_c) continue;
            const float f = 1.0f / kWeightScale * pow2(e_run);
#pragma unroll
            for (int j = 0; j < kM; j++) {
                float x[2] = {o[j][i] * f, o[j][2 + i] * f};
                if (whole)
                    finish<2>(static_cast<T *>(a.out) + (row + h) * D + 16 * j + 2 * g,
                              a.lse && j == 0 && g == 0 ? a.lse + row + h : nullptr, m_run[i], l_run[i], x);
                else
                    store_from_f32<2>(part + 2 * kHeads + h * D + 16 * j + 2 * g, x);
            }
            if (!whole && g == 0) part[h] = m_run[i], part[kHeads + h] = l_run[i];
        }
        if (!more) break;
    }
}

// Joins parts k, k + step, ... of a unit's head h, elements d .. d + V - 1 of
// them, into m, l, s; several parts are in flight.
template <int D, int V>
__device__ __forceinline__ void join_parts(const Args &a, const Split &sp, int h, int d, int k0, int step, float &m, float &l,
                                           float (&s)[V]) {
    constexpr int kFlight = V == 1 ? 12 : 8;
    m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < V; i++) s[i] = 0.0f;
    for (; k0 < sp.parts; k0 += kFlight * step) {
        float pm[kFlight], pl[kFlight], t[kFlight][V];
#pragma unroll
        for (int j = 0; j < kFlight; j++) {
            const int k = k0 + j * step;
            pm[j] = -INFINITY, pl[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < V; i++) t[j][i] = 0.0f;
            if (k < sp.parts) {
                const float *p = a.parts + (2 * (int64_t)(sp.first + k) + (k == 0 ? sp.inside : 0)) * Cfg<D>::kPart;
                pm[j] = p[h], pl[j] = p[kHeads + h];
                if constexpr (V == 1)
                    t[j][0] = p[2 * kHeads + h * D + d];
                else
                    load_f32<V>(p + 2 * kHeads + h * D + d, t[j]);
            }
        }
        float mn = m;
#pragma unroll
        for (int j = 0; j < kFlight; j++) mn = fmaxf(mn, pm[j]);
        const float use = mn == -INFINITY ? 0.0f : mn, f0 = ex2(m - use);
        l *= f0;
#pragma unroll
        for (int i = 0; i < V; i++) s[i] *= f0;
#pragma unroll
        for (int j = 0; j < kFlight; j++) {
            const float f = ex2(pm[j] - use);
            l += pl[j] * f;
#pragma unroll
            for (int i = 0; i < V; i++) s[i] += t[j][i] * f;
        }
        m = mn;
    }
}

// The same over the W warps of a CTA; the result is the first warp's.
template <int D, int V, int W>
__device__ __forceinline__ void join_cta(const Args &a, const Split &sp, int h, int d, float &m, float &l, float (&s)[V]) {
    __shared__ float sm[W], sl[W], sums[W][32 * V];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    join_parts<D, V>(a, sp, h, d, warp, W, m, l, s);
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int i = 0; i < V; i++) sums[warp][lane * V + i] = s[i];
    __syncthreads();
    if (warp > 0) return;
    const float lm = lane < W ? sm[lane] : -INFINITY;
    m = lm;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float f = m == -INFINITY ? 0.0f : ex2(lm - m);
    l = lane < W ? sl[lane] * f : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
    for (int i = 0; i < V; i++) s[i] = 0.0f;
#pragma unroll
    for (int x = 0; x < W; x++) {
        const float fx = __shfl_sync(0xffffffffu, f, x);
#pragma unroll
        for (int i = 0; i < V; i++) s[i] = fmaf(sums[x][lane * V + i], fx, s[i]);
    }
}

// Output row of head h of unit u; -1 if it has no such head.  (A call whose units
// pass 32 bits has more tiles than positions, and no parts.)
__device__ __forceinline__ int64_t row_of_head(const Args &a, int64_t u, int h) {
    const unsigned kv = (unsigned)u / (unsigned)a.chunks, chunk = (unsigned)u - kv * a.chunks;
    const unsigned seq = kv / (unsigned)a.kv_heads, kvh = kv - seq * a.kv_heads;
    if (h >= a.group - (int)chunk * a.per_chunk) return -1;
    return (int64_t)seq * a.q_heads + (int)(kvh * a.group + chunk * a.per_chunk) + h;
}
// Its elements from d on, and its lse.
template <int D, typename T, int V>
__device__ __forceinline__ void finish_row(const Args &a, int64_t row, int d, float m, float l, float (&s)[V]) {
    T *out = static_cast<T *>(a.out) + row * D + d;
    float *lse = a.lse && d == 0 ? a.lse + row : nullptr;
    if constexpr (V == 1) {
        const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
        *out = (T)(s[0] * inv);
        if (lse) *lse = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    } else {
        finish<V>(out, lse, m, l, s);
    }
}

// Joins a unit that lies in parts: W warps take head blockIdx.y of it, a lane
// holding D / (32 Z) elements of slice blockIdx.z.
template <int D, typename T, int W, int Z>
__global__ void __launch_bounds__(32 * W)
attn_decode_join_kernel(const Args a) {
    constexpr int V = D / (32 * Z);
    const int h = blockIdx.y, d = blockIdx.z * 32 * V + (threadIdx.x & 31) * V;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t u = blockIdx.x;
    const Split sp = a.splits[u];
    const int64_t row = row_of_head(a, u, h);
    if (sp.parts < 2 || row < 0) return;
    float m, l, s[V];
    join_cta<D, V, W>(a, sp, h, d, m, l, s);
    if (threadIdx.x < 32) finish_row<D, T, V>(a, row, d, m, l, s);
}

// The same for many units, a warp each.  How many parts a unit lies in is known
// here only: one long sequence among many short ones can have nearly all of
// them, and takes the CTA's warps together (131071 tokens and 299 sequences of 32,
// one head: 154 us with a warp for each unit, 41 so; 100000 and 63 of 100, 8 heads: 88
// and 70).  Neighbouring units, a sequence's heads, are in different CTAs.
constexpr int kAlone = 16;  // parts that a warp joins by itself, in two rounds of loads
template <int D, typename T>
__global__ void __launch_bounds__(256)
attn_decode_join_many_kernel(const Args a, int64_t units) {
    constexpr int V = D / 32;
    __shared__ Split split[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y, d = lane * V;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t u = (int64_t)warp * gridDim.x + blockIdx.x;
    Split sp = {0, 0, 0, 0};
    if (u < units) sp = a.splits[u];
    const int64_t row = row_of_head(a, u, h);
    if (row < 0) sp.parts = 0;
    if (lane == 0) split[warp] = sp;
    const bool any = __syncthreads_or(sp.parts > kAlone);
    float m, l, s[V];
    if (sp.parts >= 2 && sp.parts <= kAlone) {
        join_parts<D, V>(a, sp, h, d, 0, 1, m, l, s);
        finish_row<D, T, V>(a, row, d, m, l, s);
    }
    if (!any) return;
    for (int i = 0; i < 8; i++) {
        const Split one = split[i];
        if (one.parts <= kAlone) continue;
        join_cta<D, V, 8>(a, one, h, d, m, l, s);
        if (warp == 0) finish_row<D, T, V>(a, row_of_head(a, (int64_t)i * gridDim.x + blockIdx.x, h), d, m, l, s);
        __syncthreads();  // the first warp has read what the others left
    }
}

// The cache's codes as rows of head_dim bytes, boxes of a tile's rows in one page.
bool make_map(CUtensorMap *m, const int8_t *codes, const bitnet_kv_cache &c) {
    auto enc = tensor_map_encode();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.num_pages * c.kv_heads * c.page_size};
    cuuint64_t strides[1] = {(cuuint64_t)c.head_dim};
    cuuint32_t box[2] = {(cuuint32_t)c.head_dim, (cuuint32_t)(c.page_size >= kTile ? kTile : kKvBlock)};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(codes), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, c.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, typename T>
cudaError_t launch(const Args &a, const bitnet_kv_cache &cache, int grid, cudaStream_t st) {
    static std::atomic<bool> configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(attn_decode_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)Cfg<D>::kSmem);
        if (e != cudaSuccess) return e;
        configured[dev].store(true, std::memory_order_release);
    }
    CUtensorMap mk, mv;
    if (!make_map(&mk, cache.k, cache) || !make_map(&mv, cache.v, cache)) return cudaErrorInvalidValue;
    static_assert(kStages == 3, "a unit begins with two tiles, whose scales wait in two registers");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<D>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attn_decode_kernel<D, T>, mk, mv, a);
    if (e != cudaSuccess) return e;
    // On average a unit has warps / units parts and one more: up to five are one
    // warp's, up to about 100 a CTA's of eight (32 x 750, 5 kv heads, seven parts: 15.2
    // us either way; 8 x 32k, 64 units: 95 us, with a warp's 111); beyond, a CTA of 32
    // warps takes a slice of 32 elements (1 x 700: 8.7 us, with a warp's 14.6).  More
    // CTAs of eight warps than the SMs hold at once cost more than the parts: those
    // units are a warp's too (150 x 250, heads of 64, 2 kv heads of 8 heads: 15.8 ->
    // 11.1 us; 100 x 1500: 22.0 -> 20.0; 64 x 4k, 16 on each of 2 heads of 128: 61.9 -> 58.2).
    const int64_t units = (int64_t)a.seqs * a.kv_heads * a.chunks, warps = (int64_t)grid * kWarps;
    cfg.dynamicSmemBytes = 0;
    if (units * 4 >= warps || units * a.per_chunk > 8 * num_sms()) {
        cfg.gridDim = dim3((unsigned)((units + 7) / 8), (unsigned)a.per_chunk);
        cfg.blockDim = dim3(256);
        return cudaLaunchKernelEx(&cfg, attn_decode_join_many_kernel<D, T>, a, units);
    }
    cfg.gridDim = dim3((unsigned)units, (unsigned)a.per_chunk);
    if (units * 100 >= warps) {
        cfg.blockDim = dim3(32 * 8);
        return cudaLaunchKernelEx(&cfg, attn_decode_join_kernel<D, T, 8, 1>, a);
    }
    cfg.gridDim.z = D / 32;
    cfg.blockDim = dim3(32 * 32);
    return cudaLaunchKernelEx(&cfg, attn_decode_join_kernel<D, T, 32, D / 32>, a);
}

template <int D>
cudaError_t launch_t(const Args &a, const bitnet_kv_cache &c, int grid, int dtype, cudaStream_t st) {
    switch (dtype) {
        case BITNET_F32: return launch<D, float>(a, c, grid, st);
        case BITNET_BF16: return launch<D, __nv_bfloat16>(a, c, grid, st);
        default: return launch<D, __half>(a, c, grid, st);
    }
}

int grid_ctas(int head_dim) {
    const int g = num_sms() * ctas_per_sm(head_dim);
    return g < kMaxCtas ? g : kMaxCtas;
}

}  // namespace

// The units' records, then the parts.
static size_t splits_bytes(int32_t seqs, int32_t q_heads, int32_t kv_heads) {
    const int group = q_heads / kv_heads;
    return align_up((size_t)seqs * kv_heads * ((group + kHeads - 1) / kHeads) * sizeof(Split), 256);
}

size_t attn_decode_workspace_bytes(int32_t seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    return splits_bytes(seqs, q_heads, kv_heads) + (size_t)grid_ctas(head_dim) * kWarps * 2 * kHeads * (head_dim + 2) * 4;
}

cudaError_t launch_attn_decode(const DecodeCall &d, const DeviceGlobals &g, cudaStream_t st) {
    Args a;
    a.ks = d.c.k_scale, a.vs = d.c.v_scale;
    a.num_pages = d.c.num_pages;
    a.kv_heads = d.c.kv_heads;
    a.page_shift = 0;
    while ((1 << a.page_shift) < d.c.page_size) a.page_shift++;
    a.q = d.q, a.q_stride = d.q_stride;
    a.seq_len = d.seq_len, a.table = d.table;
    a.seqs = d.seqs, a.max_pages = d.max_pages;
    a.q_heads = d.q_heads, a.group = d.q_heads / d.c.kv_heads;
    a.chunks = (a.group + kHeads - 1) / kHeads;
    a.per_chunk = (a.group + a.chunks - 1) / a.chunks;
    a.scale_log2 = (float)((double)d.scale * 1.4426950408889634);
    a.out = d.out, a.lse = d.lse;
    const int grid = grid_ctas(d.c.head_dim);
    a.splits = static_cast<Split *>(d.workspace);
    a.parts = reinterpret_cast<float *>(static_cast<char *>(d.workspace) + splits_bytes(d.seqs, d.q_heads, d.c.kv_heads));
    a.err = g.err;
    a.wait_limit = g.wait_limit;
    return d.c.head_dim == 128 ? launch_t<128>(a, d.c, grid, d.dtype, st) : launch_t<64>(a, d.c, grid, d.dtype, st);
}

}  // namespace bitnet
