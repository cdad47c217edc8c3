// attn_prompt.cu -- attention over packed prompts on the tcgen05 tensor cores:
//   out = softmax(scale q k^T) v, causal or not, grouped heads, fp32 scores and
// sums, the weights rounded once to the inputs' 16-bit type.
//
// A CTA holds two 128-row tiles ("slots") of queries that share a kv head, and
// walks the keys 128 (heads of 64: 64, with two CTAs an SM) at a time.  The slots
// are neighbours in the order (row tile, head of the group), so they mostly are
// two heads on the same rows and need the same keys.  While the softmax of one
// slot runs on its warps, the tensor cores work on the other:
//   warps 0-3, 4-7  softmax of slot 0 / 1: thread = row.  Reads its scores
//                   from tensor memory, exponentials, writes the weights back
//                   over the scores as 16-bit operand A of the second product.
//   warp 8          TMA: both query tiles, then K and V tiles in a ring.
//   warp 9          issues the MMAs:  S = Q K^T (both from shared memory),
//                   O += P V (P from tensor memory, V with N contiguous), in
//                   the order PV0(j) S0(j+1) PV1(j) S1(j+1), which holds the
//                   slots half a step apart: with an issuer for each slot both
//                   softmaxes ran at the same time, then both slots' MMAs
//                   (566 us on 8192 tokens and 32 heads of 128).
//   warps 10, 11    check the bounds of 32 sequences, then V in the guarded tiles, beside
//                   the softmax of the same tile.
// Tensor memory: S0 | S1 | O0 | O1.
//
// The running maximum is only a reference: a row keeps it while its scores
// exceed it by less than 2^8, which leaves the weights inside fp16 (scaled, see kUp) and
// bf16, so O is rescaled (by the slot's softmax warps, in place) a few times per
// row at most instead of once per tile.  S of tile j complete means that
// PV of tile j-1 is (both are tracked by the commit after S), so O is free then.
//
// Scores outside a row's keys become -inf before they are used, so K rows of
// other sequences never reach a row.  A weight of 0 times a NaN or infinity would
// not be 0, so in the tiles that some row sees in part ("guarded": around the diagonal,
// or past the sequence's end; the last few) warps 10 and 11 look over V before the MMA
// takes it: rows behind the sequence's last become 0, and so does an element that is
// not finite, whose column and first key are kept and added to the rows that see it.
//
// Bound: the tensor cores' 4 D operations a score at D = 128, the softmax (a
// special function unit's exponential and about four instructions a score) at
// D = 64.  Causal, 32 heads on 8 kv heads, 8192 tokens, bf16: 426-440 us in a burst
// (1250-1290 TFLOP/s), 505-530 in calls one after another, whose clock the power
// limit lowers (1040-1090); heads of 64 (fp16): 388 us, 705 TFLOP/s.  Prompts of a few
// hundred tokens (16 x 512, the same heads of 64: 66 us) are a CTA's start, end and the
// imbalance of a few tiles.  The softmax's registers spill a little (ptxas: 12 bytes
// stored at heads of 128, 20 to 36 at 64).
//
// Every wait is bounded; a CTA whose wait ran out latches the error word, ends
// its copies and MMAs (bounded) and frees its tensor memory.
#include <limits.h>

#include <atomic>
#include <type_traits>

#include "attn.cuh"
#include "tcgen05_f16.cuh"

namespace bitnet {
namespace {

constexpr int kTile = 128;  // queries of a slot
constexpr int kSlots = 2;
constexpr int kTmaWarp = 8, kMmaWarp = 9, kGuardWarp = 10;
constexpr int kThreads = 384;  // three warpgroups: two softmax, one for loads and MMAs
constexpr int kGuarded = 5;    // most guarded tiles of a CTA: 256 rows and 64 keys that do not begin with a tile
constexpr int kParts = 2;      // the weights of a tile are handed to the MMA in two parts
constexpr uint32_t kDrainLimit = 1u << 22;
constexpr long long kDrainCycles = 2000000;  // ~1 ms
constexpr float kLag = 8.0f;                 // log2 units that scores may exceed the reference maximum by
// Weights are held at 2^kUp of their size.  fp16's would leave the normal numbers at 2^-14 of
// the reference and end at 2^-25, and a prompt's many small ones beside a large one
// are lost; from 2^(kLag + kUp) = 2^15 down to 2^-21 they are normal now.
template <typename T>
constexpr float kUp = std::is_same<T, __half>::value ? 7.0f : 0.0f;

struct Args {
    const int32_t *cu_q, *cu_k;
    void *out;
    float *lse;
    int64_t q_tokens, k_tokens;
    float scale_log2;  // |scale| * log2(e)
    int neg;           // scale < 0: the MMA negates q
    int seqs, q_heads, kv_heads, group, pairs_per_tile, causal;
    unsigned *err;
    const unsigned *wait_limit;
};

template <int D>
struct Cfg {
    // Keys of a step.  At D = 128 two slots of 128 x 128 scores and 128 x 128
    // output fill the tensor memory: one CTA an SM.  At D = 64 the softmax is what
    // bounds it, and 64 keys a step leave room for two CTAs, four slots, whose
    // waits for each other's MMAs overlap.
    static constexpr int kKeys = D == 64 ? 64 : 128;
    static constexpr int kCtas = D == 64 ? 2 : 1;
    static constexpr bool kMaxFirst = D == 64;
    static constexpr int kMoved = D == 64 ? 16 : 32;       // output columns rescaled at once (registers)
    static constexpr int kStages = D == 64 ? 6 : 4;        // K and V tiles in flight
    static constexpr int kChunks = kKeys / 32;             // of 32 scores
    static constexpr int kMmas = kKeys / 16;               // of a tile's second product
    // The first part of the weights: 96 of 128 keys, 32 of 64.  The second product
    // starts while the last exponentials run, and little of it is left after them.
    static constexpr int kFirstPart = D == 64 ? 2 : 6;     // MMAs
    static constexpr int kHalves = D / 64;                 // 128-byte wide pieces of a row
    static constexpr int kQPiece = kTile * 128;            // bytes of a piece of a query tile
    static constexpr int kPiece = kKeys * 128;             // ... of a K or V tile
    static constexpr int kQBytes = kHalves * kQPiece;
    static constexpr int kTileBytes = kHalves * kPiece;
    static constexpr int kOffKv = kSlots * kQBytes;
    static constexpr int kOffBar = kOffKv + kStages * kTileBytes;
    static constexpr int kOffFirst = kOffBar + 320;        // int[3][D]: first key of a column that is NaN, +inf, -inf
    static constexpr size_t kSmem = 1024 + kOffFirst + 3 * D * 4;
    // Tensor-memory columns: S0 | S1 | O0 | O1.
    static constexpr int kTmemCols = kSlots * (kKeys + D);
    // Registers: softmax threads hold a row of scores, the others little; the
    // shares add up to what the block is launched with (384 x 168, 384 x 80).
    static constexpr int kRegsSoftmax = D == 64 ? 104 : 224, kRegsOther = D == 64 ? 32 : 56;
    static __device__ __forceinline__ uint32_t s_at(int s) { return (uint32_t)(kKeys * s); }
    static __device__ __forceinline__ uint32_t o_at(int s) { return (uint32_t)(kSlots * kKeys + D * s); }
};

// NaN where an operand is.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// Two fp32 values in one 64-bit register, one instruction for both.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t ex2_unit(uint64_t y) {
    float a, b;
    unpack2(y, a, b);
    return pack2(ex2(a), ex2(b));
}
// 2^y without the special function unit, whose 16 a cycle and SM take as long
// for a tile's scores as the tile's two products do at D = 128: y = n + r with
// n the nearest integer, 2^r by a polynomial of degree 4 with constant 1,
// a minimax fit of the relative error on [-1/2, 1/2] (2^-18.4, far
// below the weights' 16-bit rounding), n added to the exponent.  From -127
// down (a masked score's -inf) it is 0, as 1's exponent field less 127 is: a
// masked value's weight times the type's largest value is nothing.
__device__ __forceinline__ uint64_t ex2_poly(uint64_t y) {
    float a, b;
    unpack2(y, a, b);
    const uint64_t x = pack2(fmaxf(a, -127.0f), fmaxf(b, -127.0f));
    const uint64_t t = add2(x, pack2(12582912.0f, 12582912.0f));  // 1.5 2^23: n in the low bits
    const uint64_t n = add2(t, pack2(-12582912.0f, -12582912.0f));
    const uint64_t r = fma2(n, pack2(-1.0f, -1.0f), x);
    uint64_t p = fma2(r, pack2(0.009582852945f, 0.009582852945f), pack2(0.05590642616f, 0.05590642616f));
    p = fma2(p, r, pack2(0.2402409911f, 0.2402409911f));
    p = fma2(p, r, pack2(0.6931241751f, 0.6931241751f));
    p = fma2(p, r, pack2(1.0f, 1.0f));
    float t0, t1, p0, p1;
    unpack2(t, t0, t1);
    unpack2(p, p0, p1);
    return pack2(__uint_as_float((__float_as_uint(t0) << 23) + __float_as_uint(p0)),
                 __uint_as_float((__float_as_uint(t1) << 23) + __float_as_uint(p1)));
}
// Of every kPolyOf pairs of scores, those whose exponentials are polynomials.  At
// D = 128, 8192 tokens and 32 heads: none 452, one 461, two 447, three 454, four
// 477 us (four prompts of 2048: 109, 108, 102, 104, 113).  At D = 64 the issue of
// instructions bounds it as much as the special function unit does: none 348, two
// 353, three 380 us.
constexpr int kPolyOf = 8;
template <int D>
constexpr int kPolyPairs = D == 128 ? 2 : 0;

template <int D, typename T, typename Out>
__global__ void __launch_bounds__(kThreads, Cfg<D>::kCtas)
attn_prompt_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const Args a) {
    using C = Cfg<D>;
    constexpr int kKeys = C::kKeys, kStages = C::kStages;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t bars = base + C::kOffBar;
    auto q_full = [&](int s) { return bars + 8u * s; };
    auto s_full = [&](int s) { return bars + 8u * (2 + s); };
    auto o_full = [&](int s) { return bars + 8u * (4 + s); };
    auto p_full = [&](int s, int part) { return bars + 8u * (6 + kParts * s + part); };
    auto kv_full = [&](int t) { return bars + 8u * (6 + kSlots * kParts + t); };
    auto kv_empty = [&](int t) { return kv_full(kStages + t); };
    // V of a guarded tile lands here (each is used once) and is full, in kv_full, when both guards have arrived there.
    auto v_land = [&](int g) { return kv_full(2 * kStages + g); };
    const uint32_t drain = kv_full(2 * kStages + kGuarded);
    static_assert((6 + kSlots * kParts + 2 * kStages + kGuarded + 1) * 8 + 12 <= C::kOffFirst - C::kOffBar, "barriers");
    const uint32_t tmem_slot = drain + 8u, abort_flag = drain + 12u, not_finite = drain + 16u;  // words
    auto first_at = [&](int kind, int d) { return base + C::kOffFirst + 4u * (kind * D + d); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // What needs no memory of an earlier kernel comes before the wait for it.
    if (threadIdx.x == 0) {
        for (int s = 0; s < kSlots; s++) {
            ptx::mbar_init(q_full(s), 1);
            ptx::mbar_init(s_full(s), 1);
            for (int part = 0; part < kParts; part++) ptx::mbar_init(p_full(s, part), 4);
            ptx::mbar_init(o_full(s), 1);
        }
        for (int t = 0; t < kStages; t++) {
            ptx::mbar_init(kv_full(t), 1 + (t & 1));  // odd stages hold V: two guards, or two arrivals of the loader
            ptx::mbar_init(kv_empty(t), 1);
        }
        for (int g = 0; g < kGuarded; g++) ptx::mbar_init(v_land(g), 1);
        ptx::mbar_init(drain, 1);
        ptx::sts_flag(abort_flag, 0);
        ptx::sts_flag(not_finite, 0);
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&map_q);
        ptx::prefetch_tmap(&map_k);
        ptx::prefetch_tmap(&map_v);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp >= kGuardWarp) {  // 32 sequences a CTA: there are more CTAs than sequences
        const int64_t i = (int64_t)blockIdx.x * 32 + lane;
        const bool of_q = warp == kGuardWarp;
        if (i < a.seqs) check_sequence(of_q ? a.cu_q : a.cu_k, of_q ? a.q_tokens : a.k_tokens, nullptr, i, a.err);
    }

    // The work: kv head, sequence, two neighbours of the list (row tile, head
    // of the group), the last rows (the longest walks) first.
    const int kvh = blockIdx.x % a.kv_heads;
    const int64_t rest = blockIdx.x / a.kv_heads;
    const int64_t unit = rest / a.pairs_per_tile;
    const int seq = find_seq(a.cu_q, a.seqs, unit, kTile, 1);
    const int64_t q0 = a.cu_q[seq], q1 = a.cu_q[seq + 1], k0 = a.cu_k[seq], k1 = a.cu_k[seq + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.q_tokens || k0 < 0 || k1 < k0 || k1 > a.k_tokens) return;  // latched by check_sequence
    const int lq = (int)(q1 - q0), lk = (int)(k1 - k0);
    const int64_t local = unit - unit_base(a.cu_q, seq, kTile, 1);
    const int64_t items = (int64_t)((lq + kTile - 1) / kTile) * a.group;
    const int64_t pairs = (items + 1) / 2;
    const int64_t pair = pairs - 1 - (local * a.pairs_per_tile + rest % a.pairs_per_tile);
    if (local < 0 || pair < 0) return;

    int row0[kSlots], head[kSlots], tiles[kSlots];  // first query, head, key tiles of each slot
    const int shift = lk - lq;                      // causal: query r sees keys up to r + shift
#pragma unroll
    for (int s = 0; s < kSlots; s++) {
        const int64_t item = 2 * pair + s;
        row0[s] = (int)(item / a.group) * kTile;
        head[s] = kvh * a.group + (int)(item % a.group);
        int keys = lk;
        if (a.causal) keys = min(lk, min(row0[s] + kTile, lq) + shift);
        tiles[s] = item < items && keys > 0 ? (keys + kKeys - 1) / kKeys : 0;
        if (item >= items) row0[s] = lq;  // no such row: nothing is written
    }
    const int most = max(tiles[0], tiles[1]);
    // Tiles before it are seen whole by every row of the slots.
    const int guard0 = max(0, a.causal ? min(lk, row0[0] + shift + 1) : lk) / kKeys;
    for (int i = threadIdx.x; i < 3 * D; i += kThreads) ptx::sts_flag(first_at(0, i), INT_MAX);
    const uint32_t limit = *a.wait_limit;

    if (warp == kMmaWarp) {
        ptx::tmem_alloc(tmem_slot, C::kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = ptx::lds_flag(tmem_slot);

    auto give_up = [&]() {
        ptx::sts_flag(abort_flag, 1);
        atomicOr(a.err, kErrTimeout);
    };
    auto kv_at = [&](int t) { return base + C::kOffKv + (uint32_t)(t % kStages) * C::kTileBytes; };

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
    if (warp == kTmaWarp) {
        // ------------------------------------------------ loads; step t: K of tile t / 2, then V
        if (lane == 0) {
            int issued = 0;
            static_assert(kStages % 2 == 0, "a stage holds K only or V only");
            auto guarded = [&](int t) { return (t & 1) && (t >> 1) >= guard0; };
            auto load = [&](uint32_t dst, const CUtensorMap *m, uint32_t bar, int h, int64_t row, int piece) {
                ptx::mbar_arrive_expect_tx(bar, C::kHalves * piece);
#pragma unroll
                for (int p = 0; p < C::kHalves; p++) ptx::tma_load_3d(dst + p * piece, m, bar, p * 64, h, (int)row);
            };
            bool ok = true;
            for (int t = 0; t < 2 * most && ok; t++) {
                if (t == 0 && tiles[0]) load(base, &map_q, q_full(0), head[0], q0 + row0[0], C::kQPiece);
                if (t >= kStages && !ptx::mbar_wait_flag(kv_empty(t % kStages), (t / kStages - 1) & 1, limit, abort_flag)) {
                    give_up();
                    ok = false;
                    break;
                }
                const uint32_t full = kv_full(t % kStages);
                load(kv_at(t), (t & 1) ? &map_v : &map_k, guarded(t) ? v_land((t >> 1) - guard0) : full, kvh,
                     k0 + (int64_t)(t >> 1) * kKeys, C::kPiece);
                if ((t & 1) && !guarded(t)) ptx::mbar_arrive(full);
                issued++;
                if (t == 0 && tiles[1]) load(base + C::kQBytes, &map_q, q_full(1), head[1], q0 + row0[1], C::kQPiece);
            }
            // No copy may be in flight when the CTA ends: wait (bounded) for
            // the last round of every stage, and the queries.
            auto landed = [&](uint32_t bar, uint32_t parity) {
                const long long t0 = clock64();
                while (!ptx::mbar_try_wait(bar, parity))
                    if (clock64() - t0 > kDrainCycles) break;
            };
            for (int t = max(0, issued - kStages); t < issued; t++)
                guarded(t) ? landed(v_land((t >> 1) - guard0), 0) : landed(kv_full(t % kStages), (t / kStages) & 1);
            for (int s = 0; s < kSlots; s++)
                if (tiles[s] && issued > 0) landed(q_full(s), 0);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------ MMA issuer
        // One lane does all of it.  Its instruction stream is as long as the
        // MMAs' time, so barriers are tried in groups (a try that succeeds still
        // takes about 100 cycles), each waited for only if its try failed.
        if (ptx::elect_one() && most > 0) {
            const uint32_t id_s = ptx::idesc_f16(kTile, kKeys, kBf16, false, a.neg != 0);
            constexpr uint32_t id_o = ptx::idesc_f16(kTile, D, kBf16, true);
            const uint64_t dq = ptx::desc_k_sw128(base), dk = ptx::desc_k_sw128(base + C::kOffKv),
                           dv = ptx::desc_mn_sw128(base + C::kOffKv, C::kPiece);
            const uint32_t q_lo = (uint32_t)dq, k_lo = (uint32_t)dk, v_lo = (uint32_t)dv;
            const uint32_t qk_hi = (uint32_t)(dq >> 32), v_hi = (uint32_t)(dv >> 32);
            const int n0 = tiles[0], n1 = tiles[1];
            bool ok = true;
            auto wait = [&](bool tried, uint32_t bar, uint32_t parity) {
                if (!tried && ok && !ptx::mbar_wait_flag(bar, parity, limit, abort_flag)) {
                    give_up();
                    ok = false;
                }
            };
            auto scores = [&](int s, int t) {  // S of slot s with the keys in stage t
                const uint32_t qs = q_lo + s * (C::kQBytes >> 4), ks = k_lo + t * (C::kTileBytes >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; k++)
                    ptx::mma_f16(tmem + C::s_at(s), qs + (k / 4) * (C::kQPiece >> 4) + 2 * (k % 4), qk_hi,
                                 ks + (k / 4) * (C::kPiece >> 4) + 2 * (k % 4), qk_hi, id_s, k > 0);
                ptx::mma_commit(s_full(s));
            };
            wait(false, kv_full(0), 0);
            if (n0) wait(false, q_full(0), 0);
            if (ok && n0) scores(0, 0);
            if (n1) wait(false, q_full(1), 0);
            if (ok && n1) scores(1, 0);
            ptx::mma_commit(kv_empty(0));
            for (int j = 0; j < most && ok; j++) {
                const int tv = (2 * j + 1) % kStages, tk = (2 * j + 2) % kStages;
                const uint32_t pv = ((2 * j + 1) / kStages) & 1, pk = ((2 * j + 2) / kStages) & 1;
                const uint32_t vs = v_lo + tv * (C::kTileBytes >> 4);
                const bool more = j + 1 < most;
#pragma unroll
                for (int s = 0; s < kSlots; s++) {
                    const int n = s ? n1 : n0;
                    if (j < n && ok) {
                        const bool got_v = ptx::mbar_try_wait(kv_full(tv), pv);
                        const bool got_a = ptx::mbar_try_wait(p_full(s, 0), j & 1);
                        const bool got_k = more && ptx::mbar_try_wait(kv_full(tk), pk);
                        const bool got_b = ptx::mbar_try_wait(p_full(s, 1), j & 1);
                        wait(got_v, kv_full(tv), pv);
                        wait(got_a, p_full(s, 0), j & 1);
                        if (!ok) break;
                        ptx::tc_fence_after();
#pragma unroll
                        for (int k = 0; k < C::kFirstPart; k++)
                            ptx::mma_f16_ta(tmem + C::o_at(s), tmem + C::s_at(s) + 8u * k, vs + k * (2048u >> 4), v_hi,
                                            id_o, j > 0 || k > 0);
                        wait(got_b, p_full(s, 1), j & 1);
                        if (j + 1 < n) wait(got_k, kv_full(tk), pk);
                        if (!ok) break;
                        ptx::tc_fence_after();
#pragma unroll
                        for (int k = C::kFirstPart; k < C::kMmas; k++)
                            ptx::mma_f16_ta(tmem + C::o_at(s), tmem + C::s_at(s) + 8u * k, vs + k * (2048u >> 4), v_hi,
                                            id_o, 1);
                        if (j + 1 < n)
                            scores(s, tk);
                        else
                            ptx::mma_commit(o_full(s));
                    }
                }
                // both slots are done with V of this tile and K of the next
                ptx::mma_commit(kv_empty(tv));
                if (more) ptx::mma_commit(kv_empty(tk));
            }
            ptx::mma_commit(drain);
            ptx::mbar_wait(drain, 0, kDrainLimit, nullptr);
        }
        __syncwarp();
    } else if (warp < 8) {
        // ------------------------------------------------ softmax and epilogue of a slot
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
        const int s = warp >> 2;
        const int n = s ? tiles[1] : tiles[0], r0 = s ? row0[1] : row0[0], h = s ? head[1] : head[0];
        const int r = r0 + (warp & 3) * 32 + lane;  // this thread's query
        const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + C::s_at(s) + quarter, to = tmem + C::o_at(s) + quarter;
        const float c = a.scale_log2;
        float ref = -INFINITY, l = 0.0f;
        // Rows behind the sequence's last are another sequence's queries: no vote on the reference.
        const float lag = r < lq ? kLag : INFINITY;
        int limit_col = lk;  // keys that the row sees
        if (a.causal) limit_col = min(lk, r + shift + 1);
        const int first_masked = (a.causal ? min(lk, r0 + shift + 1) : lk) / kKeys;  // tiles before it need no mask
        bool ok = true;
        for (int j = 0; j < n; j++) {
            if (!ptx::mbar_wait_flag(s_full(s), j & 1, limit, abort_flag)) {
                give_up();
                ok = false;
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            uint32_t v[C::kChunks][32];
#pragma unroll
            for (int q = 0; q < C::kChunks; q++) ptx::tmem_ld_32x32b_x32(ts + 32u * q, v[q]);
            ptx::tmem_wait_ld();
            if (j >= first_masked) {
                const int lim = limit_col - j * kKeys;
#pragma unroll
                for (int q = 0; q < C::kChunks; q++)
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        if (q * 32 + i >= lim) v[q][i] = 0xff800000u;  // -inf
            }
            auto val = [&](int i) { return __uint_as_float(v[i >> 5][i & 31]); };
            auto row_max = [&]() {
                float mx[4] = {val(0), val(1), val(2), val(3)};
#pragma unroll
                for (int i = 4; i < kKeys; i += 8)
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        mx[q] = i + 4 < kKeys ? max3(mx[q], val(i + q), val(i + 4 + q)) : max_nan(mx[q], val(i + q));
                return max_nan(max3(mx[0], mx[1], mx[2]), mx[3]);
            };
            auto passed = [&](float m) { return __any_sync(0xffffffffu, (m - ref) * c > lag); };
            auto move_ref = [&](float m) {  // to m, where m is above it; sums and output follow
                const float up = fmaxf(ref, m);
                const float f = up == -INFINITY ? 1.0f : ex2((ref - up) * c);
                ref = up;
                l *= f;
#pragma unroll
                for (int q = 0; q < D / C::kMoved; q++) {
                    uint32_t o[C::kMoved];
                    if constexpr (C::kMoved == 32)
                        ptx::tmem_ld_32x32b_x32(to + 32u * q, o);
                    else
                        ptx::tmem_ld_32x32b_x16(to + 16u * q, o);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < C::kMoved; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                    if constexpr (C::kMoved == 32)
                        ptx::tmem_st_32x32b_x32(to + 32u * q, o);
                    else
                        ptx::tmem_st_32x32b_x16(to + 16u * q, o);
                }
            };
            if (j == 0 || C::kMaxFirst) {
                const float m = row_max();
                if (j == 0)
                    ref = m;
                else if (passed(m))
                    move_ref(m);
            }
            // At D = 128 the exponentials start with the reference as it is, and
            // the maximum is found beside them; half the tile is done again in the
            // few tiles where the reference has to move.  (At D = 64 other slots
            // fill the time, and the registers for it are not there.)
            uint64_t sum[2];
            uint64_t c2 = pack2(c, c), mc2;
            auto weights = [&](int q) {  // columns 32 q .. 32 q + 31
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const uint64_t y = fma2(pack2(val(32 * q + 2 * i), val(32 * q + 2 * i + 1)), c2, mc2);
                    const uint64_t p = i % kPolyOf < kPolyPairs<D> ? ex2_poly(y) : ex2_unit(y);
                    sum[i & 1] = add2(sum[i & 1], p);
                    float p0, p1;
                    unpack2(p, p0, p1);
                    const typename Pair<T>::type x2 = Pair<T>::down(p0, p1);
                    w[i] = *reinterpret_cast<const uint32_t *>(&x2);
                }
                ptx::tmem_st_32x32b_x16(ts + 16u * q, w);
            };
            auto set_ref = [&]() {
                const float mc = ref == -INFINITY ? 0.0f : ref * c;
                mc2 = pack2(kUp<T> - mc, kUp<T> - mc);
                sum[0] = sum[1] = 0;
            };
            set_ref();
            if constexpr (C::kMaxFirst) {
                weights(0);
            } else {
                while (true) {
                    float mx[4];
#pragma unroll
                    for (int q = 0; q < 4; q++) mx[q] = val(q);
#pragma unroll
                    for (int q = 0; q < C::kChunks / 2; q++) {
                        weights(q);
#pragma unroll
                        for (int i = 4 + 64 * q; i < min(kKeys, 68 + 64 * q); i += 8)
#pragma unroll
                            for (int k = 0; k < 4; k++)
                                mx[k] = i + 4 < kKeys ? max3(mx[k], val(i + k), val(i + 4 + k)) : max_nan(mx[k], val(i + k));
                    }
                    const float m = max_nan(max3(mx[0], mx[1], mx[2]), mx[3]);
                    if (!(m < INFINITY)) l = NAN;  // a polynomial's weight of a NaN is 0
                    if (!passed(m)) break;
                    move_ref(m);
                    set_ref();
                }
            }
            if constexpr (C::kChunks == 4) weights(2);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(p_full(s, 0));
            weights(C::kChunks - 1);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(p_full(s, 1));
            float l0, l1;
            unpack2(add2(sum[0], sum[1]), l0, l1);
            l += l0 + l1;
        }
        bool hurt = false;  // values that are not finite, which the guards have taken out
        if (ok && n > 0) {
            // The guards are done with the slot's last V (the slots' walks differ by 128
            // rows, less than the ring holds: its stage has not gone on).
            static_assert(kTile / kKeys < kStages / 2, "phase of the last V");
            const int tv = 2 * n - 1;
            hurt = ptx::mbar_wait_flag(kv_full(tv % kStages), tv / kStages & 1, limit, abort_flag) && ptx::lds_flag(not_finite);
            if (!ptx::mbar_wait_flag(o_full(s), 0, limit, abort_flag)) {
                give_up();
                ok = false;
            }
            ok = __all_sync(0xffffffffu, ok);
            ptx::tc_fence_after();
        }
        // A row with a score that is NaN has l = NaN by now; one whose reference overflows
        // has no softmax either.  A row without keys has l = 0.
        if (!(ref * c < INFINITY)) l = NAN;
        if (ok) {
            const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
            Out *dst = static_cast<Out *>(a.out) + ((q0 + r) * a.q_heads + h) * D;
#pragma unroll
            for (int q = 0; q < D / 32; q++) {
                uint32_t o[32];
                float f[32];
                if (n > 0) {
                    ptx::tmem_ld_32x32b_x32(to + 32u * q, o);
                    ptx::tmem_wait_ld();
                }
#pragma unroll
                for (int i = 0; i < 32; i++) f[i] = l == 0.0f ? 0.0f : __uint_as_float(o[i]) * inv;
                if (r < lq) store_from_f32<32>(dst + 32 * q, f);
            }
            if (hurt && r < lq) {
#pragma unroll 1
                for (int d = 0; d < D; d++) {
                    float x = (float)dst[d];
                    if (ptx::lds_flag(first_at(0, d)) < limit_col) x = NAN;
                    if (ptx::lds_flag(first_at(1, d)) < limit_col) x += INFINITY;
                    if (ptx::lds_flag(first_at(2, d)) < limit_col) x -= INFINITY;
                    dst[d] = (Out)x;
                }
            }
            if (a.lse && r < lq)
                a.lse[(q0 + r) * a.q_heads + h] =
                    l == 0.0f ? -INFINITY : (ref * c + (log2f(l) - kUp<T>)) * 0.69314718055994531f;
        }
    } else if (warp >= kGuardWarp) {
        // ------------------------------------------------ V of the guarded tiles
        // Bound: the softmax beside it, whose time it mostly fits in.  3 prompts of up to 150
        // tokens take 9.6 us with it and 9.3 without, 8192 tokens the same; 16 ragged ones of
        // heads of 64 take 71 and 69, as long when no tile is guarded: the code around
        // is compiled otherwise.  (More loads at once in a lane: 451 us against 444 on 8192.)
        using P2 = typename Pair<T>::type;
        constexpr int kPieceChunks = C::kPiece / 16;
        constexpr uint32_t kInf = kBf16 ? 0x7f80u : 0x7c00u;
        const int me = (warp - kGuardWarp) * 32 + lane;
        for (int g = 0; g < most - guard0; g++) {
            bool ok = ptx::mbar_wait_flag(v_land(g), 0, limit, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                if (lane == 0) give_up();
                break;
            }
            const int key0 = (guard0 + g) * kKeys, keys = lk - key0;  // from this tile on
            unsigned char *const smem = smem_raw + (base - raw);
            uint4 *v = reinterpret_cast<uint4 *>(smem + (kv_at(2 * (guard0 + g) + 1) - base));
            // 16-byte chunk e of a piece is number e & 7 (swizzled) of row e / 8.
            const int own = min(keys, kKeys) * 8;
            P2 sum[4];  // of 0 times the values: NaN if one is not finite
#pragma unroll
            for (int i = 0; i < 4; i++) sum[i] = Pair<T>::down(0.0f, 0.0f);
#pragma unroll 1
            for (int p = 0; p < C::kHalves; p++) {
                uint4 *piece = v + p * kPieceChunks;
#pragma unroll 1
                for (int e = own + me; e < kPieceChunks; e += 64) piece[e] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
                for (int e = me; e < own; e += 64) {
                    const uint4 x = piece[e];
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        sum[k] = __hfma2(*reinterpret_cast<const P2 *>(&w[k]), Pair<T>::down(0.0f, 0.0f), sum[k]);
                }
            }
            const float2 all = up2(__hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3])));
            if (__any_sync(0xffffffffu, !(all.x + all.y == 0.0f))) {
#pragma unroll 1
                for (int e = me; e < C::kHalves * kPieceChunks; e += 64) {
                    const int row = e / 8 & (kKeys - 1), column = e / kPieceChunks * 64 + ((e ^ row) & 7) * 8;
                    unsigned short *x = reinterpret_cast<unsigned short *>(v + e);
#pragma unroll 1
                    for (int i = 0; i < 8; i++) {
                        if ((x[i] & kInf) != kInf) continue;
                        const int kind = (x[i] & 0x7fffu) != kInf ? 0 : x[i] == kInf ? 1 : 2;
                        atomicMin(reinterpret_cast<int *>(smem + (first_at(kind, column + i) - base)), key0 + row);
                        x[i] = 0;
                    }
                }
                if (lane == 0) ptx::sts_flag(not_finite, 1);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(kv_full((2 * (guard0 + g) + 1) % kStages));
        }
        __syncwarp();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, C::kTmemCols);
}

// [tokens][heads][dim] rows of `stride` elements, boxes of `rows` tokens x 64
// elements of one head; rows behind the last token read as 0.
bool make_map(CUtensorMap *m, const void *p, bool bf16, int dim, int heads, int64_t tokens, int64_t stride, int rows) {
    auto enc = tensor_map_encode();
    if (!enc) return false;
    if (tokens == 1 && stride < (int64_t)heads * dim) stride = (int64_t)heads * dim;  // one row: no stride is used
    cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(p), dims,
               strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, typename T, typename Out>
cudaError_t launch(const bitnet_attn_prompt_args &p, const Args &a, cudaStream_t st) {
    static std::atomic<bool> configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(attn_prompt_kernel<D, T, Out>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)Cfg<D>::kSmem);
        if (e != cudaSuccess) return e;
        configured[dev].store(true, std::memory_order_release);
    }
    constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, p.q, bf16, D, p.q_heads, p.q_tokens, p.q_stride, kTile)) return cudaErrorInvalidValue;
    if (p.k_tokens > 0) {
        if (!make_map(&mk, p.k, bf16, D, p.kv_heads, p.k_tokens, p.k_stride, Cfg<D>::kKeys) ||
            !make_map(&mv, p.v, bf16, D, p.kv_heads, p.k_tokens, p.v_stride, Cfg<D>::kKeys))
            return cudaErrorInvalidValue;
    } else {
        mk = mv = mq;  // no keys: not used
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.q_tokens / kTile + p.seqs) * a.pairs_per_tile * p.kv_heads));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<D>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_prompt_kernel<D, T, Out>, mq, mk, mv, a);
}

template <int D>
cudaError_t launch_t(const bitnet_attn_prompt_args &p, const Args &a, cudaStream_t st) {
    if (p.dtype == BITNET_BF16)
        return p.out_dtype == BITNET_F32 ? launch<D, __nv_bfloat16, float>(p, a, st)
                                         : launch<D, __nv_bfloat16, __nv_bfloat16>(p, a, st);
    return p.out_dtype == BITNET_F32 ? launch<D, __half, float>(p, a, st) : launch<D, __half, __half>(p, a, st);
}

}  // namespace

cudaError_t launch_attn_prompt(const bitnet_attn_prompt_args &p, const DeviceGlobals &g, cudaStream_t st) {
    Args a;
    a.cu_q = p.cu_q, a.cu_k = p.cu_k;
    a.out = p.out, a.lse = p.lse;
    a.q_tokens = p.q_tokens, a.k_tokens = p.k_tokens;
    a.neg = p.scale < 0.0f;
    // A scale of 0 stays above 0, so that -inf times it is -inf.
    a.scale_log2 = fmaxf((float)(fabs((double)p.scale) * 1.4426950408889634), 1e-30f);
    a.seqs = p.seqs, a.q_heads = p.q_heads, a.kv_heads = p.kv_heads, a.group = p.q_heads / p.kv_heads;
    a.pairs_per_tile = (a.group + 1) / 2;
    a.causal = p.causal;
    a.err = g.err;
    a.wait_limit = g.wait_limit;
    return p.head_dim == 128 ? launch_t<128>(p, a, st) : launch_t<64>(p, a, st);
}

}  // namespace bitnet
