// Causal attention of whole prompts: packed sequences whose q, k and v lie
// next to each other, before (or without) any trip through the paged pool
// ("Inside vLLM", page 1, "Run forward pass", step 3: all sequences flattened
// into one super sequence, each attending to its own tokens only). For token
// i of a sequence and query head h:
//
//   out_i = sum_{j <= i} p_j v_j / sum_{j <= i} p_j,   p_j = 2^(s_j - m)
//   s_j = scale * log2(e) * q_i . k_j,                 m a reference near max s
//
// A work item is up to two 128-row query tiles, A and B (rows = tokens x the
// q heads of one kv head, token-major; B holds the tokens after A's), of one
// sequence and kv head, over key tiles of 128. Per key tile, K and V are
// copied once (one TMA box each) and serve both tiles:
//   S_t = Q_t K^T     tcgen05.mma, bf16 operands in 128-byte-swizzled shared
//                     memory, fp32 accumulator in TMEM;
//   P_t               one thread per row: S to registers, causal mask,
//                     exponentials against a running reference that moves (O
//                     rescaled) only when some p outgrows 2^14; bf16 pairs in
//                     TMEM, handed on in two parts so that the product of the
//                     first keys runs during the exponentials of the last;
//   O_t += P_t V      tcgen05.mma, A = P_t from TMEM, B = V as it lies.
// The softmax of A runs while the tensor core works for B and the other way
// round. (Where there are few items, an item is one query tile, and A and B are
// its even and odd key tiles, joined at the end.) The sums l are of the unrounded
// p; P is rounded to bf16 (at most 2^-8 of each term, half a step), since a
// product's operands have one type and V is bf16. It shows: rms error 0.0019 to
// 0.0020 of the output against 64 bits, where the output's own rounding makes
// 0.0016. The rounding of the reference is one step of m for a whole row and
// falls out; see row_scale() for scores so large that it would not.
//
// Warps: 0 MMA issue and TMEM, 1 copies and the item list, 2-3 guard of V, 4-7
// softmax of A, 8-11 of B, 12-15 output. The host does not know the lengths, and
// no workspace is needed: items are numbered by tile level (longest keys first)
// over all sequences, every CTA counts the tiles once, and its copy warp finds
// an item by a binary search over levels. Each probe reads every sequence, which
// is nothing at 24 and what sets the time at thousands (prompts of 200 tokens: 4.8
// us an item and SM with 150 of them, 5.6 with 700, 17 with 4000). The launch
// has a block for every item there may be; the blocks that start (one an SM)
// fetch the items of the others from the hardware one by one, so that an SM
// takes its next item when it is ready for it. (Items dealt out in turn left
// the last SM working 17 % longer than the average on ragged prompts.)
//
// Bound, for long prompts, by the turn from a P product to the S that takes over
// its columns and by softmax parts that come late: the tensor core is at work
// 69 % of the time. Measured, over several boxes: 4 prompts of 4096 tokens, 32/8
// heads of 128: 373 to 383 us, 1.44 to 1.47 PFLOP/s (0.75 to 0.77 of the 1.92
// measured for a large bf16 product); one of 16384: 1342 to 1372 us, 1.60 to 1.64
// PFLOP/s; 24 ragged ones of 16 to 2048: 57 to 60 us, 0.82 to 0.86 PFLOP/s, where
// items of three key tiles start and end as long as they run. With heads of 64
// (6 prompts of 700 to 4096: 68 to 69 us) neither the tensor core (34 %) nor the
// exponentials (34 %) fill the time: two softmax warps a scheduler wait for TMEM.
//
// Every wait is bounded; on a timeout the CTA raises PKV_DEV_TIMEOUT, stops,
// lets its copies and MMAs in flight finish and frees its TMEM.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <cstdint>
#include <mutex>

#include "pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_short_wait.cuh"

namespace pkv {
namespace {

constexpr int kRows = 128, kKeys = 128;
constexpr int kMmaWarp = 0, kCopyWarp = 1, kGuardWarp = 2, kSoftmaxWarp = 4, kOutWarp = 12;
constexpr int kThreads = 512;
// Registers a thread: the softmax holds a row of 128 scores and 32 words of P.
// Four warpgroups of 128 at launch: 2 * (72 + 184) = 4 * 128.
constexpr int kSoftmaxRegs = 184, kOtherRegs = 72;
constexpr uint32_t kTmemCols = 512;
// TMEM columns: S_A 0, S_B 128, O_A 256, O_B 256 + D. P lies over the first
// half of its S for D = 128, where nothing is left; for D = 64 it has columns of
// its own, 384 and 448, and the next S need not wait for the product of P.
constexpr uint32_t kColO = 256;
template <int D>
constexpr bool kOwnP = D == 64;
template <int D>
__device__ __forceinline__ constexpr uint32_t col_p(int t) {
    return kOwnP<D> ? 384 + t * 64 : t * 128;
}
// P is handed on in two parts of 96 and 32 keys: the product of the first (six
// MMAs, 384 cycles) runs while the second is made, and little is left to do
// once the second is there.
constexpr int kFirstKeys = 96;
constexpr float kRescaleBits = 14.f, kRescaleSum = 16384.f;  // P stays <= 2^14, exact in bf16's range and in l
constexpr int kSlots = 4;                 // items between the copy warp and the output
constexpr int kNoGuard = INT_MAX;
constexpr int kGuardTiles = 3;            // an item's at most 256 tokens touch at most three key tiles
constexpr int kSeqCache = 4096;           // sequences whose tile counts are kept in shared memory
constexpr float kLog2e = 1.4426950408889634f;

struct PromptArgs {
    const __nv_bfloat16 *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    __nv_bfloat16 *out;
    const int32_t *qsl;
    int num_tokens, num_reqs, num_q_heads, num_kv_heads, group;
    int tile_tokens, item_tokens;  // tokens of a query tile (128 / group), of an item
    float scale;
    int wide_out;  // out is on a 32-byte boundary
    int32_t *status;
};

// One work item: tokens [i0, i0 + 2 tile_tokens) of the sequence of n tokens
// that starts at token q0; n_keys[t]: key tiles that query tile t sees; guard:
// kNoGuard, or the first key tile that some row sees only in part, when the
// item is done again because an output was not finite.
struct Item {
    int valid, q0, n, i0, h, n_keys[2], guard;
};

struct Bars {
    static constexpr int kQFull = 0, kQEmpty = 2, kSFull = 4, kPFull = 6 /* [tile][part] */, kPvDone = 10, kOFull = 12,
                         kLFull = 14, kOFree = 16, kSTaken = 18, kDrain = 20, kBlock = 21, kDFull = 22, kDEmpty = kDFull + kSlots,
                         kBadFull = kDEmpty + kSlots, kKvFull = kBadFull + kSlots;
};

// Key tiles whose K and V an item copies: those that its tiles share, or, where
// they split the keys, all of both.
template <bool kSplit>
__device__ __forceinline__ int item_tiles(const Item &w) {
    return kSplit ? w.n_keys[0] + w.n_keys[1] : max(w.n_keys[0], w.n_keys[1]);
}

__device__ __forceinline__ Item guarded(Item w) {
    w.guard = w.i0 / kKeys;
    return w;
}

template <int D>
struct Smem {
    static constexpr int kStages = D == 128 ? 4 : 8;  // K and V tiles in turn
    static constexpr int kHalf = 16384;               // 128 rows x 128 B (64 bf16 columns)
    static constexpr int kTile = (D / 64) * kHalf;
    static constexpr int kOffQ = 0;
    static constexpr int kOffKv = 2 * kTile;
    static constexpr int kOffItem = kOffKv + kStages * kTile;
    static constexpr int kOffBlock = kOffItem + kSlots * (int)sizeof(Item);  // the launch control's answer
    static constexpr int kOffBar = kOffBlock + 16;
    static constexpr int kBars = Bars::kKvFull + 4 * kStages;  // K/V full, empty; guarded V: there, safe
    static constexpr int kOffSum = kOffBar + kBars * 8;  // float [tile][row]: sums of p
    static constexpr int kOffMax = kOffSum + 2 * kRows * 4;  // float [tile][row]: references (split items)
    static constexpr int kOffBad = kOffMax + 2 * kRows * 4;  // bits [slot][guarded tile][key]
    static constexpr int kOffRedo = kOffBad + kSlots * kGuardTiles * (kKeys / 8);  // int [slot]
    static constexpr int kOffSeq = kOffRedo + kSlots * 4;
    static constexpr int kBytes = kOffSeq + kSeqCache * 4;
    static constexpr int kAlloc = kBytes + 1024;
};
static_assert(Smem<128>::kAlloc <= 232448 - 1024, "prompt kernel shared memory");
static_assert(Smem<64>::kAlloc <= 232448 - 1024, "prompt kernel shared memory");

// Cluster launch control: asks the hardware for a block of this launch that
// has not started, to be done here instead; its index is ~0 when none is left
// (after which there must be no further request).
__device__ __forceinline__ void block_request(void *answer, uint64_t *bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(answer)),
                 "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ uint32_t block_answer(const void *answer) {
    uint32_t index;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\tld.shared.b128 h, [%1];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tmov.u32 %0, 0xffffffff;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n\t}"
        : "=r"(index)
        : "r"(smem_u32(answer))
        : "memory");
    return index;
}

__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// A value that all lanes hold, as the compiler can know it too.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_or_sync(0xffffffffu, v); }

// pkv_device.cuh's umma_..._warp forms with the shared-memory matrix descriptors
// (128-byte swizzle) as their two words, and its commit by address: what changes
// from MMA to MMA is one 32-bit sum, which stays in a uniform register, where
// 64-bit descriptors and generic pointers did not. The low word holds the address
// and the leading offset, the high one is the same for every operand here (8-row
// groups 1024 bytes apart).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
    return ((addr & 0x3FFFF) >> 4) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi));
}

// Ties the values to this place among the volatile instructions: what is
// computed from them cannot move ahead of it.
__device__ __forceinline__ void keep(float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]),
                          "+f"(v[i + 6]), "+f"(v[i + 7]));
}

// P = 2^(s * scale - m) of 32 keys as bf16 pairs, and the sums of the unrounded
// values. One exponential a value on the MUFU (8 lanes a cycle per SM quarter),
// everything else on packed pairs.
__device__ __forceinline__ void exps(const float (&s)[32], float scale_log2, float m, float2 (&sum)[2], uint32_t *p) {
    const float2 sc = make_float2(scale_log2, scale_log2), nm = make_float2(-m, -m);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float2 z = ffma2(make_float2(s[2 * e], s[2 * e + 1]), sc, nm);
        const float2 v = make_float2(fast_exp2(z.x), fast_exp2(z.y));
        sum[e & 1] = fadd2(sum[e & 1], v);
        p[e] = pack_bf16x2(v.x, v.y);
    }
}

__device__ __forceinline__ float max32(const float (&s)[32]) {
    float a = fmaxf(s[0], s[1]), b = fmaxf(s[2], s[3]);
#pragma unroll
    for (int e = 4; e < 32; e += 4) {
        a = fmax3(a, s[e], s[e + 1]);
        b = fmax3(b, s[e + 2], s[e + 3]);
    }
    return fmaxf(a, b);
}

__device__ __forceinline__ void store_p(uint32_t col, const uint32_t (&p)[48]) {
    uint32_t a[32], b[16];
#pragma unroll
    for (int i = 0; i < 32; ++i) a[i] = p[i];
#pragma unroll
    for (int i = 0; i < 16; ++i) b[i] = p[32 + i];
    tmem_st32u(col, a);
    tmem_st16u(col + 32, b);
}

// Item tiles of sequence r; 0 for an empty or a bad one (bad: reported).
__device__ __forceinline__ int seq_tiles(const PromptArgs &a, int r, bool report) {
    const int q0 = __ldg(a.qsl + r), q1 = __ldg(a.qsl + r + 1);
    if (q0 < 0 || q1 < q0 || q1 > a.num_tokens) {
        if (report) raise_status(a.status, PKV_DEV_BAD_QSL);
        return 0;
    }
    return (int)(((uint32_t)(q1 - q0) + a.item_tokens - 1) / (uint32_t)a.item_tokens);
}

__device__ __forceinline__ __nv_bfloat162 pair_of(uint32_t w) { return *reinterpret_cast<__nv_bfloat162 *>(&w); }
// Whether one of a word's two bf16 values is infinite or NaN (all exponent
// bits set): their complements' exponent fields have a zero half.
__device__ __forceinline__ bool odd_pair(uint32_t w) {
    const uint32_t x = ~w & 0x7f807f80u;
    return ((x - 0x00010001u) & ~x & 0x80008000u) != 0;
}
__device__ __forceinline__ bool odd_value(uint32_t bf16_bits) { return (bf16_bits & 0x7f80u) == 0x7f80u; }
__device__ __forceinline__ uint32_t clean_pair(uint32_t w) {
    return (odd_value(w) ? 0u : w & 0xffffu) | (odd_value(w >> 16) ? 0u : w & 0xffff0000u);
}

// The noted keys' values that are not finite, added to the output row of token
// i, just written by this thread, for the keys it sees: their probability is
// above 0, whatever it is, and what they are added to is not finite then.
template <int D>
__device__ __forceinline__ void add_bad(const PromptArgs &a, const Item &w, const uint32_t *bad, int i, __nv_bfloat16 *dst) {
#pragma unroll 1
    for (int b = 0; b < kGuardTiles * (kKeys / 32); ++b) {
        uint32_t bits = bad[b];
        while (bits) {
            const int key = w.guard * kKeys + b * 32 + __ffs(bits) - 1;
            bits &= bits - 1;
            if (key > i) continue;
            const __nv_bfloat16 *v = a.v + ((long long)w.q0 + key) * a.v_stride + w.h * D;
#pragma unroll 1
            for (int e = 0; e < D; ++e) {
                const float x = __bfloat162float(v[e]);
                if (!(fabsf(x) < INFINITY)) dst[e] = __float2bfloat16_rn(__bfloat162float(dst[e]) + x);
            }
        }
    }
}

// To 2^-23 of the value, a step and a half of fp32; the output is rounded to 2^-8.
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The scale of a row whose reference is the score m: the call's, or, where that
// would take the reference past 2^30, a power of two that does not. scale * s -
// reference is rounded once and so keeps the reference's own rounding, half a
// step of it: below 2^5 up to 2^30, and soon more than p has exponents for; with
// a power of two there is none. Scores of that size that differ at all are 2^5
// apart with either scale, so that the largest alone counts.
__device__ __forceinline__ float row_scale(float scale, float m) {
    const float cap = rcp(fabsf(m) * 0x1p-30f);
    return fminf(scale, __uint_as_float(__float_as_uint(cap) & 0x7f800000u));
}

// Columns [c, c + 32) of an output row: O / l, rounded, in 32-byte stores
// (16-byte stores, a sector half filled, held the output warps twice as long)
// that pass by L1, whose memory the operands are read from too (24 ragged prompts
// 64.0 -> 60.3 us; through shared memory and TMA 63.8).
__device__ __forceinline__ void put_row(bool wide, bool valid, int c, float inv, float (&o)[32], __nv_bfloat162 &odd,
                                        __nv_bfloat16 *dst) {
    const float2 inv2 = make_float2(inv, inv);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        const float2 v = fmul2(make_float2(o[e], o[e + 1]), inv2);
        o[e] = v.x;
        o[e + 1] = v.y;
    }
    if (!valid) return;
    uint32_t p[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        p[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
        odd = __hfma2(pair_of(p[e]), __floats2bfloat162_rn(0.f, 0.f), odd);
    }
    if (wide) {
#pragma unroll
        for (int e = 0; e < 16; e += 8)
            asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + c + 2 * e),
                         "r"(p[e]), "r"(p[e + 1]), "r"(p[e + 2]), "r"(p[e + 3]), "r"(p[e + 4]), "r"(p[e + 5]),
                         "r"(p[e + 6]), "r"(p[e + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<uint4 *>(dst + c + 2 * e) = make_uint4(p[e], p[e + 1], p[e + 2], p[e + 3]);
    }
}

template <int D, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
              const __grid_constant__ CUtensorMap v_map, const __grid_constant__ PromptArgs a) {
    using M = Smem<D>;
    constexpr int kStages = M::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_abort, s_levels;
    __shared__ unsigned long long s_tiles;
    __shared__ uint32_t s_tmem;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + M::kOffBar);
    uint64_t *q_full = bar + Bars::kQFull, *q_empty = bar + Bars::kQEmpty, *s_full = bar + Bars::kSFull;
    uint64_t *p_full = bar + Bars::kPFull, *pv_done = bar + Bars::kPvDone, *d_full = bar + Bars::kDFull;
    uint64_t *d_empty = bar + Bars::kDEmpty, *o_full = bar + Bars::kOFull, *l_full = bar + Bars::kLFull;
    uint64_t *o_free = bar + Bars::kOFree, *s_taken = bar + Bars::kSTaken, *drain = bar + Bars::kDrain;
    float *row_sum = reinterpret_cast<float *>(smem + M::kOffSum);
    float *row_ref = reinterpret_cast<float *>(smem + M::kOffMax);
    uint64_t *bad_full = bar + Bars::kBadFull;
    uint64_t *kv_full = bar + Bars::kKvFull, *kv_empty = kv_full + kStages, *v_safe = kv_empty + kStages;
    uint64_t *v_guard = v_safe + kStages;
    uint32_t *bad_keys = reinterpret_cast<uint32_t *>(smem + M::kOffBad);
    volatile int *redo = reinterpret_cast<volatile int *>(smem + M::kOffRedo);
    Item *items = reinterpret_cast<Item *>(smem + M::kOffItem);
    int *seq = reinterpret_cast<int *>(smem + M::kOffSeq);
    volatile int *abort = &s_abort;
    int32_t *status = a.status;
    // broadcast: the compiler then knows that a role's branch is the whole warp's (see uniform())
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

    if (warp == kCopyWarp) {
        // barriers by index, with the arrivals that each waits for
        if (lane == 0) {
            s_abort = 0;
            s_levels = 0;
            s_tiles = 0;
        }
        if (lane < kSlots) redo[lane] = 0;
        for (int i = lane; i < M::kBars; i += 32) {
            const bool four = (i >= Bars::kPFull && i < Bars::kPFull + 4) || (i >= Bars::kLFull && i < Bars::kLFull + 2) ||
                              (i >= Bars::kOFree && i < Bars::kOFree + 2) || (i >= Bars::kSTaken && i < Bars::kSTaken + 2);
            const int v_safe0 = Bars::kKvFull + 2 * kStages;
            const bool two = (i >= Bars::kBadFull && i < Bars::kBadFull + kSlots) ||
                             (i >= v_safe0 && i < v_safe0 + kStages);
            // an item's description: the MMA, guard, softmax and output warps
            const bool all = i >= Bars::kDEmpty && i < Bars::kDEmpty + kSlots;
            mbar_init(bar + i, all ? 15 : four ? 4 : two ? 2 : 1);
        }
        mbar_fence_init();
    }
    if (warp == kGuardWarp && lane == 0) {
        tma_prefetch_desc(&q_map);
        tma_prefetch_desc(&k_map);
        tma_prefetch_desc(&v_map);
    }
    pdl_launch_dependents();
    pdl_wait();
    // not before the wait: the kernel before may have TMEM to take yet
    if (warp == kMmaWarp) tmem_alloc(&s_tmem, kTmemCols);
    __syncthreads();
    {
        int most = 0;
        unsigned long long sum = 0;
#pragma unroll 1
        for (int r = threadIdx.x; r < a.num_reqs; r += kThreads) {
            const int n = seq_tiles(a, r, true);
            if (r < kSeqCache) seq[r] = n;
            most = max(most, n);
            sum += n;
        }
        // One atomic a warp: a 64-bit one in shared memory tries again while
        // others are at it.
        most = __reduce_max_sync(0xffffffffu, most);
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (sum && lane == 0) {
            atomicMax(&s_levels, most);
            atomicAdd(&s_tiles, sum);
        }
    }
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tm = s_tmem;
    if (warp == kCopyWarp) {
        // ------------------------ items, Q, K and V ------------------------
        setmaxnreg_dec<kOtherRegs>();
        const uint32_t Hkv = a.num_kv_heads;
        const int R = a.num_reqs;
        // More items than the launch has blocks: the sequences overlap, and
        // none is computed.
        uint32_t total = 0;
        if (s_tiles * Hkv <= gridDim.x) {
            total = (uint32_t)s_tiles * Hkv;
        } else if (lane == 0) {
            raise_status(status, PKV_DEV_BAD_QSL);
        }
        auto tiles_of = [&](int r) { return r < kSeqCache ? seq[r] : seq_tiles(a, r, false); };
        // Items of level m or above (level m: a sequence's m-th pair of query
        // tiles, so m grows with the keys seen).
        auto items_from = [&](int m) {
            uint32_t c = 0;
#pragma unroll 1
            for (int r = lane; r < R; r += 32) c += max(0, tiles_of(r) - m);
            return __reduce_add_sync(0xffffffffu, c) * Hkv;
        };
        // Items come in rising order, so the search goes on downward; were one
        // to come out of order, it would start anew.
        int hi = s_levels;        // items_from(hi) <= the item looked for
        uint32_t above = 0;       // items_from(hi)
        uint32_t x = 0;           // K and V tiles issued
        uint32_t q_used = 0, q_any = 0;  // bit t: parity of Q_t's tiles copied; any copied
        uint32_t g_used = 0, g_any = 0;  // by stage: guarded V tiles copied
        bool ok = true;
        // Item `it` of the launch.
        auto find = [&](uint32_t it) {
            Item w{};
            if (it < total) {
                // largest level m with items_from(m) > it
                if (it < above) {
                    hi = s_levels;
                    above = 0;
                }
                int lo = 0;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    const uint32_t c = items_from(mid);
                    if (c > it) {
                        lo = mid;
                    } else {
                        hi = mid;
                        above = c;
                    }
                }
                const uint32_t idx = it - above;
                int want = (int)(idx / Hkv);  // the want-th sequence with more than lo tiles
                w.h = (int)(idx - want * Hkv);
                int r = 0;
#pragma unroll 1
                for (int r0 = 0; r0 < R; r0 += 32) {
                    const unsigned has = __ballot_sync(0xffffffffu, r0 + lane < R && tiles_of(r0 + lane) > lo);
                    const int c = __popc(has);
                    if (want < c) {  // the lane with want set bits below its own
                        const unsigned at = __ballot_sync(
                            0xffffffffu, (has >> lane & 1) && __popc(has & ((1u << lane) - 1)) == want);
                        r = r0 + __ffs(at) - 1;
                        break;
                    }
                    want -= c;
                }
                w.valid = 1;
                w.q0 = __ldg(a.qsl + r);
                w.n = __ldg(a.qsl + r + 1) - w.q0;
                w.i0 = lo * a.item_tokens;
                w.guard = kNoGuard;
                if (kSplit) {
                    const int all = (min(w.n, w.i0 + a.tile_tokens) + kKeys - 1) / kKeys;
                    w.n_keys[0] = (all + 1) / 2;
                    w.n_keys[1] = all / 2;
                } else {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int last = min(w.n, w.i0 + (t + 1) * a.tile_tokens);  // past the tile's last token
                        w.n_keys[t] = last > w.i0 + t * a.tile_tokens ? (last + kKeys - 1) / kKeys : 0;
                    }
                }
            }
            return w;
        };
        Item w{}, ahead{};
        uint32_t asked = 0;   // blocks asked for
        bool again = false;
        auto ask = [&]() {
            if (lane == 0) {
                mbar_arrive_expect_tx(bar + Bars::kBlock, 16);
                block_request(smem + M::kOffBlock, bar + Bars::kBlock);
            }
            ++asked;
        };
        auto answer = [&](uint32_t &index) {
            if (!warp_wait(bar + Bars::kBlock, (asked - 1) & 1, abort)) return false;
            index = block_answer(smem + M::kOffBlock);
            fence_proxy_async_smem();  // read before the next answer is written
            __syncwarp();
            return true;
        };
#pragma unroll 1
        for (int k = -1; ok; ++k) {
            // Q_A, K(0), Q_B, V(0), K(1), V(1), ... of item k, by one lane (split:
            // one Q; K(0), K(1), V(0), K(2), V(1), ..., as the products take
            // them); the next item is looked up once the ring is full.
            const int tiles = item_tiles<kSplit>(w), all = 2 * tiles;
            int i = 0;
            if (k >= 0 && !again) ask();
#pragma unroll 1
            for (int round = 0; round < 2 && ok; ++round) {
                const int stop = round ? all : min(all, kStages);
                if (lane == 0) {
#pragma unroll 1
                    for (; i < stop; ++i, ++x) {
                        if (i < (kSplit ? 1 : 2) && w.n_keys[i]) {
                            if (!lane_wait(&q_empty[i], ((q_used >> i) & 1) ^ 1, abort)) { ok = false; break; }
                            q_used ^= 1u << i;
                            q_any |= 1u << i;
                            mbar_arrive_expect_tx(&q_full[i], a.tile_tokens * a.group * D * 2);
#pragma unroll
                            for (int b = 0; b < D / 64; ++b)
                                tma_load_3d(smem + M::kOffQ + i * M::kTile + b * M::kHalf, &q_map, b * 64,
                                            w.h * a.group, w.q0 + w.i0 + i * a.tile_tokens, &q_full[i]);
                        }
                        int j = i >> 1;
                        bool is_v = i & 1;
                        if (kSplit) {
                            const int f = i - 2;  // behind K(0), K(1)
                            is_v = i > 0 && (f < 0 ? tiles == 1 : !(f & 1) || f >= 2 * (tiles - 2));
                            j = f < 0 ? (is_v ? 0 : i) : f >= 2 * (tiles - 2) ? f - (tiles - 2) : is_v ? f >> 1 : (f >> 1) + 2;
                        }
                        const int st = x % kStages;
                        if (!lane_wait(&kv_empty[st], ((x / kStages) & 1) ^ 1, abort)) { ok = false; break; }
                        // A guarded V tile is told to the guard, which tells the
                        // MMA warp; its turn at kv_full passes at once.
                        uint64_t *full = &kv_full[st];
                        if (is_v && j >= w.guard) {
                            mbar_arrive(full);
                            full = &v_guard[st];
                            g_used ^= 1u << st;
                            g_any |= 1u << st;
                        }
                        mbar_arrive_expect_tx(full, kKeys * D * 2);
                        tma_load_4d(smem + M::kOffKv + st * M::kTile, is_v ? &v_map : &k_map, 0, w.q0 + j * kKeys, 0,
                                    w.h, full);
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (ok && round == 0 && !again) {
                    uint32_t index = blockIdx.x;
                    if (k >= 0) {
                        ok = answer(index);
                        // past the last item: blocks that have nothing to do
                        while (ok && index != ~0u && index >= total) {
                            ask();
                            ok = answer(index);
                        }
                    }
                    ahead = find(ok ? index : ~0u);
                }
            }
            if (!ok) break;
            // The item that had the next slot is through, output and all: it,
            // or a new one, comes next. With nothing new the other slots' items
            // may still have to be done again.
            int slot = 0;
            again = false;
            for (int e = 1; e <= kSlots && !again && (e == 1 || !ahead.valid); ++e) {
                slot = (k + e) % kSlots;
                ok = warp_wait(&d_empty[slot], (((k + e) / kSlots) & 1) ^ 1, abort);
                if (!ok) break;
                again = redo[slot];
            }
            if (!ok) break;
            w = again ? guarded(items[slot]) : ahead;
            __syncwarp();
            if (lane == 0) {
                redo[slot] = 0;
                items[(k + 1) % kSlots] = w;
                mbar_arrive(&d_full[(k + 1) % kSlots]);
            }
            __syncwarp();
            if (!w.valid) break;
        }
        if (!ok && lane == 0) {
            // let copies already issued land before the CTA can leave
            if (asked) mbar_drain(bar + Bars::kBlock, (asked - 1) & 1, status, nullptr, 0);
            for (uint32_t y = x > (uint32_t)kStages ? x - kStages : 0; y < x; ++y)
                mbar_drain(&kv_full[y % kStages], (y / kStages) & 1, status, nullptr, 0);
            for (int t = 0; t < 2; ++t)
                if (q_any >> t & 1) mbar_drain(&q_full[t], ((q_used >> t) & 1) ^ 1, status, nullptr, 0);
            for (int v = 0; v < kStages; ++v)
                if (g_any >> v & 1) mbar_drain(&v_guard[v], ((g_used >> v) & 1) ^ 1, status, nullptr, 0);
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------- MMA issue ----------------------------
        setmaxnreg_dec<kOtherRegs>();
        constexpr uint32_t kIdS = umma_idesc_bf16(kRows, kKeys, 0, 0);
        constexpr uint32_t kIdPV = umma_idesc_bf16(kRows, D, 0, 1);
        const uint32_t tmu = uniform(tm);
        const uint32_t q_lo = desc_lo(smem_u32(smem + M::kOffQ), 16);
        const uint32_t k_lo = desc_lo(smem_u32(smem + M::kOffKv), 16);          // as K: K-major
        const uint32_t v_lo = desc_lo(smem_u32(smem + M::kOffKv), M::kHalf);    // as V: MN-major
        const uint32_t bars = smem_u32(bar);
        auto at = [&](int i) { return bars + 8 * i; };
        auto wait = [&](uint32_t b, uint32_t parity) { return warp_wait(b, parity, abort); };
        auto kv_wait = [&](uint32_t y) { return wait(at(Bars::kKvFull + y % kStages), (y / kStages) & 1); };
        auto kv_release = [&](uint32_t y) { commit(at(Bars::kKvFull + kStages + y % kStages)); };
        auto pv_part = [&](int t, int part, uint32_t y, uint32_t fresh) {
            const uint32_t b_lo = v_lo + (y % kStages) * (M::kTile >> 4);
#pragma unroll
            for (int kk = part * (kFirstKeys / 16); kk < (part ? kKeys : kFirstKeys) / 16; ++kk)
                mma_ts(tmu + kColO + t * D, tmu + col_p<D>(t) + kk * 8, b_lo + kk * (2048 >> 4), kIdPV,
                       kk > 0 ? 1u : 1u - fresh);
        };
        // S of a last tile: the keys used, in thirty-twos as the softmax reads
        // them (ragged prompts 58.5 -> 57.6 us; with D = 64 a narrower product is
        // no shorter, and one of P that leaves out keys costs more than it saves).
        constexpr bool kNarrow = D == 128;
        auto id_keys = [&](int sixteens) { return kIdS - ((uint32_t)(8 - (sixteens + 1) / 2 * 2) << 18); };
        auto s_product = [&](int t, uint32_t y, uint32_t ids) {
            const uint32_t a_lo = q_lo + (kSplit ? 0 : t) * (M::kTile >> 4), b_lo = k_lo + (y % kStages) * (M::kTile >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                mma_ss(tmu + t * kKeys, a_lo + (kk / 4) * (M::kHalf >> 4) + (kk % 4) * 2,
                       b_lo + (kk / 4) * (M::kHalf >> 4) + (kk % 4) * 2, ids, kk > 0 ? 1u : 0u);
        };
        // What S_t's columns have to wait for before a new S: with P in them its
        // product, else only the softmax's reading.
        constexpr int kSFree = kOwnP<D> ? Bars::kSTaken : Bars::kPvDone;
        uint32_t x = 0;                   // K and V tiles of the items so far
        uint32_t pv0 = 0, pv1 = 0;        // PV products issued for A, B
        uint32_t q_used = 0, o_used = 0;  // parity bits by query tile: Q tiles taken, outputs written
        uint32_t v_used = 0;              // by stage: guarded V tiles
        auto v_wait = [&](uint32_t y, bool guarded) {
            if (!guarded) return kv_wait(y);
            const uint32_t st = y % kStages;
            const bool there = wait(at(Bars::kKvFull + 2 * kStages + st), (v_used >> st) & 1);
            v_used ^= 1u << st;
            return there;
        };
        bool ok = true;
        int have = -1, next_a = 0, next_b = 0, next_guard = 0;  // the item read last
        int next_ka = 0, next_kb = 0;  // keys that its last tiles are used with, in sixteens
        auto read = [&](int k) {
            const Item w = items[k % kSlots];
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[k % kSlots]);
            next_a = uniform(w.n_keys[0]);  // none: the end
            next_b = uniform(w.n_keys[1]);
            next_guard = uniform(w.guard);
            const int end_a = min(w.n, w.i0 + a.tile_tokens), end_b = min(w.n, w.i0 + 2 * a.tile_tokens);
            next_ka = uniform((end_a - (w.n_keys[0] - 1) * kKeys + 15) / 16);
            next_kb = uniform((end_b - (w.n_keys[1] - 1) * kKeys + 15) / 16);
            have = k;
        };
        for (int k = 0; ok; ++k) {
            if (have < k) {
                if (!wait(at(Bars::kDFull + k % kSlots), (k / kSlots) & 1)) { ok = false; break; }
                read(k);
            }
            const int nA = next_a, nB = next_b, nt = max(nA, nB), guard = next_guard, kA = next_ka, kB = next_kb;  // split: A has no fewer
            if (nt == 0) break;
            if (kSplit) {
                // The same steps, where A has the even key tiles and B the odd
                // ones of one query tile: every K and V is taken by one product.
                const int tiles = nA + nB;
                uint32_t y = x;
                ok = wait(at(Bars::kQFull), q_used & 1);
                q_used ^= 1;
                auto s_tile = [&](int t, uint32_t at_y, int tile) {
                    const uint32_t done = t ? pv1 : pv0;
                    if (!kv_wait(at_y)) return false;
                    if (kOwnP<D> && tile >= 2) {
                        if (!wait(at(kSFree + t), done & 1)) return false;
                    } else if (done > 0 && !wait(at(kSFree + t), (done - 1) & 1)) {
                        return false;
                    }
                    tmem_fence_after_sync();
                    s_product(t, at_y, kIdS);
                    commit(at(Bars::kSFull + t));
                    kv_release(at_y);
                    if (tile + 1 == tiles) commit(at(Bars::kQEmpty));
                    return true;
                };
                if (ok) ok = s_tile(0, y++, 0);
                if (ok && nB) ok = s_tile(1, y++, 1);
#pragma unroll 1
                for (int j = 0; j < nA && ok; ++j) {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int n_t = t ? nB : nA, tile = 2 * j + t;
                        if (j >= n_t) continue;
                        const uint32_t par = (t ? pv1 : pv0) & 1, yv = y++;
                        if (kOwnP<D> && j + 1 < n_t && !s_tile(t, y++, tile + 2)) { ok = false; break; }
                        if (j == 0) {  // the previous item's O has been read
                            if (!wait(at(Bars::kOFree + t), ((o_used >> t) & 1) ^ 1)) { ok = false; break; }
                            o_used ^= 1u << t;
                            if (t == 0 && is_done(at(Bars::kDFull + (k + 1) % kSlots), ((k + 1) / kSlots) & 1)) read(k + 1);
                        }
                        if (!v_wait(yv, tile >= guard) || !wait(at(Bars::kPFull + 2 * t), par)) { ok = false; break; }
                        tmem_fence_after_sync();
                        pv_part(t, 0, yv, j == 0);
                        if (!wait(at(Bars::kPFull + 2 * t + 1), par)) { ok = false; break; }
                        tmem_fence_after_sync();
                        pv_part(t, 1, yv, 0);
                        commit(at(Bars::kPvDone + t));
                        if (t) ++pv1; else ++pv0;
                        kv_release(yv);
                        if (j + 1 == n_t) commit(at(Bars::kOFull + t));
                        if (!kOwnP<D> && j + 1 < n_t && !s_tile(t, y++, tile + 2)) { ok = false; break; }
                    }
                }
                if (!ok) break;
                x = y;
                continue;
            }
            // S_A(0), S_B(0); then step j: O_t += P_t(j) V(j) and S_t(j + 1),
            // for A, then for B. A sees no more key tiles than B, unless B is
            // empty. What can be asked for ahead (the next tiles) is, while
            // the tensor core is at a product.
            if (!kv_wait(x)) { ok = false; break; }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int n_t = t ? nB : nA;
                const uint32_t done = t ? pv1 : pv0;
                if (n_t == 0) continue;
                ok = wait(at(Bars::kQFull + t), (q_used >> t) & 1);
                q_used ^= 1u << t;
                if (ok && done > 0) ok = wait(at(kSFree + t), (done - 1) & 1);
                if (!ok) break;
                tmem_fence_after_sync();
                s_product(t, x, kNarrow && n_t == 1 ? id_keys(t ? kB : kA) : kIdS);
                commit(at(Bars::kSFull + t));
                if (n_t == 1) commit(at(Bars::kQEmpty + t));
            }
            if (!ok) break;
            kv_release(x);
#pragma unroll 1
            for (int j = 0; j < nt; ++j) {
                const uint32_t yv = x + 2 * j + 1, yk = yv + 1;  // V(j), K(j + 1)
                ok = v_wait(yv, j >= guard);
                if (!ok) break;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int n_t = t ? nB : nA;
                    if (j >= n_t) continue;
                    const uint32_t par = (t ? pv1 : pv0) & 1;
                    auto next_s = [&]() {
                        if ((t == 0 || j + 1 >= nA) && !kv_wait(yk)) return false;
                        if (!wait(at(kSFree + t), par)) return false;
                        tmem_fence_after_sync();
                        s_product(t, yk, kNarrow && j + 2 == n_t ? id_keys(t ? kB : kA) : kIdS);
                        commit(at(Bars::kSFull + t));
                        if (t == 1 || j + 1 >= nB) kv_release(yk);
                        if (j + 2 == n_t) commit(at(Bars::kQEmpty + t));
                        return true;
                    };
                    if (kOwnP<D> && j + 1 < n_t && !next_s()) { ok = false; break; }
                    if (j == 0) {  // the previous item's O has been read
                        if (!wait(at(Bars::kOFree + t), ((o_used >> t) & 1) ^ 1)) { ok = false; break; }
                        o_used ^= 1u << t;
                        if (t == 0 && is_done(at(Bars::kDFull + (k + 1) % kSlots), ((k + 1) / kSlots) & 1)) read(k + 1);
                    }
                    if (!wait(at(Bars::kPFull + 2 * t), par)) { ok = false; break; }
                    tmem_fence_after_sync();
                    pv_part(t, 0, yv, j == 0);
                    if (!wait(at(Bars::kPFull + 2 * t + 1), par)) { ok = false; break; }
                    tmem_fence_after_sync();
                    pv_part(t, 1, yv, 0);
                    commit(at(Bars::kPvDone + t));
                    if (t) ++pv1; else ++pv0;
                    if (t == 1 || j >= nB) kv_release(yv);
                    if (j + 1 == n_t) commit(at(Bars::kOFull + t));
                    if (!kOwnP<D> && j + 1 < n_t && !next_s()) { ok = false; break; }
                }
                if (!ok) break;
            }
            if (!ok) break;
            x += 2 * nt;
        }
        // no MMA may still be writing TMEM when it is freed
        umma_commit_warp(drain);
        if (lane == 0) mbar_drain(drain, 0, status, nullptr, 0);
        __syncwarp();
    } else if (warp >= kSoftmaxWarp && warp < kOutWarp) {
        // ----------------------------- softmax -----------------------------
        setmaxnreg_inc<kSoftmaxRegs>();
        const int t = (warp - kSoftmaxWarp) >> 2;  // query tile A or B
        const int row = (warp & 3) * 32 + lane;   // its row = TMEM lane
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_col = tm + lane_off + t * kKeys, o_col = tm + lane_off + kColO + t * D;
        const uint32_t p_col = tm + lane_off + col_p<D>(t);
        const int g = a.group;
        const int row_token = row / g;
        const bool row_used = row < a.tile_tokens * g;
        uint32_t n = 0, n_out = 0;  // key tiles and items this query tile has been through
        for (int k = 0;; ++k) {
            if (!warp_wait(&d_full[k % kSlots], (k / kSlots) & 1, abort)) break;
            const Item w = items[k % kSlots];
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[k % kSlots]);
            if (!w.valid) break;
            const int n_t = w.n_keys[t];
            if (n_t == 0) continue;
            const int i0 = w.i0 + (kSplit ? 0 : t * a.tile_tokens);
            const int i = i0 + row_token;
            const bool valid = row_used && i < w.n;
            // Rows past the tile's tokens hold other tokens or nothing; what
            // they compute is dropped.
            const int limit = valid ? i : min(w.n, i0 + a.tile_tokens) - 1;
            const int first_limit = __reduce_min_sync(0xffffffffu, limit);
            const int last_limit = __reduce_max_sync(0xffffffffu, limit);
            // Masked tiles in pieces, twice over S; not where the softmax is
            // what bounds all (two query tiles of D = 64: 67.9 against 69.4 us).
            constexpr bool kPieces = D == 128 || kSplit;
            // The row's reference, as a score and scaled, its scale, its sum of
            // p. Products with the scale are rounded by themselves: p, alpha and
            // the join of split rows have to mean the same reference.
            float m_score = 0.f, m = 0.f, sc = 0.f, l = 0.f;
            auto scaled = [&](float score) { return __fmul_rn(score, sc); };
            auto refer = [&](float score) {
                m_score = score;
                sc = row_scale(a.scale * kLog2e, score);
                m = scaled(score);
            };
            bool ok = true;
            auto scale_o = [&](float alpha) {
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                    float o[16];
                    tmem_ld16(o_col + c * 16, o);
                    tmem_wait_ld_regs(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] *= alpha;
                    tmem_st16(o_col + c * 16, o);
                }
            };
            for (int j = 0; j < n_t; ++j, ++n) {
                if (!warp_wait(&s_full[t], n & 1, abort)) { ok = false; break; }
                tmem_fence_after_sync();
                auto hand_on = [&](int part) {
                    tmem_wait_st();
                    tmem_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * t + part]);
                };
                const int key0 = (kSplit ? 2 * j + t : j) * kKeys;
                const bool masked = key0 + kKeys - 1 > first_limit;
                if (kPieces && masked) {
                    // A tile with masked keys: 32 keys at a time, first for the
                    // maximum, then for p; keys that no row of the warp sees are
                    // neither read nor computed, and only pieces where the rows
                    // differ are compared key by key (prompts of 17 and 40 tokens
                    // 6.9 -> 6.6 us, ragged ones 59.4 -> 58.4).
                    const int lim = limit - key0, sure = first_limit - key0, seen = last_limit - key0;
                    float c[32], top = -INFINITY;
                    auto piece = [&](int at) {
                        tmem_ld32(s_col + at, c);
                        tmem_wait_ld_regs(c);
                        if (at + 31 > sure) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) c[e] = e <= lim - at ? c[e] : -INFINITY;
                        }
                    };
#pragma unroll 1
                    for (int at = 0; at < kKeys && at <= seen; at += 32) {
                        piece(at);
                        top = fmaxf(top, max32(c));
                    }
                    if (kOwnP<D> && n > 0) {
                        ok = warp_wait(&pv_done[t], (n - 1) & 1, abort);
                        if (!ok) break;
                        tmem_fence_after_sync();
                    }
                    if (j == 0) {
                        refer(fmaxf(top, -FLT_MAX));
                    } else if (__any_sync(0xffffffffu, scaled(top) - m > kRescaleBits)) {
                        // each row by its own scores: what the others of the warp
                        // hold (some hold nothing) must not show in its bits
                        const bool moves = scaled(top) - m > kRescaleBits;
                        const float alpha = moves ? fast_exp2(m - scaled(top)) : 1.f;
                        if (moves) refer(top);
                        l *= alpha;
                        scale_o(alpha);
                    }
                    float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                    for (int at = 0; at < kKeys; at += 32) {
                        uint32_t q[16];
                        if (at <= seen) {
                            piece(at);
                            exps(c, sc, m, part, q);
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e) q[e] = 0;
                        }
                        if (kOwnP<D> && at == kKeys - 32) {
                            tmem_fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&s_taken[t]);
                        }
                        tmem_st16u(p_col + at / 2, q);
                        if (at + 32 >= kFirstKeys) hand_on(at + 32 > kFirstKeys);
                    }
                    l += (part[0].x + part[0].y) + (part[1].x + part[1].y);
                    continue;
                }
                float s[4][32];
                uint32_t p[kFirstKeys / 2];
                float sum;
                // P against a reference that need not be the maximum: with all p
                // below 2^kRescaleBits nothing overflows, and the common factor
                // falls out of O / l. So after a row's first tile, whose maximum
                // sets the reference, the maximum is not taken: where the sum of
                // the first keys' p or the largest of the last keys' scores is
                // past the bound (rare), the reference moves up to the maximum,
                // O follows, and the tile is done again; S is still there.
                bool moves = j == 0;
                while (true) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(s_col + c * 32, s[c]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_wait_ld_regs(s[c]);
                    if (!kPieces && masked) {
                        const int lim = limit - key0, sure = first_limit - key0;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            if (c * 32 + 31 <= sure) continue;
#pragma unroll
                            for (int e = 0; e < 32; ++e) s[c][e] = c * 32 + e <= lim ? s[c][e] : -INFINITY;
                        }
                    }
                    float alpha = 1.f;
                    const bool any = __any_sync(0xffffffffu, moves);
                    if (any) {
                        const float top = fmaxf(fmaxf(max32(s[0]), max32(s[1])), fmaxf(max32(s[2]), max32(s[3])));
                        if (j == 0) {
                            refer(fmaxf(top, -FLT_MAX));  // a number even where every score is minus infinity
                        } else if (moves && scaled(top) > m) {
                            alpha = fast_exp2(m - scaled(top));
                            refer(top);
                        }
                    }
                    float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int c = 0; c < kFirstKeys / 32; ++c) exps(s[c], sc, m, part, p + 16 * c);
                    const float last = fmaf(max32(s[3]), sc, -m);
                    sum = (part[0].x + part[0].y) + (part[1].x + part[1].y);
                    if (kOwnP<D> && n > 0) {  // O and P are at rest once the product before is over
                        ok = warp_wait(&pv_done[t], (n - 1) & 1, abort);
                        if (!ok) break;
                        tmem_fence_after_sync();
                    }
                    if (!any) {
                        moves = sum > kRescaleSum || last > kRescaleBits;
                        if (!__any_sync(0xffffffffu, moves)) break;
                        continue;
                    }
                    if (j == 0) break;
                    l *= alpha;
                    // (P over S: PV(j - 1) was over before S(j) was issued.)
                    scale_o(alpha);
                    break;
                }
                if (!ok) break;
                if (kOwnP<D>) {
                    tmem_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_taken[t]);
                }
                store_p(p_col, p);
                hand_on(0);
                keep(s[3]);  // its exponentials not ahead of the first part's hand-over
                {
                    float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    uint32_t q[16];
                    exps(s[3], sc, m, part, q);
                    tmem_st16u(p_col + kFirstKeys / 2, q);
                    hand_on(1);
                    l += sum + ((part[0].x + part[0].y) + (part[1].x + part[1].y));
                }
            }
            if (!ok || !warp_wait(&o_free[t], (n_out & 1) ^ 1, abort)) break;
            ++n_out;
            row_sum[t * kRows + row] = l;
            if (kSplit) row_ref[t * kRows + row] = m_score;
            __syncwarp();
            if (lane == 0) mbar_arrive(&l_full[t]);
        }
    } else if (warp >= kOutWarp) {
        // ------------------------------ output ------------------------------
        setmaxnreg_dec<kOtherRegs>();
        // O / l to memory while the softmax and the tensor core are at the
        // next item; O is theirs again once it has been read.
        const int row = (warp & 3) * 32 + lane;
        const uint32_t o_col = tm + ((uint32_t)((warp & 3) * 32) << 16) + kColO;
        const int g = a.group;
        const int row_token = row / g, row_head = row % g;
        const bool row_used = row < a.tile_tokens * g;
        uint32_t used = 0;  // parity bits of the outputs so far
        bool ok = true;
        for (int k = 0; ok; ++k) {
            if (!warp_wait(&d_full[k % kSlots], (k / kSlots) & 1, abort)) break;
            const Item w = items[k % kSlots];
            if (!w.valid) break;
            if (!warp_wait(&bad_full[k % kSlots], (k / kSlots) & 1, abort)) break;
            const uint32_t *bad = bad_keys + (k % kSlots) * kGuardTiles * (kKeys / 32);
            __nv_bfloat162 odd = __floats2bfloat162_rn(0.f, 0.f);  // NaN once an output of a valid row is not finite
            const bool any_bad = __any_sync(0xffffffffu, lane < kGuardTiles * (kKeys / 32) && bad[lane]);
            if (kSplit) {
                // One row from two: out = sum_t O_t 2^(m_t - m) / sum_t l_t 2^(m_t - m).
                for (int t = 0; t < 2 && ok; ++t) {
                    if (!w.n_keys[t]) continue;
                    const uint32_t par = (used >> t) & 1;
                    used ^= 1u << t;
                    ok = warp_wait(&l_full[t], par, abort) && warp_wait(&o_full[t], par, abort);
                }
                if (!ok) break;
                tmem_fence_after_sync();
                const bool both = w.n_keys[1] > 0;
                const int i = w.i0 + row / g;
                const bool valid = row < a.tile_tokens * g && i < w.n;
                const float ref0 = row_ref[row], ref1 = both ? row_ref[kRows + row] : ref0;
                const float sc = row_scale(a.scale * kLog2e, fmaxf(fabsf(ref0), fabsf(ref1)));
                const float m0 = __fmul_rn(ref0, sc), m1 = __fmul_rn(ref1, sc), m = fmaxf(m0, m1);
                float f0 = fast_exp2(m0 - m), f1 = both ? fast_exp2(m1 - m) : 0.f;
                const float inv = 1.f / (row_sum[row] * f0 + (both ? row_sum[kRows + row] * f1 : 0.f));
                f0 *= inv;
                f1 *= inv;
                const int head = w.h * g + row % g;
                __nv_bfloat16 *dst = a.out + (((long long)w.q0 + i) * a.num_q_heads + head) * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tmem_ld32(o_col + c, o);
                    tmem_wait_ld_regs(o);
                    if (both) {
#pragma unroll
                        for (int e = 0; e < 32; e += 16) {
                            float q[16];
                            tmem_ld16(o_col + D + c + e, q);
                            tmem_wait_ld_regs(q);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[e + i] = fmaf(q[i], f1, o[e + i] * f0);
                        }
                    }
                    put_row(a.wide_out, valid, c, both ? 1.f : f0, o, odd, dst);
                }
                if (any_bad && valid) add_bad<D>(a, w, bad, i, dst);
                tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&o_free[0]);
                    if (both) mbar_arrive(&o_free[1]);
                }
            }
#pragma unroll 1
            for (int t = 0; t < 2 && !kSplit; ++t) {
                if (!w.n_keys[t]) continue;
                const uint32_t par = (used >> t) & 1;
                used ^= 1u << t;
                ok = warp_wait(&l_full[t], par, abort) && warp_wait(&o_full[t], par, abort);
                if (!ok) break;
                tmem_fence_after_sync();
                const int i = w.i0 + t * a.tile_tokens + row_token;
                const bool valid = row_used && i < w.n;
                const float inv = rcp(row_sum[t * kRows + row]);
                const int head = w.h * g + row_head;
                __nv_bfloat16 *dst = a.out + (((long long)w.q0 + i) * a.num_q_heads + head) * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tmem_ld32(o_col + t * D + c, o);
                    tmem_wait_ld_regs(o);
                    put_row(a.wide_out, valid, c, inv, o, odd, dst);
                }
                if (any_bad && valid) add_bad<D>(a, w, bad, i, dst);
                tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_free[t]);
            }
            const float2 sum = __bfloat1622float2(odd);
            if (__any_sync(0xffffffffu, sum.x != 0.f || sum.y != 0.f) && w.guard == kNoGuard && lane == 0)
                redo[k % kSlots] = 1;
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[k % kSlots]);
        }
    } else {
        // --------------------------- guard of V ---------------------------
        // The tensor core multiplies masked values by a probability of 0,
        // which leaves nothing of them unless they are infinite or NaN. Where
        // an item's output is not finite, the item is done again with its
        // last key tiles, the only ones with masked keys, looked over first:
        // rows past the sequence are cleared, other values that are not finite
        // too, and those keys noted; the output warps add them to the rows
        // that see them. (Looking over every item's tiles cost 3 to 5 %.)
        setmaxnreg_dec<kOtherRegs>();
        const int row0 = (warp - kGuardWarp) * (kKeys / 2);  // each warp has half of a tile's keys
        uint32_t x = 0, g_used = 0;  // g_used: parity bits of guarded tiles by V slot
        bool ok = true;
        for (int k = 0; ok; ++k) {
            if (!warp_wait(&d_full[k % kSlots], (k / kSlots) & 1, abort)) break;
            const Item w = items[k % kSlots];
            if (!w.valid) break;
            const int nt = item_tiles<kSplit>(w);
            uint32_t *bad = bad_keys + (k % kSlots) * kGuardTiles * (kKeys / 32);
            if (lane < 2 * kGuardTiles) bad[lane / 2 * (kKeys / 32) + row0 / 32 + lane % 2] = 0;
            __syncwarp();
            for (int j = w.guard; j < nt; ++j) {
                const uint32_t y = x + (kSplit ? min(2 * j + 2, 2 * nt - 1) : 2 * j + 1), v = y % kStages;  // V(j)
                if (!warp_wait(&v_guard[v], (g_used >> v) & 1, abort)) { ok = false; break; }
                g_used ^= 1u << v;
                uint4 *vt = reinterpret_cast<uint4 *>(smem + M::kOffKv + (y % kStages) * M::kTile);
                const int rows = min(kKeys, w.n - j * kKeys);
                // A value times 0 is NaN unless it is finite: one packed
                // multiply-add for two values, over this warp's half tile.
                __nv_bfloat162 odd = __floats2bfloat162_rn(0.f, 0.f);
                const __nv_bfloat162 zero = odd;
#pragma unroll 1
                for (int b = 0; b < D / 64; ++b) {
                    const uint4 *half = vt + (b * kKeys + row0) * 8 + lane;
#pragma unroll 2
                    for (int c = 0; c < kKeys / 2 * 8 / 32; ++c) {
                        const uint4 v = half[c * 32];
                        odd = __hfma2(pair_of(v.x), zero, odd);
                        odd = __hfma2(pair_of(v.y), zero, odd);
                        odd = __hfma2(pair_of(v.z), zero, odd);
                        odd = __hfma2(pair_of(v.w), zero, odd);
                    }
                }
                const float2 found = __bfloat1622float2(odd);
                if (__any_sync(0xffffffffu, found.x != 0.f || found.y != 0.f) || row0 + kKeys / 2 > rows) {
#pragma unroll 1
                    for (int b = 0; b < D / 64; ++b) {
                        uint4 *half = vt + (b * kKeys + row0) * 8;
#pragma unroll 1
                        for (int c = lane; c < kKeys / 2 * 8; c += 32) {  // the swizzle keeps a row's chunks in the row
                            const int r = row0 + c / 8;
                            const uint4 v = half[c];
                            if (r >= rows) {
                                half[c] = make_uint4(0, 0, 0, 0);
                            } else if (odd_pair(v.x) || odd_pair(v.y) || odd_pair(v.z) || odd_pair(v.w)) {
                                half[c] = make_uint4(clean_pair(v.x), clean_pair(v.y), clean_pair(v.z), clean_pair(v.w));
                                atomicOr(&bad[(j - w.guard) * (kKeys / 32) + r / 32], 1u << (r % 32));
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_safe[v]);
            }
            x += 2 * nt;
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bad_full[k % kSlots]);
                mbar_arrive(&d_empty[k % kSlots]);
            }
        }
    }

    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    if (warp == kMmaWarp) tmem_dealloc(tm, kTmemCols);
    if (threadIdx.x == 0 && s_abort) raise_status(status, PKV_DEV_TIMEOUT);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

std::mutex g_mu;
int g_sms[64];  // by device: its SMs, once the kernels' attributes are set
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

int prompt_setup(int *sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_E_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    *sms = g_sms[dev];
    if (*sms) return PKV_OK;
    const cudaFuncAttribute smem = cudaFuncAttributeMaxDynamicSharedMemorySize;
    if (cudaFuncSetAttribute(prompt_kernel<64, false>, smem, Smem<64>::kAlloc) != cudaSuccess ||
        cudaFuncSetAttribute(prompt_kernel<64, true>, smem, Smem<64>::kAlloc) != cudaSuccess ||
        cudaFuncSetAttribute(prompt_kernel<128, false>, smem, Smem<128>::kAlloc) != cudaSuccess ||
        cudaFuncSetAttribute(prompt_kernel<128, true>, smem, Smem<128>::kAlloc) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return PKV_E_CUDA;
    if (!g_encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess || !fn)
            return PKV_E_CUDA;
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    g_sms[dev] = *sms;
    return PKV_OK;
}

int encode(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
           const cuuint32_t *box) {
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, ones,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? PKV_OK
               : PKV_E_CUDA;
}

// k or v as {64 columns, token, 64-column half, head}: one box is 128 tokens
// of one head, landing as [D / 64][128 rows][128 B].
int encode_kv(CUtensorMap *map, const void *base, int tokens, long long stride, int heads, int D) {
    const cuuint64_t dims[4] = {64, (cuuint64_t)tokens, (cuuint64_t)D / 64, (cuuint64_t)heads};
    const cuuint64_t strides[3] = {(cuuint64_t)stride * 2, 128, (cuuint64_t)D * 2};
    const cuuint32_t box[4] = {64, kKeys, (cuuint32_t)D / 64, 1};
    return encode(map, base, 4, dims, strides, box);
}

// q as {columns, head, token}: a box is a tile's tokens x the group's heads
// x 64 columns.
int encode_q(CUtensorMap *map, const void *base, int tokens, long long stride, int heads, int D, int group) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)(kRows / group)};
    return encode(map, base, 3, dims, strides, box);
}

bool stride_ok(long long stride, long long width) {
    return stride % 8 == 0 && stride >= width && stride < (1LL << 38);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" PKV_API int pkv_prompt_attention(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                            const void *v, int64_t v_stride, int32_t num_tokens, int32_t num_q_heads,
                                            int32_t num_kv_heads, int32_t head_size, const int32_t *query_start_loc,
                                            int32_t num_reqs, float scale, void *out, int32_t *status, void *stream) {
    if (head_size != 64 && head_size != 128) return PKV_E_HEAD_SIZE;
    if (num_tokens < 0 || num_reqs < 0 || num_kv_heads <= 0 || num_kv_heads > 4096) return PKV_E_DIMS;
    if (num_tokens > INT32_MAX - 65536 || (long long)num_reqs * num_kv_heads > INT32_MAX - 65536) return PKV_E_DIMS;
    if (num_q_heads <= 0 || num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > kRows) return PKV_E_GQA;
    if (!(scale > 0.f) || scale > 1e30f) return PKV_E_DIMS;
    if (num_tokens == 0 || num_reqs == 0) return PKV_OK;
    if (!q || !k || !v || !query_start_loc || !out) return PKV_E_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(query_start_loc, 4) ||
        !aligned(status, 4))
        return PKV_E_ALIGN;
    const long long wq = (long long)num_q_heads * head_size, wkv = (long long)num_kv_heads * head_size;
    if (!stride_ok(q_stride, wq) || !stride_ok(k_stride, wkv) || !stride_ok(v_stride, wkv)) return PKV_E_DIMS;
    // a row that is done again reads its inputs again
    if (out == q || out == k || out == v) return PKV_E_DIMS;
    int sms = 0;
    int rc = prompt_setup(&sms);
    if (rc) return rc;
    PromptArgs a{};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.qsl = query_start_loc;
    a.num_tokens = num_tokens;
    a.num_reqs = num_reqs;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.group = num_q_heads / num_kv_heads;
    a.tile_tokens = kRows / a.group;
    a.scale = scale;
    a.wide_out = aligned(out, 32);
    a.status = status;
    CUtensorMap q_map, k_map, v_map;
    rc = encode_q(&q_map, q, num_tokens, q_stride, num_q_heads, head_size, a.group);
    if (!rc) rc = encode_kv(&k_map, k, num_tokens, k_stride, num_kv_heads, head_size);
    if (!rc) rc = encode_kv(&v_map, v, num_tokens, v_stride, num_kv_heads, head_size);
    if (rc) return rc;
    // A block for every item there may be (every sequence rounds up to whole
    // items); those that start fetch the others' items.
    auto items = [&](int tokens) { return ((long long)num_tokens / tokens + num_reqs) * num_kv_heads; };
    // While items of two query tiles leave SMs idle, items of one, its keys split
    // between A and B: half the steps, and twice the SMs (one prompt of 512
    // tokens, 72 such items at most: 14.0 -> 11.5 us; 2048 tokens of 12/4 heads,
    // 100: 30.5 -> 25.4). Beyond, K and V copied twice and twice the items cost
    // more (4 x 300 tokens, 176: 14.1 -> 17.1 us; a ragged batch of 24: 64.6 -> 86.9).
    const bool split = items(2 * a.tile_tokens) <= sms;
    a.item_tokens = split ? a.tile_tokens : 2 * a.tile_tokens;
    const long long grid = items(a.item_tokens);
    if (grid > INT32_MAX) return PKV_E_DIMS;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto kernel = head_size == 128 ? (split ? prompt_kernel<128, true> : prompt_kernel<128, false>)
                                   : (split ? prompt_kernel<64, true> : prompt_kernel<64, false>);
    const cudaError_t err = launch_pdl(kernel, dim3((unsigned)grid), dim3(kThreads),
                                       head_size == 128 ? Smem<128>::kAlloc : Smem<64>::kAlloc, st, q_map, k_map, v_map, a);
    return err == cudaSuccess ? PKV_OK : PKV_E_CUDA;
}
