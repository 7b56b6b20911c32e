// Attention over the 4-bit pool on tcgen05 tensor cores, for requests that bring
// many rows in one step (chunks of a prompt).
//
// An item is 128 rows (tokens x the q heads of one kv head, token-major) of one
// request over all keys that they see, in tiles of 128. Per key tile:
//     S = Q K^T    M 128, N 128: q and K as fp16 in shared memory, S in TMEM;
//     P = 2^(mul (s - m)), fp16, over S in TMEM;
//     O += P V     M 128, N D: P from TMEM, V as fp16 in shared memory.
// Eight warps do all of it: each turns one block of 16 keys of the tile from codes
// to fp16 (exactly), and takes 64 keys of 32 rows through the softmax. While S is
// being multiplied V is unpacked, while P V is, the next tile's K; codes are read a
// tile ahead, straight into registers. What is left of the chain S - softmax - P V
// is filled by a second CTA on the same SM (100 KB of shared memory, 256 columns of
// TMEM and 128 registers a thread each). Items are claimed one by one from a counter
// in the workspace, those of the longest contexts first, so that what runs last is
// short (158 us against 188 for what follows). In batches of more than 256 requests,
// decode rows counted, they go in the batch's order: with the longest request last and
// requests of one key around them the ones below take 164 us among 256 requests and 185
// among 257. Where they are too few for the CTAs, an
// item's keys are split (kv4_plan.h), and the last CTA to arrive adds its parts up, in
// order, from fp32 O, m and l in the workspace (1 request of 512 tokens and 30000 keys
// 393 -> 275 us, 4 of 64 and 4000 60 -> 42).
//
// A row's reference m moves only when the sum of a tile's p shows that one of them
// may be past 2^12: no pass for the maximum but the first (188 against 293 us).
//
// Measured: chunks of 60 to 512 tokens of 16 requests with 600 to 4000 keys, 32 heads
// on 8 of 128: 142 us, 750 TFLOP/s of the two products, floor 54.7 (1948 TFLOP/s). The
// tensor cores are busy 35 % of the time, the issue slots 47 %: a tile and CTA take
// 1024 cycles of products, 512 of exponentials and about 570 instructions a warp (200
// of them unpacking), and four warps a scheduler, as many as registers allow, do not
// cover the waits between them. 256 rows an item, which unpack keys half as often, 17
// warps and one CTA an SM: 163 us (longer items, fewer of them).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "kv4_args.h"
#include "kv4_format.cuh"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_short_wait.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 128;
constexpr uint32_t kTmemCols = 256, kColO = 128;  // S (P over it), O

template <int D>
struct Smem {
    static constexpr int kHalf = 128 * 128;         // q, K, V: 128 rows x 64 columns
    static constexpr int kTile = (D / 64) * kHalf;
    static constexpr int kQ = 0, kK = kTile, kV = 2 * kTile;
    static constexpr int kX = 3 * kTile;         // float [2][128]: the halves' maxima, at last their sums
    static constexpr int kMul = kX + 2 * 128 * 4;
    static constexpr int kNan = kMul + 128 * 4;  // first key whose V is no number, by groups of 16 columns
    static constexpr int kBar = kNan + 8 * 4;
    static constexpr int kBytes = kBar + 3 * 8;
    static constexpr int kAlloc = kBytes + 1024;
};

constexpr uint32_t idesc_f16(int M, int N, int b_mn_major) {
    return (1u << 4) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// A value that all lanes hold, as the compiler can know it too.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_or_sync(0xffffffffu, v); }

// Products and commits by one elected lane, four MMAs at a time, with operands that
// stay in uniform registers: of a matrix descriptor (128-byte swizzle) only the low
// word changes from one to the next, with the address (and the leading offset).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups 1024 bytes apart
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t leading) { return ((addr & 0x3FFFF) >> 4) | ((leading >> 4) << 16); }
// Four steps of 16 of a product from shared memory: both operands' columns go on
// 32 bytes a step.
__device__ __forceinline__ void mma_ss4(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t.reg .b32 a, b;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "add.u32 a, %1, 2;\n\tadd.u32 b, %2, 2;\n\tmov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, 1;\n\t"
        "add.u32 a, %1, 4;\n\tadd.u32 b, %2, 4;\n\tmov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, 1;\n\t"
        "add.u32 a, %1, 6;\n\tadd.u32 b, %2, 6;\n\tmov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, 1;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}
// Four steps of a product of P, in tensor memory, and V: 8 columns and 16 rows a step.
__device__ __forceinline__ void mma_ts4(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\t.reg .b32 a, b;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t"
        "add.u32 a, %1, 8;\n\tadd.u32 b, %2, 128;\n\tmov.b64 db, {b, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, 1;\n\t"
        "add.u32 a, %1, 16;\n\tadd.u32 b, %2, 256;\n\tmov.b64 db, {b, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, 1;\n\t"
        "add.u32 a, %1, 24;\n\tadd.u32 b, %2, 384;\n\tmov.b64 db, {b, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, 1;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ uint32_t half_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ uint4 unpack8(uint32_t codes, __half2 scale) {
    return make_uint4(half_bits(__hmul2(kv4_pair<0>(codes), scale)), half_bits(__hmul2(kv4_pair<1>(codes), scale)),
                      half_bits(__hmul2(kv4_pair<2>(codes), scale)), half_bits(__hmul2(kv4_pair<3>(codes), scale)));
}

// What a lane (4 g + t) reads of a block's K or V (kv4_format.cuh).
template <int D>
struct Raw {
    static constexpr int kW = D / 32;
    uint32_t w[2][kW], scales;

    __device__ __forceinline__ void load(const uint8_t *tile, bool v, int lane) {  // tile null: zeros
        if (!tile) {
#pragma unroll
            for (int i = 0; i < kW; ++i) w[0][i] = w[1][i] = 0;
            scales = 0;
            return;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint8_t *at = tile + (v ? 8 * D : 0) + h * 4 * D + 4 * kW * lane;
            if constexpr (D == 128) {
                const uint4 x = __ldg(reinterpret_cast<const uint4 *>(at));
                w[h][0] = x.x, w[h][1] = x.y, w[h][2] = x.z, w[h][3] = x.w;
            } else {
                const uint2 x = __ldg(reinterpret_cast<const uint2 *>(at));
                w[h][0] = x.x, w[h][1] = x.y;
            }
        }
        if (v)
            scales = __ldg(reinterpret_cast<const uint32_t *>(tile + 17 * D + (D == 128 ? 4 * lane : 16 * (lane >> 3) + 4 * (lane & 3))));
        else if (D == 128)
            scales = __ldg(reinterpret_cast<const uint32_t *>(tile + 16 * D + 4 * lane));
        else
            scales = __ldg(reinterpret_cast<const uint16_t *>(tile + 16 * D + 2 * lane));
    }

    // K: tokens g and g + 8 of the block, a quarter of the columns each, to rows of
    // 128 bytes (64 columns), 16-byte chunks swizzled. D 128: lanes of the upper
    // columns take their words in another order, or two lanes would meet in a bank.
    // `to`: this lane's place (k_place); the chunk's number is XOR-ed into it.
    static __device__ __forceinline__ uint32_t k_place(int lane) {
        const int g = lane >> 2, t = lane & 3;
        return D == 128 ? (t >> 1) * Smem<D>::kHalf + g * 128 + ((((t & 1) * 4 + (t & 2)) ^ g) << 4) : g * 128 + (((2 * t) ^ g) << 4);
    }
    __device__ __forceinline__ void put_k(uint32_t to, int lane) const {
        const bool upper = lane & 2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const __half2 sc = kv4_scales(D == 128 ? scales >> (16 * h) : scales);
            const __half2 lo = __low2half2(sc), hi = __high2half2(sc);
#pragma unroll
            for (int i = 0; i < kW; ++i) {
                const uint32_t x = D == 128 && upper ? w[h][i ^ 2] : w[h][i];
                const __half2 s = D == 128 ? ((i < 2) != upper ? lo : hi) : h ? hi : lo;
                store((to + h * 1024) ^ (i << 4), unpack8(x, s));
            }
        }
    }
    // V: tokens 2 t and 2 t + 1 of each half block, an eighth of the columns. Tokens
    // at or past `end` become zero, and those whose scale is no number, which are noted.
    static __device__ __forceinline__ uint32_t v_place(int lane) {
        const int g = lane >> 2, t = lane & 3;
        return D == 128 ? (g >> 2) * Smem<D>::kHalf + 2 * t * 128 + ((((g & 3) * 2 + (g & 1)) ^ (2 * t)) << 4) : 2 * t * 128 + ((g ^ (2 * t)) << 4);
    }
    __device__ __forceinline__ void put_v(uint32_t to, int end, int key0, int *first_nan, int lane) {
        const int g = lane >> 2, t = lane & 3;
        // a byte is 0x7f or 0xff where adding 1 to its low seven bits reaches the eighth
        if (end < 16 || (((scales & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = 8 * (i >> 1) + 2 * t + (i & 1);
                const bool nan = (scales >> (8 * i) & 0x7fu) == 0x7fu;
                if (nan && tok < end) atomicMin(first_nan + (D == 128 ? g : g >> 1), key0 + tok);
                if (nan || tok >= end) scales &= ~(0xffu << (8 * i));
            }
        }
        const bool odd = g & 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const __half2 sc = kv4_scales(scales >> (16 * h));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const __half2 s = e ? __high2half2(sc) : __low2half2(sc);
                const uint32_t line = to + h * 1024 + e * 128;
                if constexpr (D == 128) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        store(line ^ ((i ^ e) << 4), unpack8(odd ? w[h][2 * e + (i ^ 1)] : w[h][2 * e + i], s));
                } else {
                    store(line ^ (e << 4), unpack8(w[h][e], s));
                }
            }
        }
    }
    static __device__ __forceinline__ void store(uint32_t at, uint4 x) {
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
    }
};

// Barrier of two warps, and whether any of their threads says so.
__device__ __forceinline__ bool pair_any(uint32_t id, bool mine) {
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %2, 0;\n\tbarrier.cta.red.or.pred p, %1, 64, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(any)
                 : "r"(id), "r"((uint32_t)mine)
                 : "memory");
    return any != 0;
}

// Half a row of an item from its parts, `step` floats apart, in order. A call: inlined it
// takes registers from the loop over keys (145 us instead of 142 where nothing is split).
template <int D>
__device__ __noinline__ void join_parts(const float *first, size_t step, int parts, float mul, float v_scale, int row, int half, __nv_bfloat16 *out) {
    float2 ml[kKv4MaxSplits];
#pragma unroll
    for (int k = 0; k < kKv4MaxSplits; ++k)
        ml[k] = k < parts ? __ldcg(reinterpret_cast<const float2 *>(first + k * step + kKv4ChunkRows * D) + row) : make_float2(-INFINITY, 0.0f);
    float to = -INFINITY, all = 0.0f;
#pragma unroll
    for (int k = 0; k < kKv4MaxSplits; ++k) to = fmaxf(to, ml[k].x);
#pragma unroll
    for (int k = 0; k < kKv4MaxSplits; ++k) {
        ml[k].x = fast_exp2((ml[k].x - to) * mul);
        all = fmaf(ml[k].x, ml[k].y, all);
    }
    const float f = __fdividef(v_scale, all);
#pragma unroll 2
    for (int c = 0; c < D / 8; ++c) {
        const float *from = first + 4 * ((size_t)(half * (D / 8) + c) * kKv4ChunkRows + row);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f), x[kKv4MaxSplits];
#pragma unroll
        for (int k = 0; k < kKv4MaxSplits; ++k)
            if (k < parts) x[k] = __ldcg(reinterpret_cast<const float4 *>(from + k * step));
#pragma unroll
        for (int k = 0; k < kKv4MaxSplits; ++k)
            if (k < parts) o = make_float4(fmaf(x[k].x, ml[k].x, o.x), fmaf(x[k].y, ml[k].x, o.y), fmaf(x[k].z, ml[k].x, o.z), fmaf(x[k].w, ml[k].x, o.w));
        reinterpret_cast<uint2 *>(out)[c] = make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, kKv4ChunkCtas) kv4_chunk_kernel(const Kv4Args a) {
    using S = Smem<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ long long s_units[kThreads / 32];
    __shared__ int s_items[kThreads], s_len[kThreads], s_order[kThreads], s_sum[kThreads / 32], s_most[kThreads / 32];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_claim, s_last;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *s_x = reinterpret_cast<float *>(smem + S::kX), *s_mul = reinterpret_cast<float *>(smem + S::kMul);
    int *s_nan = reinterpret_cast<int *>(smem + S::kNan);
    uint64_t *bar_s = reinterpret_cast<uint64_t *>(smem + S::kBar), *bar_pv = bar_s + 1, *bar_end = bar_s + 2;
    volatile int *abort = &s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (tid == 0) {
        s_abort = 0;
        mbar_init(bar_s, 1);
        mbar_init(bar_pv, 1);
        mbar_init(bar_end, 1);
        mbar_fence_init();
    }
    pdl_launch_dependents();
    pdl_wait();

    // Which requests are this kernel's, and how many items they have: `each` of them
    // a thread, in order; up to a thread each, those with the longest contexts first,
    // so that what runs last is short.
    const int each = (a.num_reqs + kThreads - 1) / kThreads;
    int items = 0, most = 0, bits = 0;  // the other kernel reports them
    long long units = 0;
    auto take = [&](int r, int *have, int *bits) {
        const Kv4Request q = kv4_request_of(a, r, kKv4ChunkRows, bits);
        *have = kv4_is_chunk(q, a.group) ? q.tiles * a.num_kv_heads : 0;
        return q;
    };
    for (int r = tid * each; r < min((tid + 1) * each, a.num_reqs); ++r) {
        int have;
        const Kv4Request q = take(r, &have, &bits);
        if (!have) continue;
        items += have;
        units += kv4_chunk_units(q, a.num_kv_heads);
        most = max(most, kv4_chunk_tiles(q.len));
    }
    s_len[tid] = items ? most : -1;
    if (__syncthreads_or(bits & PKV_DEV_BAD_QSL) && kv4_overlap<kThreads>(a, each, reinterpret_cast<long long *>(smem))) return;
    if (each == 1) {
        int place = 0;
        for (int i = 0; i < min(kThreads, a.num_reqs); ++i) place += s_len[i] > s_len[tid] || (s_len[i] == s_len[tid] && i < tid);
        if (tid < a.num_reqs) {
            s_order[place] = tid;
            s_items[place] = items;
        }
        __syncthreads();
        items = tid < a.num_reqs ? s_items[tid] : 0;
        __syncthreads();
    } else {
        s_order[tid] = tid;
    }
    int sum = items;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        const long long u = __shfl_xor_sync(0xffffffffu, units, d);
        if (lane >= d) sum += o;
        units += u;
        most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
    }
    if (lane == 31) {
        s_sum[warp] = sum;
        s_units[warp] = units;
        s_most[warp] = most;
    }
    __syncthreads();
    int total = 0;
    units = most = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) sum += s_sum[i];
        total += s_sum[i];
        units += s_units[i];
        most = max(most, s_most[i]);
    }
    s_items[tid] = sum;
    total = (int)uniform((uint32_t)total);
    // pieces: items, or as many parts of each; all of those run at once
    const Kv4Splits sp = kv4_splits(total, (int)gridDim.x / kKv4ChunkCtas);
    const int splits = (int)uniform((uint32_t)sp.count), pieces = total * splits;
    // what steers this kernel is uniform for the compiler too: see mma_ss4
    if (uniform(!kv4_use_chunks(units, most, sp) || (int)blockIdx.x >= pieces)) return;  // the items go by `total` claims and no more CTAs
    const int ctas = min((int)gridDim.x, total);
    if (warp == 0) tmem_alloc(&s_tmem, kTmemCols);
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tm = s_tmem, tmu = uniform(tm);

    constexpr uint32_t kIdS = idesc_f16(128, kKeys, 0), kIdPv = idesc_f16(128, D, 1);
    const uint32_t q_s = smem_u32(smem + S::kQ), k_s = smem_u32(smem + S::kK), v_s = smem_u32(smem + S::kV);
    const uint32_t q_lo = desc_lo(q_s, 16), k_lo = desc_lo(k_s, 16), v_lo = desc_lo(v_s, S::kHalf);
    const int part = warp >> 2, row = (warp & 3) * 32 + lane;  // this thread's keys (of 64) and row in the softmax
    const uint32_t tm_row = tm + ((uint32_t)((warp & 3) * 32) << 16);
    uint32_t phase = 0;  // of both barriers: they complete once a key tile
    const long long block_bytes = (long long)a.num_kv_heads * Kv4Tile<D>::kBytes;

    for (int piece = blockIdx.x; piece < pieces;) {
        int split = 0, item = piece;
        for (; item >= total; item -= total) ++split;
        // the item: request, tile and head
        Kv4Request q;
        int r, i, h;
        {
            int lo = 0, hi = kThreads - 1;  // the first thread with s_items > item
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (s_items[mid] > item) hi = mid; else lo = mid + 1;
            }
            int off = item - (lo ? s_items[lo - 1] : 0), have, none = 0;
            for (r = s_order[lo] * each;; ++r) {
                q = take(r, &have, &none);
                if (off < have) break;
                off -= have;
            }
            // longest tiles of a request first
            i = q.tiles - 1 - off / a.num_kv_heads;
            h = off % a.num_kv_heads;
        }
        const Kv4Tiling tl = kv4_tile(q, i, a.group, kKv4ChunkRows);
        const int nt = (int)uniform((uint32_t)kv4_chunk_tiles(tl.keys));
        int parts = 1, j0 = 0, j1 = nt;  // of this item; this part's key tiles
        if (splits > 1) {
            parts = kv4_parts(nt, sp);
            if (uniform(split >= parts)) break;
            j0 = (int)uniform((uint32_t)kv4_part_begin(nt, parts, split));
            j1 = (int)uniform((uint32_t)kv4_part_begin(nt, parts, split + 1));
        }
        const int row0 = i * kKv4ChunkRows;
        const int32_t *ids = a.table + (long long)r * a.max_blocks;
        const uint8_t *heads = a.pool + (long long)h * Kv4Tile<D>::kBytes;
        bits = 0;
        // this warp's block of key tile j
        auto id_of = [&](int j) { return j * 8 + warp < tl.blocks ? __ldg(ids + j * 8 + warp) : -1; };
        auto tile_of = [&](int j, int id) -> const uint8_t * {
            if (j * 8 + warp >= tl.blocks) return nullptr;
            if (id < 0 || id >= a.num_blocks) {
                bits = PKV_DEV_BAD_BLOCK;
                return nullptr;
            }
            return heads + id * block_bytes;
        };
        const int id0 = id_of(j0);
        int id1 = id_of(j0 + 1), id2 = id_of(j0 + 2);  // of the tiles that V and K are read of next
        Raw<D> rk, rv;
        const uint8_t *at = tile_of(j0, id0);
        rk.load(at, false, lane);
        rv.load(at, true, lane);

        // q: two threads a row, fp16 scaled by a power of two to lie in (-4, 4)
        {
            const int qr = tid >> 1, half = tid & 1, rr = row0 + qr, tok = kv4_over(rr, a.group, a.group_inv);
            constexpr int kC = D / 16;  // 16-byte chunks of a thread
            uint4 x[kC];
            uint32_t top = 0;
            if (qr < tl.rows) {
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    a.q + (long long)(q.q0 + tok) * a.q_stride + (long long)(h * a.group + rr - tok * a.group) * D) + half * kC;
#pragma unroll
                for (int c = 0; c < kC; ++c) x[c] = __ldg(src + c);
            } else {
#pragma unroll
                for (int c = 0; c < kC; ++c) x[c] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const uint32_t mk = 0x7fff7fffu;
                const uint32_t y = __vmaxu2(__vmaxu2(x[c].x & mk, x[c].y & mk), __vmaxu2(x[c].z & mk, x[c].w & mk));
                top = max(top, max(y & 0xffffu, y >> 16));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            // as in kv4_attention.cu
            int e = (int)(top >> 7);
            e = e == 255 ? 127 : min(max(e, 1), 253);
            const float down = __uint_as_float((uint32_t)(254 - e) << 23), up = __uint_as_float((uint32_t)e << 23);
            // neither 0 nor infinite
            if (half == 0) s_mul[qr] = qr < tl.rows ? fminf(fmaxf(up * a.small * a.scale_log2, 0x1p-126f), 0x1p127f) : 1.0f;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
                uint32_t f[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f[j] = half_bits(__floats2half2_rn(__uint_as_float(w[j] << 16) * down, __uint_as_float(w[j] & 0xffff0000u) * down));
                const int cc = half * kC + c;
                *reinterpret_cast<uint4 *>(smem + S::kQ + (cc >> 3) * S::kHalf + qr * 128 + (((cc & 7) ^ (qr & 7)) << 4)) =
                    make_uint4(f[0], f[1], f[2], f[3]);
            }
            if (tid < 8) s_nan[tid] = 0x7fffffff;
        }
        const uint32_t k_to = k_s + warp * 2048 + Raw<D>::k_place(lane), v_to = v_s + warp * 2048 + Raw<D>::v_place(lane);
        rk.put_k(k_to, lane);
        rk.load(tile_of(j0 + 1, id1), false, lane);
        fence_proxy_async_smem();
        __syncthreads();
        // keys that this row sees: some of any part, which is longer than a tile (padding
        // rows: one)
        const int rr = row0 + row;
        const int limit = row < tl.rows ? q.len - q.n + kv4_over(rr, a.group, a.group_inv) + 1 : j0 * kKeys + 1;
        const float mul = s_mul[row];
        float m = -INFINITY, l = 0.0f;
        bool large = false;  // some row's reference is

        for (int j = j0; j < j1; ++j) {
            if (warp == 0) {
                tmem_fence_after_sync();
#pragma unroll
                for (int c = 0; c < D / 64; ++c) mma_ss4(tmu, q_lo + c * (S::kHalf >> 4), k_lo + c * (S::kHalf >> 4), kIdS, c);
                commit(smem_u32(bar_s));
            }
            const int key0 = j * kKeys;
            rv.put_v(v_to, tl.keys - key0 - 16 * warp, key0 + 16 * warp, s_nan, lane);
            fence_proxy_async_smem();
            warp_wait(bar_s, phase, abort);
            tmem_fence_after_sync();
            const uint32_t s_at = tm_row + part * 64;
            const int mine = limit - key0 - part * 64;  // of these keys, the row sees so many
            const bool masked = !__all_sync(0xffffffffu, mine >= 64);
            auto scores = [&](int c, float (&s)[32]) {  // 32 of them
                tmem_ld32(s_at + 32 * c, s);
                tmem_wait_ld_regs(s);
                if (masked) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * c + e >= mine) s[e] = -INFINITY;
                }
            };
            // The reference becomes the row's largest score so far; O and l follow.
            auto move = [&](bool all) {
                float best = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    float s[32];
                    scores(c, s);
#pragma unroll
                    for (int e = 0; e < 16; ++e) best = fmax3(best, s[2 * e], s[2 * e + 1]);
                }
                s_x[part * 128 + row] = best;
                named_barrier_sync(1 + (warp & 3), 64);
                const float to = fmaxf(m, fmaxf(s_x[row], s_x[128 + row]));
                const float f = m == to ? 1.0f : m == -INFINITY ? 0.0f : fast_exp2((m - to) * mul);
                m = to;
                l *= f;
                large = __any_sync(0xffffffffu, !(fabsf(m * mul) <= 1024.0f));
                if (all) {
#pragma unroll 1
                    for (int c = 0; c < D / 64; ++c) {
                        float o[32];
                        const uint32_t at_o = tm_row + kColO + part * (D / 2) + 32 * c;
                        tmem_ld32(at_o, o);
                        tmem_wait_ld_regs(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= f;
                        tmem_st32(at_o, o);
                    }
                    tmem_wait_st();
                }
                named_barrier_sync(1 + (warp & 3), 64);  // the maxima are read
            };
            if (j == j0) move(false);
            uint32_t p[32];
            float2 sum;
            for (int round = 0;; ++round) {
                const float2 mm = make_float2(mul, mul);
                sum = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float s[32];
                    scores(c, s);
                    auto exps = [&](auto exponent) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 y = exponent(make_float2(s[2 * e], s[2 * e + 1]));
                            const float2 z = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                            sum = fadd2(sum, z);
                            p[16 * c + e] = half_bits(__floats2half2_rn(z.x, z.y));
                        }
                    };
                    // One rounding where the reference's own, mul * m, is small: at 2^10 it is
                    // off by 2^-15, for a whole row and tile alike.
                    if (!large) {
                        const float2 nm = make_float2(-m * mul, -m * mul);
                        exps([&](float2 x) { return ffma2(x, mm, nm); });
                    } else {
                        const float2 nm = make_float2(-m, -m);
                        exps([&](float2 x) { return fmul2(fadd2(x, nm), mm); });
                    }
                }
                // The reference moves when the sum shows that a p may be large: none is
                // above 2^12 until then, and fits fp16. Behind this barrier both halves of these rows have read their
                // scores, and P may go over them.
                tmem_fence_before_sync();
                const bool again = pair_any(1 + (warp & 3), !(sum.x + sum.y <= 4096.0f));
                tmem_fence_after_sync();
                if (!again || round) break;  // against the largest score none is past it
                move(j > j0);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) tmem_st16u(tm_row + part * 32 + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(p + 16 * c));
            l += sum.x + sum.y;
            tmem_wait_st();
            tmem_fence_before_sync();
            __syncthreads();
            if (warp == 0) {
                tmem_fence_after_sync();
#pragma unroll
                for (int c = 0; c < 2; ++c) mma_ts4(tmu + kColO, tmu + c * 32, v_lo + c * (8192 >> 4), kIdPv, c | (j - j0));
                commit(smem_u32(bar_pv));
            }
            if (j + 1 < j1) {
                rv.load(tile_of(j + 1, id1), true, lane);
                rk.put_k(k_to, lane);
                rk.load(tile_of(j + 2, id2), false, lane);
                id1 = id2;
                id2 = id_of(j + 3);
                fence_proxy_async_smem();
            } else if (splits > 1) {
                if (tid == 0) s_claim = pieces;
            } else if (tid == 0) {
                // the next item: CTA b has item b without a claim, every item claims another, and
                // the last of these claims leaves the counter as it was
                const int seen = atomicAdd(a.claimed, 1) - kKv4Nobody;
                if (seen == total - 1) atomicExch(a.claimed, kKv4Nobody);
                if (seen < 0 || seen >= total) raise_status(a.status, PKV_DEV_BAD_WORKSPACE);
                s_claim = seen < 0 || seen >= total ? total : ctas + seen;
            }
            warp_wait(bar_pv, phase, abort);
            phase ^= 1;
            __syncthreads();
            if (uniform(*abort)) break;
        }
        if (uniform(*abort)) break;
        tmem_fence_after_sync();
        s_x[part * 128 + row] = l;
        named_barrier_sync(1 + (warp & 3), 64);
        l = s_x[row] + s_x[128 + row];
        if (parts > 1) {
            // this part for the last of the item's to arrive, which adds them up in order
            float *mine = reinterpret_cast<float *>(a.parts) + (size_t)piece * kv4_chunk_part(D);
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
                float o[32];
                tmem_ld32(tm_row + kColO + part * (D / 2) + 32 * c, o);
                tmem_wait_ld_regs(o);
#pragma unroll
                for (int gI = 0; gI < 2; ++gI)
                    if (s_nan[part * (D / 32) + 2 * c + gI] < limit)
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[16 * gI + e] = __uint_as_float(0x7fffffffu);
                // rows next to each other: [4 columns][row]
                float4 *to = reinterpret_cast<float4 *>(mine) + (part * (D / 8) + 8 * c) * kKv4ChunkRows + row;
#pragma unroll
                for (int e = 0; e < 8; ++e) to[e * kKv4ChunkRows] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
            if (part == 0) reinterpret_cast<float2 *>(mine + kKv4ChunkRows * D)[row] = make_float2(m, l);
            __syncthreads();
            if (tid == 0) {
                int seen;
                asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(seen) : "l"(a.arrived + item) : "memory");
                seen -= kKv4Nobody;
                if (seen == parts - 1) atomicExch(a.arrived + item, kKv4Nobody);
                if (seen < 0 || seen >= parts) raise_status(a.status, PKV_DEV_BAD_WORKSPACE);
                s_last = seen == parts - 1;
            }
            __syncthreads();
            if (s_last && row < tl.rows) {
                const int tok = kv4_over(rr, a.group, a.group_inv);
                join_parts<D>(reinterpret_cast<const float *>(a.parts) + (size_t)item * kv4_chunk_part(D), (size_t)total * kv4_chunk_part(D), parts, mul,
                              a.v_scale, row, part,
                              a.out + ((long long)(q.q0 + tok) * a.num_kv_heads * a.group + h * a.group + rr - tok * a.group) * D + part * (D / 2));
            }
            if (__any_sync(0xffffffffu, bits != 0) && lane == 0) raise_status(a.status, PKV_DEV_BAD_BLOCK);
            break;
        }
        const float f = a.v_scale / l;
        const int tok = kv4_over(rr, a.group, a.group_inv);
        __nv_bfloat16 *out = a.out + ((long long)(q.q0 + tok) * a.num_kv_heads * a.group + h * a.group + rr - tok * a.group) * D + part * (D / 2);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            float o[32];
            tmem_ld32(tm_row + kColO + part * (D / 2) + 32 * c, o);
            tmem_wait_ld_regs(o);
            if (row < tl.rows) {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= f;
#pragma unroll
                for (int gI = 0; gI < 2; ++gI)
                    if (s_nan[part * (D / 32) + 2 * c + gI] < limit)
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[16 * gI + e] = __uint_as_float(0x7fffffffu);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    reinterpret_cast<uint4 *>(out + 32 * c)[e] =
                        make_uint4(pack_bf16x2(o[8 * e], o[8 * e + 1]), pack_bf16x2(o[8 * e + 2], o[8 * e + 3]),
                                   pack_bf16x2(o[8 * e + 4], o[8 * e + 5]), pack_bf16x2(o[8 * e + 6], o[8 * e + 7]));
            }
        }
        if (__any_sync(0xffffffffu, bits != 0) && lane == 0) raise_status(a.status, PKV_DEV_BAD_BLOCK);
        tmem_fence_before_sync();
        piece = (int)uniform((uint32_t)s_claim);
        __syncthreads();
        tmem_fence_after_sync();
    }
    if (warp == 0) {
        // no product may still be on its way when the tensor memory is freed
        commit(smem_u32(bar_end));
        int never = 0;
        if (!warp_wait(bar_end, 0, &never) || *abort)
            if (lane == 0) raise_status(a.status, PKV_DEV_TIMEOUT);
    }
    __syncthreads();
    if (warp == 0) {
        tmem_fence_after_sync();
        tmem_dealloc(tm, kTmemCols);
    }
}

std::mutex g_mu;
bool g_ready[64][2];

template <int D>
int launch(const Kv4Args &a, int sms, cudaStream_t st) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_E_CUDA;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        if (!g_ready[dev][D == 128]) {
            if (cudaFuncSetAttribute(kv4_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kAlloc) != cudaSuccess)
                return PKV_E_CUDA;
            g_ready[dev][D == 128] = true;
        }
    }
    return launch_pdl(kv4_chunk_kernel<D>, dim3(kKv4ChunkCtas * sms), dim3(kThreads), Smem<D>::kAlloc, st, a) == cudaSuccess ? PKV_OK : PKV_E_CUDA;
}

}  // namespace

int kv4_chunk_launch(const Kv4Args &a, int head_size, int sms, cudaStream_t stream) {
    return head_size == 128 ? launch<128>(a, sms, stream) : launch<64>(a, sms, stream);
}

}  // namespace pkv
