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
//   P_t               one thread per row: S to registers, causal mask, row
//                     maximum, exponentials against a running reference that
//                     moves (O rescaled) only when the maximum outgrows it by
//                     2^8; bf16 pairs over S's own columns in TMEM, handed on
//                     in two halves so that the product of the first half of
//                     the keys runs during the second half's exponentials;
//   O_t += P_t V      tcgen05.mma, A = P_t from TMEM, B = V as it lies.
// The softmax of A runs while the tensor core works for B and the other way
// round. The sums l are of the unrounded p; rounding P to bf16 (2^-9 of each
// term) is what the tensor core takes.
//
// Warps: 0-3 softmax and output of A, 4-7 of B, 8 MMA issue and TMEM, 9
// copies and the item list. The grid is persistent. The host does not know
// the lengths, and no workspace is needed: items are numbered by tile level
// (longest keys first) over all sequences, every CTA counts the tiles once,
// and its copy warp finds its next item by a binary search over levels while
// the current one runs. CTA b takes item b, then counts back from the end of
// every second round, so that the rounds' longest items alternate.
//
// Every wait is bounded; on a timeout the CTA raises PKV_DEV_TIMEOUT, stops,
// lets its copies and MMAs in flight finish and frees its TMEM.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <mutex>

#include "pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr int kRows = 128, kKeys = 128;
constexpr int kMmaWarp = 0, kCopyWarp = 1, kSoftmaxWarp = 4, kOutWarp = 12;  // softmax 4-11, output 12-15
constexpr int kThreads = 512;
// Registers a thread: the softmax holds a row of 128 scores and 32 words of P.
// Four warpgroups of 128 at launch: 2 * (64 + 192) = 4 * 128.
constexpr int kSoftmaxRegs = 192, kOtherRegs = 64;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;           // S_A 0, S_B 128, O_A 256, O_B 256 + D
constexpr float kRescaleThreshold = 8.f;  // log2 units: P stays <= 2^8
constexpr int kSeqCache = 4096;           // sequences whose tile counts are kept in shared memory
constexpr float kLog2e = 1.4426950408889634f;

struct PromptArgs {
    const __nv_bfloat16 *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    __nv_bfloat16 *out;
    const int32_t *qsl;
    int num_tokens, num_reqs, num_q_heads, num_kv_heads, group, tile_tokens;  // tile_tokens = 128 / group
    float scale;
    int32_t *status;
};

// One work item: tokens [i0, i0 + 2 tile_tokens) of the sequence of n tokens
// that starts at token q0; n_keys[t]: key tiles that query tile t sees.
struct Item {
    int valid, q0, n, i0, h, n_keys[2], pad;
};

struct Bars {
    static constexpr int kQFull = 0, kQEmpty = 2, kSFull = 4, kPFull = 6 /* [tile][half] */, kPvDone = 10, kDFull = 12,
                         kDEmpty = 14, kOFull = 16, kLFull = 18, kOFree = 20, kDrain = 22, kKvFull = 23;
};

template <int D>
struct Smem {
    static constexpr int kStages = D == 128 ? 4 : 8;  // K and V tiles in turn
    static constexpr int kHalf = 16384;               // 128 rows x 128 B (64 bf16 columns)
    static constexpr int kTile = (D / 64) * kHalf;
    static constexpr int kOffQ = 0;
    static constexpr int kOffKv = 2 * kTile;
    static constexpr int kOffItem = kOffKv + kStages * kTile;
    static constexpr int kOffBar = kOffItem + 2 * (int)sizeof(Item);
    static constexpr int kBars = Bars::kKvFull + 2 * kStages;
    static constexpr int kOffSum = kOffBar + kBars * 8;  // float [tile][row]: sums of p
    static constexpr int kOffSeq = kOffSum + 2 * kRows * 4;
    static constexpr int kBytes = kOffSeq + kSeqCache * 4;
    static constexpr int kAlloc = kBytes + 1024;
};
static_assert(Smem<128>::kAlloc <= 232448 - 1024, "prompt kernel shared memory");
static_assert(Smem<64>::kAlloc <= 232448 - 1024, "prompt kernel shared memory");

// A bounded wait that the whole warp leaves with one answer. No call in it:
// values that live across a call are kept out of uniform registers, where the
// MMA instructions want them (60 to 90 cycles an MMA instead of 15, more than
// the tensor core's 64), and a role's registers must not pass through one.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int32_t *status, volatile int *abort) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const unsigned long long t0 = global_timer_ns();
    for (uint32_t n = 1;; ++n) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (n % 32 == 0) {
            const bool late = global_timer_ns() - t0 > kWaitTimeoutNs;
            if (late) {
                raise_status(status, PKV_DEV_TIMEOUT);
                *abort = 1;
            }
            if (__any_sync(0xffffffffu, late || *abort)) return false;
        }
    }
}

// A value that all lanes hold, as the compiler can know it too.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_or_sync(0xffffffffu, v); }

// Shared-memory matrix descriptors (128-byte swizzle) as their two words: the
// low one holds the address and the leading offset, the high one is the same
// for every operand here (8-row groups 1024 bytes apart).
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

// Item tiles of sequence r; 0 for an empty or a bad one (bad: reported).
__device__ __forceinline__ int seq_tiles(const PromptArgs &a, int r, bool report) {
    const int q0 = __ldg(a.qsl + r), q1 = __ldg(a.qsl + r + 1);
    if (q0 < 0 || q1 < q0 || q1 > a.num_tokens) {
        if (report) raise_status(a.status, PKV_DEV_BAD_QSL);
        return 0;
    }
    const int per = 2 * a.tile_tokens;
    return (int)(((long long)q1 - q0 + per - 1) / per);
}

// One output row by the definition, by a whole warp: for rows whose tile
// product met an infinity or NaN. The product multiplies masked values by a
// probability of 0, which is exact unless the value is not finite; here a
// token's sum takes its visible keys only.
template <int D>
__device__ __noinline__ void exact_row(const PromptArgs &a, int q0, int i, int head, int lane) {
    constexpr int kE = D / 32;
    const int h = head / a.group;
    const __nv_bfloat16 *q = a.q + ((long long)q0 + i) * a.q_stride + head * D + lane * kE;
    const __nv_bfloat16 *k = a.k + (long long)q0 * a.k_stride + h * D + lane * kE;
    const __nv_bfloat16 *v = a.v + (long long)q0 * a.v_stride + h * D + lane * kE;
    float qv[kE], acc[kE], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        qv[e] = __bfloat162float(q[e]);
        acc[e] = 0.f;
    }
    auto score = [&](int j) {
        const __nv_bfloat16 *kj = k + j * a.k_stride;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < kE; ++e) s = fmaf(qv[e], __bfloat162float(kj[e]), s);
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        return s * a.scale;
    };
#pragma unroll 1
    for (int j = 0; j <= i; ++j) m = fmaxf(m, score(j));
#pragma unroll 1
    for (int j = 0; j <= i; ++j) {
        const float p = exp2f((score(j) - m) * kLog2e);
        const __nv_bfloat16 *vj = v + j * a.v_stride;
        l += p;
#pragma unroll
        for (int e = 0; e < kE; ++e) acc[e] = fmaf(p, __bfloat162float(vj[e]), acc[e]);
    }
    __nv_bfloat16 *o = a.out + (((long long)q0 + i) * a.num_q_heads + head) * D + lane * kE;
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = __float2bfloat16(acc[e] / l);
}

template <int D>
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
    uint64_t *o_free = bar + Bars::kOFree, *drain = bar + Bars::kDrain;
    float *row_sum = reinterpret_cast<float *>(smem + M::kOffSum);
    uint64_t *kv_full = bar + Bars::kKvFull, *kv_empty = kv_full + kStages;
    Item *items = reinterpret_cast<Item *>(smem + M::kOffItem);
    int *seq = reinterpret_cast<int *>(smem + M::kOffSeq);
    volatile int *abort = &s_abort;
    int32_t *status = a.status;
    // broadcast: the compiler then knows that a role's branch is the whole warp's (see uniform())
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        s_abort = 0;
        s_levels = 0;
        s_tiles = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[2 * i], 4);
            mbar_init(&p_full[2 * i + 1], 4);
            mbar_init(&pv_done[i], 1);
            mbar_init(&d_full[i], 1);
            mbar_init(&d_empty[i], 13);  // the MMA, softmax and output warps
            mbar_init(&o_full[i], 1);
            mbar_init(&l_full[i], 4);
            mbar_init(&o_free[i], 4);
        }
        mbar_init(drain, 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        mbar_fence_init();
    }
    pdl_launch_dependents();
    pdl_wait();
    __syncthreads();
    {
        int most = 0;
        unsigned long long sum = 0;
        for (int r = threadIdx.x; r < a.num_reqs; r += kThreads) {
            const int n = seq_tiles(a, r, blockIdx.x == 0);
            if (r < kSeqCache) seq[r] = n;
            most = max(most, n);
            sum += n;
        }
        if (sum) {
            atomicMax(&s_levels, most);
            atomicAdd(&s_tiles, sum);
        }
    }
    if (warp == kMmaWarp) tmem_alloc(&s_tmem, kTmemCols);
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tm = s_tmem;
    if (warp == kCopyWarp) {
        // ------------------------ items, Q, K and V ------------------------
        setmaxnreg_dec<kOtherRegs>();
        if (lane == 0) {
            tma_prefetch_desc(&q_map);
            tma_prefetch_desc(&k_map);
            tma_prefetch_desc(&v_map);
        }
        const int Hkv = a.num_kv_heads, R = a.num_reqs;
        const long long total = (long long)s_tiles * Hkv;
        auto tiles_of = [&](int r) { return r < kSeqCache ? seq[r] : seq_tiles(a, r, false); };
        // Items of level m or above (level m: a sequence's m-th pair of query
        // tiles, so m grows with the keys seen).
        auto items_from = [&](int m) {
            long long c = 0;
            for (int r = lane; r < R; r += 32) c += max(0, tiles_of(r) - m);
#pragma unroll
            for (int d = 16; d; d >>= 1) c += __shfl_xor_sync(0xffffffffu, c, d);
            return c * Hkv;
        };
        int hi = s_levels;        // items_from(hi) <= every item still to come
        long long above = 0;      // items_from(hi)
        uint32_t x = 0;           // K and V tiles issued
        uint32_t q_used = 0, q_any = 0;  // bit t: parity of Q_t's tiles copied; any copied
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const long long it = (long long)k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            Item w{};
            if (it < total) {
                // largest level m with items_from(m) > it
                int lo = 0;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    const long long c = items_from(mid);
                    if (c > it) {
                        lo = mid;
                    } else {
                        hi = mid;
                        above = c;
                    }
                }
                const long long idx = it - above;
                long long want = idx / Hkv;  // the want-th sequence with more than lo tiles
                w.h = (int)(idx % Hkv);
                int r = 0;
                for (int r0 = 0; r0 < R; r0 += 32) {
                    const unsigned has = __ballot_sync(0xffffffffu, r0 + lane < R && tiles_of(r0 + lane) > lo);
                    const int c = __popc(has);
                    if (want < c) {
                        r = r0 + (int)__fns(has, 0, (int)want + 1);
                        break;
                    }
                    want -= c;
                }
                w.valid = 1;
                w.q0 = __ldg(a.qsl + r);
                w.n = __ldg(a.qsl + r + 1) - w.q0;
                w.i0 = lo * 2 * a.tile_tokens;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int last = min(w.n, w.i0 + (t + 1) * a.tile_tokens);  // past the tile's last token
                    w.n_keys[t] = last > w.i0 + t * a.tile_tokens ? (last + kKeys - 1) / kKeys : 0;
                }
            }
            if (!warp_wait(&d_empty[k & 1], ((k >> 1) & 1) ^ 1, status, abort)) { ok = false; break; }
            if (lane == 0) {
                items[k & 1] = w;
                mbar_arrive(&d_full[k & 1]);
            }
            __syncwarp();
            if (!w.valid) break;
            // Q_A, K(0), Q_B, V(0), K(1), V(1), ...
            const int nt = max(w.n_keys[0], w.n_keys[1]);
#pragma unroll 1
            for (int i = 0; i < 2 * nt && ok; ++i, ++x) {
                if (i < 2 && w.n_keys[i]) {
                    if (!warp_wait(&q_empty[i], ((q_used >> i) & 1) ^ 1, status, abort)) { ok = false; break; }
                    q_used ^= 1u << i;
                    q_any |= 1u << i;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&q_full[i], a.tile_tokens * a.group * D * 2);
#pragma unroll
                        for (int b = 0; b < D / 64; ++b)
                            tma_load_3d(smem + M::kOffQ + i * M::kTile + b * M::kHalf, &q_map, b * 64, w.h * a.group,
                                        w.q0 + w.i0 + i * a.tile_tokens, &q_full[i]);
                    }
                    __syncwarp();
                }
                const int st = x % kStages;
                if (!warp_wait(&kv_empty[st], ((x / kStages) & 1) ^ 1, status, abort)) { ok = false; break; }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&kv_full[st], kKeys * D * 2);
                    tma_load_4d(smem + M::kOffKv + st * M::kTile, i & 1 ? &v_map : &k_map, 0, w.q0 + (i >> 1) * kKeys, 0,
                                w.h, &kv_full[st]);
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) {
            // let copies already issued land before the CTA can leave
            for (uint32_t y = x > (uint32_t)kStages ? x - kStages : 0; y < x; ++y)
                mbar_drain(&kv_full[y % kStages], (y / kStages) & 1, status, nullptr, 0);
            for (int t = 0; t < 2; ++t)
                if (q_any >> t & 1) mbar_drain(&q_full[t], ((q_used >> t) & 1) ^ 1, status, nullptr, 0);
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
        uint32_t x = 0;      // K and V tiles of the items so far
        uint32_t q_used = 0, pv0 = 0, pv1 = 0;  // q_used: parity bits of Q tiles taken; pv: PV products issued
        uint32_t o_used = 0;                    // parity bits of the outputs written
        bool ok = true;
        auto kv_wait = [&](uint32_t y) {
            return warp_wait(&kv_full[y % kStages], (y / kStages) & 1, status, abort);
        };
        for (int k = 0; ok; ++k) {
            if (!warp_wait(&d_full[k & 1], (k >> 1) & 1, status, abort)) { ok = false; break; }
            const Item w = items[k & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[k & 1]);
            if (!uniform(w.valid)) break;
            const int nA = uniform(w.n_keys[0]), nB = uniform(w.n_keys[1]), nt = max(nA, nB);
            // Step j: O_t += P_t(j) V(j), then S_t(j + 1), for A, then for B.
#pragma unroll 1
            for (int j = -1; j < nt && ok; ++j) {
                const uint32_t yv = x + 2 * j + 1, yk = yv + 1;  // V(j), K(j + 1)
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    const int n_t = t ? nB : nA;
                    const uint32_t pv = t ? pv1 : pv0;
                    if (j >= 0 && j < n_t) {
                        const uint32_t b_lo = v_lo + (yv % kStages) * (M::kTile >> 4);
                        if (t == 0 || j >= nA) ok = kv_wait(yv);
                        if (ok && j == 0) {  // the previous item's O has been read
                            ok = warp_wait(&o_free[t], ((o_used >> t) & 1) ^ 1, status, abort);
                            o_used ^= 1u << t;
                        }
#pragma unroll 1
                        for (int half = 0; half < 2 && ok; ++half) {
                            ok = warp_wait(&p_full[2 * t + half], pv & 1, status, abort);
                            if (!ok) break;
                            tmem_fence_after_sync();
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_ts(tmu + kColO + t * D, tmu + t * kKeys + half * 32 + kk * 8,
                                       b_lo + (half * 4 + kk) * (2048 >> 4), kIdPV, (j > 0 || half > 0 || kk > 0) ? 1u : 0u);
                        }
                        if (!ok) break;
                        umma_commit_warp(&pv_done[t]);
                        if (t) ++pv1; else ++pv0;
                        if (j + 1 == n_t) umma_commit_warp(&o_full[t]);
                        // A sees no more key tiles than B, unless B is empty.
                        if (t == 1 || j >= nB) umma_commit_warp(&kv_empty[yv % kStages]);
                    }
                    if (j + 1 < n_t) {
                        if (j < 0) {
                            ok = warp_wait(&q_full[t], (q_used >> t) & 1, status, abort);
                            q_used ^= 1u << t;
                        }
                        if (ok && (t == 0 || j + 1 >= nA)) ok = kv_wait(yk);
                        // S_t goes into columns that hold the P of t's
                        // previous product: that one has to be over first.
                        const uint32_t done = t ? pv1 : pv0;
                        if (ok && done > 0) ok = warp_wait(&pv_done[t], (done - 1) & 1, status, abort);
                        if (!ok) break;
                        tmem_fence_after_sync();
                        const uint32_t a_lo = q_lo + t * (M::kTile >> 4);
                        const uint32_t b_lo = k_lo + (yk % kStages) * (M::kTile >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_ss(tmu + t * kKeys, a_lo + (kk / 4) * (M::kHalf >> 4) + (kk % 4) * 2,
                                   b_lo + (kk / 4) * (M::kHalf >> 4) + (kk % 4) * 2, kIdS, kk > 0 ? 1u : 0u);
                        umma_commit_warp(&s_full[t]);
                        if (t == 1 || j + 1 >= nB) umma_commit_warp(&kv_empty[yk % kStages]);
                        if (j + 2 == n_t) umma_commit_warp(&q_empty[t]);
                    }
                }
            }
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
        const float scale_log2 = a.scale * kLog2e;
        const int g = a.group;
        uint32_t x = 0;   // K and V tiles of the items so far
        uint32_t n = 0, n_out = 0;  // key tiles and items this query tile has been through
        for (int k = 0;; ++k) {
            if (!warp_wait(&d_full[k & 1], (k >> 1) & 1, status, abort)) break;
            const Item w = items[k & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[k & 1]);
            if (!w.valid) break;
            const int n_t = w.n_keys[t], nt = max(w.n_keys[0], w.n_keys[1]);
            if (n_t == 0) {
                x += 2 * nt;
                continue;
            }
            const int i0 = w.i0 + t * a.tile_tokens;
            const int i = i0 + row / g;
            const bool valid = row < a.tile_tokens * g && i < w.n;
            // Rows past the tile's tokens hold other tokens or nothing; what
            // they compute is dropped.
            const int limit = valid ? i : min(w.n, i0 + a.tile_tokens) - 1;
            const int first_limit = __reduce_min_sync(0xffffffffu, limit);
            float m = 0.f, l = 0.f;
            bool ok = true;
            for (int j = 0; j < n_t; ++j, ++n) {
                if (!warp_wait(&s_full[t], n & 1, status, abort)) { ok = false; break; }
                tmem_fence_after_sync();
                float s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(s_col + c * 32, s[c]);
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_wait_ld_regs(s[c]);
                if ((j + 1) * kKeys - 1 > first_limit) {
                    const int lim = limit - j * kKeys;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[c][e] = c * 32 + e <= lim ? s[c][e] : -INFINITY;
                }
                float mx[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    mx[c] = fmaxf(s[c][0], s[c][1]);
#pragma unroll
                    for (int e = 2; e < 32; e += 2) mx[c] = fmax3(mx[c], s[c][e], s[c][e + 1]);
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale_log2;
                // V rows past the sequence belong to the next one, or to
                // nobody: their P is 0, but 0 times NaN is not. The first
                // query tile that takes this V tile clears them.
                if ((j + 1) * kKeys > w.n && (t == 0 || j >= w.n_keys[0])) {
                    const uint32_t y = x + 2 * j + 1;
                    if (!warp_wait(&kv_full[y % kStages], (y / kStages) & 1, status, abort)) { ok = false; break; }
                    uint8_t *vt = smem + M::kOffKv + (y % kStages) * M::kTile;
                    const int first = w.n - j * kKeys, words = (kKeys - first) * 8;
#pragma unroll 1
                    for (int b = 0; b < D / 64; ++b)
#pragma unroll 1
                        for (int c = row; c < words; c += kRows)
                            *reinterpret_cast<uint4 *>(vt + b * M::kHalf + first * 128 + c * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                // P of the first 64 keys against the reference as it stands, so
                // that the exponentials need not wait for the maximum; where a
                // row of the warp moves its reference (always on the first tile)
                // they are made again.
                const float2 sc2 = make_float2(scale_log2, scale_log2);
                auto exps = [&](const float (&v0)[32], const float (&v1)[32], uint32_t (&p)[32]) {
                    const float2 nm2 = make_float2(-m, -m);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float *v = e < 16 ? &v0[2 * e] : &v1[2 * e - 32];
                        const float2 z = ffma2(make_float2(v[0], v[1]), sc2, nm2);
                        const float2 pe = make_float2(fast_exp2(z.x), fast_exp2(z.y));
                        sum[e & 1] = fadd2(sum[e & 1], pe);
                        p[e] = pack_bf16x2(pe.x, pe.y);
                    }
                    return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                };
                uint32_t p[32];
                float sum;
                bool first = j == 0;
                while (true) {
                    sum = exps(s[0], s[1], p);
                    const bool moves = first || top > m + kRescaleThreshold;
                    if (!__any_sync(0xffffffffu, moves)) break;
                    first = false;
                    const float alpha = moves ? fast_exp2(m - top) : 1.f;
                    if (moves) m = top;
                    if (j == 0) continue;
                    // PV(j - 1) was over before S(j) was issued: O is at rest.
                    l *= alpha;
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        float o[16];
                        tmem_ld16(o_col + c * 16, o);
                        tmem_wait_ld_regs(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= alpha;
                        tmem_st16(o_col + c * 16, o);
                    }
                }
                auto hand_on = [&](int half) {
                    tmem_st32u(s_col + half * 32, p);
                    tmem_wait_st();
                    tmem_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * t + half]);
                };
                hand_on(0);
                // not ahead of the first half's hand-over
                keep(s[2]);
                keep(s[3]);
                l += sum;
                l += exps(s[2], s[3], p);
                hand_on(1);
            }
            x += 2 * nt;
            if (!ok || !warp_wait(&o_free[t], (n_out & 1) ^ 1, status, abort)) break;
            ++n_out;
            row_sum[t * kRows + row] = l;
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
        uint32_t used = 0;  // parity bits of the outputs so far
        bool ok = true;
        for (int k = 0; ok; ++k) {
            if (!warp_wait(&d_full[k & 1], (k >> 1) & 1, status, abort)) break;
            const Item w = items[k & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[k & 1]);
            if (!w.valid) break;
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {
                if (!w.n_keys[t]) continue;
                const uint32_t par = (used >> t) & 1;
                used ^= 1u << t;
                ok = warp_wait(&l_full[t], par, status, abort) && warp_wait(&o_full[t], par, status, abort);
                if (!ok) break;
                tmem_fence_after_sync();
                const int i = w.i0 + t * a.tile_tokens + row / g;
                const bool valid = row < a.tile_tokens * g && i < w.n;
                const float inv = 1.f / row_sum[t * kRows + row];
                const int head = w.h * g + row % g;
                __nv_bfloat16 *dst = a.out + (((long long)w.q0 + i) * a.num_q_heads + head) * D;
                float odd = 0.f;  // NaN once an output is not finite
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    float o[16];
                    tmem_ld16(o_col + t * D + c, o);
                    tmem_wait_ld_regs(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        o[e] *= inv;
                        odd = fmaf(o[e], 0.f, odd);
                    }
                    if (valid) {
#pragma unroll
                        for (int e = 0; e < 16; e += 8)
                            *reinterpret_cast<uint4 *>(dst + c + e) =
                                make_uint4(pack_bf16x2(o[e], o[e + 1]), pack_bf16x2(o[e + 2], o[e + 3]),
                                           pack_bf16x2(o[e + 4], o[e + 5]), pack_bf16x2(o[e + 6], o[e + 7]));
                    }
                }
                tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_free[t]);
                unsigned redo = __ballot_sync(0xffffffffu, valid && odd != 0.f);
                while (redo) {
                    const int src = __ffs(redo) - 1;
                    redo &= redo - 1;
                    __syncwarp();
                    exact_row<D>(a, w.q0, __shfl_sync(0xffffffffu, i, src), __shfl_sync(0xffffffffu, head, src), lane);
                }
            }
        }
    } else {
        setmaxnreg_dec<kOtherRegs>();  // warps 2 and 3: a warpgroup gives up registers together
    }

    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    if (warp == kMmaWarp) tmem_dealloc(tm, kTmemCols);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

struct PromptDevice {
    int sm_count = 0;
    bool ready = false;
};
std::mutex g_mu;
PromptDevice g_dev[64];
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

int prompt_device(int *sm_count) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_E_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    PromptDevice &d = g_dev[dev];
    if (!d.ready) {
        if (cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaFuncSetAttribute(prompt_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<64>::kAlloc) !=
                cudaSuccess ||
            cudaFuncSetAttribute(prompt_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Smem<128>::kAlloc) != cudaSuccess)
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
        d.ready = true;
    }
    *sm_count = d.sm_count;
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
    if (num_tokens > INT32_MAX - 65536 || num_reqs > INT32_MAX - 65536) return PKV_E_DIMS;
    if (num_q_heads <= 0 || num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > kRows) return PKV_E_GQA;
    if (!(scale > 0.f) || scale > 3.0e38f) return PKV_E_DIMS;
    if (num_tokens == 0 || num_reqs == 0) return PKV_OK;
    if (!q || !k || !v || !query_start_loc || !out) return PKV_E_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(query_start_loc, 4) ||
        !aligned(status, 4))
        return PKV_E_ALIGN;
    const long long wq = (long long)num_q_heads * head_size, wkv = (long long)num_kv_heads * head_size;
    if (!stride_ok(q_stride, wq) || !stride_ok(k_stride, wkv) || !stride_ok(v_stride, wkv)) return PKV_E_DIMS;
    int sms = 0;
    int rc = prompt_device(&sms);
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
    a.status = status;
    CUtensorMap q_map, k_map, v_map;
    rc = encode_q(&q_map, q, num_tokens, q_stride, num_q_heads, head_size, a.group);
    if (!rc) rc = encode_kv(&k_map, k, num_tokens, k_stride, num_kv_heads, head_size);
    if (!rc) rc = encode_kv(&v_map, v, num_tokens, v_stride, num_kv_heads, head_size);
    if (rc) return rc;
    // at most this many items: every sequence rounds up to whole pairs of tiles
    const long long most = (num_tokens / (2LL * a.tile_tokens) + num_reqs) * num_kv_heads;
    const int grid = (int)(most < sms ? most : sms);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t err =
        head_size == 128
            ? launch_pdl(prompt_kernel<128>, dim3(grid), dim3(kThreads), Smem<128>::kAlloc, st, q_map, k_map, v_map, a)
            : launch_pdl(prompt_kernel<64>, dim3(grid), dim3(kThreads), Smem<64>::kAlloc, st, q_map, k_map, v_map, a);
    return err == cudaSuccess ? PKV_OK : PKV_E_CUDA;
}
