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
// in the workspace.
//
// Bound by: tensor core (1024 cycles a tile and CTA at D 128), exponentials (512) and
// issue slots (about 900) together.
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
    static constexpr int kHalf = 128 * 128;      // q: 128 rows x 64 columns
    static constexpr int kGrp = (D / 64) * 1024;  // K, V: 8 keys, [D / 64][8][128 B]
    static constexpr int kTile = (D / 64) * kHalf;
    static constexpr int kQ = 0, kK = kTile, kV = 2 * kTile;
    static constexpr int kX = 3 * kTile;         // float [2][128]: the halves' maxima, at last their sums
    static constexpr int kMul = kX + 2 * 128 * 4;
    static constexpr int kNan = kMul + 128 * 4;  // first key whose V is no number, by groups of 16 columns
    static constexpr int kBar = kNan + 8 * 4;
    static constexpr int kBytes = kBar + 2 * 8;
    static constexpr int kAlloc = kBytes + 1024;
};

constexpr uint32_t idesc_f16(int M, int N, int b_mn_major) {
    return (1u << 4) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
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
    __device__ __forceinline__ void put_k(uint8_t *to, int lane) const {
        const int g = lane >> 2, t = lane & 3;
        constexpr int kGrp = Smem<D>::kGrp;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint8_t *row = to + h * kGrp + (D == 128 ? (t >> 1) * 1024 : 0) + g * 128;
            const __half2 sc = kv4_scales(D == 128 ? scales >> (16 * h) : scales);
#pragma unroll
            for (int i = 0; i < kW; ++i) {
                if constexpr (D == 128) {
                    const uint32_t x = t & 2 ? w[h][i ^ 2] : w[h][i];
                    const int word = t & 2 ? i ^ 2 : i;
                    const __half2 s = word < 2 ? __low2half2(sc) : __high2half2(sc);
                    *reinterpret_cast<uint4 *>(row + ((((t & 1) * 4 + word) ^ g) << 4)) = unpack8(x, s);
                } else {
                    *reinterpret_cast<uint4 *>(row + (((2 * t + i) ^ g) << 4)) = unpack8(w[h][i], h ? __high2half2(sc) : __low2half2(sc));
                }
            }
        }
    }
    // V: tokens 2 t and 2 t + 1 of each half block, an eighth of the columns. Tokens
    // at or past `end` become zero, and those whose scale is no number, which are noted.
    __device__ __forceinline__ void put_v(uint8_t *to, int end, int key0, int *first_nan, int lane) {
        const int g = lane >> 2, t = lane & 3;
        constexpr int kGrp = Smem<D>::kGrp;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tok = 8 * (i >> 1) + 2 * t + (i & 1);
            const bool nan = (scales >> (8 * i) & 0x7fu) == 0x7fu;
            if (nan && tok < end) atomicMin(first_nan + (D == 128 ? g : g >> 1), key0 + tok);
            if (nan || tok >= end) scales &= ~(0xffu << (8 * i));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const __half2 sc = kv4_scales(scales >> (16 * h));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 2 * t + e;
                const __half2 s = e ? __high2half2(sc) : __low2half2(sc);
                if constexpr (D == 128) {
                    uint8_t *line = to + h * kGrp + (g >> 2) * 1024 + row * 128;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t x = g & 1 ? w[h][2 * e + (i ^ 1)] : w[h][2 * e + i];
                        const int word = g & 1 ? i ^ 1 : i;
                        *reinterpret_cast<uint4 *>(line + ((((g & 3) * 2 + word) ^ row) << 4)) = unpack8(x, s);
                    }
                } else {
                    *reinterpret_cast<uint4 *>(to + h * kGrp + row * 128 + ((g ^ row) << 4)) = unpack8(w[h][e], s);
                }
            }
        }
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2) kv4_chunk_kernel(const Kv4Args a) {
    using S = Smem<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ long long s_units[kThreads / 32];
    __shared__ int s_items[kThreads], s_sum[kThreads / 32], s_most[kThreads / 32];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_claim;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *s_x = reinterpret_cast<float *>(smem + S::kX), *s_mul = reinterpret_cast<float *>(smem + S::kMul);
    int *s_nan = reinterpret_cast<int *>(smem + S::kNan);
    uint64_t *bar_s = reinterpret_cast<uint64_t *>(smem + S::kBar), *bar_pv = bar_s + 1;
    volatile int *abort = &s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (tid == 0) {
        s_abort = 0;
        mbar_init(bar_s, 1);
        mbar_init(bar_pv, 1);
        mbar_fence_init();
    }
    pdl_launch_dependents();
    pdl_wait();

    // Which requests are this kernel's, and how many items they have.
    const int each = (a.num_reqs + kThreads - 1) / kThreads;
    int items = 0, most = 0;
    long long units = 0;
    {
        int bits = 0;  // the other kernel reports them
        for (int r = tid * each; r < min((tid + 1) * each, a.num_reqs); ++r) {
            const Kv4Request q = kv4_request_of(a, r, kKv4ChunkRows, &bits);
            if (!kv4_is_chunk(q, a.group)) continue;
            items += q.tiles * a.num_kv_heads;
            units += kv4_chunk_units(q, a.num_kv_heads);
            most = max(most, kv4_chunk_tiles(q.len));
        }
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
    if (!kv4_use_chunks(units, most) || (int)blockIdx.x >= total) return;  // the items go by `total` claims and no more CTAs
    const int ctas = min((int)gridDim.x, total);
    if (warp == 0) tmem_alloc(&s_tmem, kTmemCols);
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tm = s_tmem;

    constexpr uint32_t kIdS = idesc_f16(128, kKeys, 0), kIdPv = idesc_f16(128, D, 1);
    const uint32_t q_s = smem_u32(smem + S::kQ), k_s = smem_u32(smem + S::kK), v_s = smem_u32(smem + S::kV);
    const int part = warp >> 2, row = (warp & 3) * 32 + lane;  // this thread's keys (of 64) and row in the softmax
    const uint32_t tm_row = tm + ((uint32_t)((warp & 3) * 32) << 16);
    uint32_t phase = 0;  // of both barriers: they complete once a key tile
    const long long block_bytes = (long long)a.num_kv_heads * Kv4Tile<D>::kBytes;

    for (int item = blockIdx.x; item < total;) {
        // the next item is claimed now, and looked at when this one is done
        if (tid == 0) {
            const int seen = atomicAdd(a.claimed, 1) - kKv4Nobody;
            // CTA b has item b without a claim; all claim until one is past the end, and the last of those
            // leaves the counter as it was
            if (seen == total - 1) atomicExch(a.claimed, kKv4Nobody);
            if (seen < 0 || seen >= total) raise_status(a.status, PKV_DEV_BAD_WORKSPACE);
            s_claim = seen < 0 || seen >= total ? total : ctas + seen;
        }
        // the item: request, tile and head
        Kv4Request q;
        int r, i, h;
        {
            int lo = 0, hi = kThreads - 1;  // the first thread with s_items > item
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (s_items[mid] > item) hi = mid; else lo = mid + 1;
            }
            int off = item - (lo ? s_items[lo - 1] : 0), none = 0;
            for (r = lo * each;; ++r) {
                q = kv4_request_of(a, r, kKv4ChunkRows, &none);
                const int have = kv4_is_chunk(q, a.group) ? q.tiles * a.num_kv_heads : 0;
                if (off < have) break;
                off -= have;
            }
            // longest tiles of a request first
            i = q.tiles - 1 - off / a.num_kv_heads;
            h = off % a.num_kv_heads;
        }
        const Kv4Tiling tl = kv4_tile(q, i, a.group, kKv4ChunkRows);
        const int nt = (tl.keys + kKeys - 1) / kKeys;
        const int row0 = i * kKv4ChunkRows;
        const int32_t *ids = a.table + (long long)r * a.max_blocks;
        const uint8_t *heads = a.pool + (long long)h * Kv4Tile<D>::kBytes;
        int bits = 0;
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
        const int id0 = id_of(0);
        int id1 = id_of(1);
        Raw<D> rk, rv;
        const uint8_t *at = tile_of(0, id0);
        rk.load(at, false, lane);
        rv.load(at, true, lane);

        // q: two threads a row, fp16 scaled by a power of two to lie in (-4, 4)
        {
            const int qr = tid >> 1, half = tid & 1, rr = row0 + qr, tok = rr / a.group;
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
            e = e == 255 ? 127 : min(max(e, 64), 253);
            const float down = __uint_as_float((uint32_t)(254 - e) << 23), up = __uint_as_float((uint32_t)e << 23);
            if (half == 0) s_mul[qr] = qr < tl.rows ? up * a.scale_log2 : 0.0f;
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
        uint8_t *k_to = smem + S::kK + warp * 2 * S::kGrp, *v_to = smem + S::kV + warp * 2 * S::kGrp;
        rk.put_k(k_to, lane);
        rk.load(tile_of(1, id1), false, lane);
        fence_proxy_async_smem();
        __syncthreads();
        // keys that this row sees (padding rows: one)
        const int rr = row0 + row;
        const int limit = row < tl.rows ? q.len - q.n + rr / a.group + 1 : 1;
        const float mul = s_mul[row];
        float m = -INFINITY, l = 0.0f;

        for (int j = 0; j < nt; ++j) {
            if (warp == 0) {
                tmem_fence_after_sync();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_bf16_warp(tm, umma_desc_sw128(q_s + (kk / 4) * S::kHalf + (kk % 4) * 32, 16, 1024),
                                   umma_desc_sw128(k_s + (kk / 4) * 1024 + (kk % 4) * 32, 16, S::kGrp), kIdS, kk > 0 ? 1u : 0u);
                umma_commit_warp(bar_s);
            }
            const int key0 = j * kKeys;
            rv.put_v(v_to, tl.keys - key0 - 16 * warp, key0 + 16 * warp, s_nan, lane);
            rv.load(tile_of(j + 1, id1), true, lane);
            id1 = id_of(j + 2);
            fence_proxy_async_smem();

            warp_wait(bar_s, phase, abort);
            tmem_fence_after_sync();
            float s[64];
            tmem_ld32(tm_row + part * 64, *reinterpret_cast<float(*)[32]>(s));
            tmem_ld32(tm_row + part * 64 + 32, *reinterpret_cast<float(*)[32]>(s + 32));
            tmem_wait_ld_regs(*reinterpret_cast<float(*)[32]>(s));
            tmem_wait_ld_regs(*reinterpret_cast<float(*)[32]>(s + 32));
            const int mine = limit - key0 - part * 64;  // of these keys, the row sees so many
            if (!__all_sync(0xffffffffu, mine >= 64)) {
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    if (e >= mine) s[e] = -INFINITY;
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 32; ++e) top[e & 3] = fmax3(top[e & 3], s[2 * e], s[2 * e + 1]);
            s_x[part * 128 + row] = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            // both halves of these rows have their scores in registers now: P may go over them
            tmem_fence_before_sync();
            named_barrier_sync(1 + (warp & 3), 64);
            tmem_fence_after_sync();
            const float best = fmaxf(s_x[row], s_x[128 + row]);
            // the reference moves when a score passes it by 2^10: p fits fp16 until then
            const bool moves = j == 0 || (best - m) * mul > 10.0f;
            if (__any_sync(0xffffffffu, moves)) {
                const float to = moves ? fmaxf(m, best) : m;
                const float f = m == to ? 1.0f : m == -INFINITY ? 0.0f : fast_exp2((m - to) * mul);
                m = to;
                l *= f;
                if (j > 0) {
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        float o[32];
                        const uint32_t at_o = tm_row + kColO + part * (D / 2) + 32 * c;
                        tmem_ld32(at_o, o);
                        tmem_wait_ld_regs(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= f;
                        tmem_st32(at_o, o);
                    }
                }
            }
            const float2 nm = make_float2(-m, -m), mm = make_float2(mul, mul);
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t p[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 x = fmul2(fadd2(make_float2(s[32 * c + 2 * e], s[32 * c + 2 * e + 1]), nm), mm);
                    const float2 y = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                    sum = fadd2(sum, y);
                    p[e] = half_bits(__floats2half2_rn(y.x, y.y));
                }
                tmem_st16u(tm_row + part * 32 + 16 * c, p);
            }
            l += sum.x + sum.y;
            tmem_wait_st();
            tmem_fence_before_sync();
            __syncthreads();
            if (warp == 0) {
                tmem_fence_after_sync();
#pragma unroll
                for (int kk = 0; kk < kKeys / 16; ++kk)
                    umma_bf16_tmem_a_warp(tm + kColO, tm + kk * 8, umma_desc_sw128(v_s + kk * 2 * S::kGrp, 1024, S::kGrp), kIdPv,
                                          (j > 0 || kk > 0) ? 1u : 0u);
                umma_commit_warp(bar_pv);
            }
            if (j + 1 < nt) {
                rk.put_k(k_to, lane);
                rk.load(tile_of(j + 2, id1), false, lane);
                fence_proxy_async_smem();
            }
            warp_wait(bar_pv, phase, abort);
            phase ^= 1;
            __syncthreads();
            if (*abort) break;
        }
        if (*abort) break;
        tmem_fence_after_sync();
        s_x[part * 128 + row] = l;
        named_barrier_sync(1 + (warp & 3), 64);
        const float f = a.v_scale / (s_x[row] + s_x[128 + row]);
        const int tok = rr / a.group;
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
        item = s_claim;
        __syncthreads();
        tmem_fence_after_sync();
    }
    if (*abort && tid == 0) raise_status(a.status, PKV_DEV_TIMEOUT);
    __syncthreads();
    if (warp == 0) tmem_dealloc(tm, kTmemCols);
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
    return launch_pdl(kv4_chunk_kernel<D>, dim3(2 * sms), dim3(kThreads), Smem<D>::kAlloc, st, a) == cudaSuccess ? PKV_OK : PKV_E_CUDA;
}

}  // namespace

int kv4_chunk_launch(const Kv4Args &a, int head_size, int sms, cudaStream_t stream) {
    return head_size == 128 ? launch<128>(a, sms, stream) : launch<64>(a, sms, stream);
}

}  // namespace pkv
