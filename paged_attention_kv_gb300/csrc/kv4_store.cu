// K and V of new tokens into the 4-bit pool, and tokens of the pool back as bf16.
//
// A group of 16 columns with largest magnitude A gets the scale s = A / 6 in
// e4m3 (at least 2^-9, at most 448), a value x the e2m1 code nearest to x / s.
// Both roundings are exact, ties to even: A has 8 significant bits and a tie
// between scales times 6 at most 7, so the 32-bit quotient never crosses one it
// does not hit; the same holds for x against a tie between codes times s.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "kv4_format.cuh"
#include "pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;

struct StoreArgs {
    const uint4 *k, *v;
    long long k_stride, v_stride;  // 16-byte chunks from token to token
    const int32_t *slots;
    int num_tokens, num_kv_heads, num_blocks;
    uint8_t *pool;
    float k_inv, v_inv;
    int32_t *status;
};

// The largest magnitude of 8 bf16 values as its bits (NaN above infinity above
// all others).
__device__ __forceinline__ uint32_t max_bits(uint4 x) {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t a = __vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m));
    return max(a & 0xffffu, a >> 16);
}

__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
    uint32_t c;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(c) : "f"(lo), "f"(hi));
    return c;
}

__device__ __forceinline__ float with_sign(float y, float x) {
    return __uint_as_float(__float_as_uint(y) | (__float_as_uint(x) & 0x80000000u));
}

// Eight values of a group (the other eight are in the neighbouring lane) as
// codes; *scale: the group's scale byte. A quotient is x / s as x * (1 / s),
// corrected once by its remainder, which one fused operation gives exactly: a tie
// (x a code's border times s) comes out as that border itself, which the
// reciprocal's own rounding would miss, and everything else is 2^-8 away from one.
__device__ __forceinline__ uint32_t quantise(uint4 x, float inv, uint32_t *scale) {
    uint32_t top = max_bits(x);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const float most = __uint_as_float(top << 16) * inv;
    const float want = fmaxf(most / 6.0f, 0x1p-9f);
    uint16_t byte;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;" : "=h"(byte) : "f"(want));
    if (top > 0x7f80u) byte = 0x7f;  // a NaN among them: the whole group is one
    *scale = byte & 0xffu;
    const float s = __low2float(kv4_scales(byte)), r = 1.0f / s;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = fmul2(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)), make_float2(inv, inv));
    if (isinf(most)) {  // an infinity has no remainder; the largest finite value becomes the same code
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = make_float2(fminf(fmaxf(v[i].x, -3e38f), 3e38f), fminf(fmaxf(v[i].y, -3e38f), 3e38f));
    }
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 q = fmul2(v[i], make_float2(r, r));
        const float2 rem = ffma2(make_float2(-q.x, -q.y), make_float2(s, s), v[i]);
        const float2 y = ffma2(rem, make_float2(r, r), q);
        // the correction makes +0 of -0
        codes |= codes2(with_sign(y.x, v[i].x), with_sign(y.y, v[i].y)) << (8 * i);
    }
    return codes;
}

// A CTA has 16 tokens, and the block that starts among them if a run of tokens
// fills it: those (prompts) are turned into whole tiles, one warp a head's K or V,
// and leave as 16-byte chunks; other tokens (decode rows, a prompt's ends) are
// written code by code, a warp each. 32768 tokens of 8 heads of 128: see below.
constexpr int kWriteThreads = 512;

template <int D>
__global__ void __launch_bounds__(kWriteThreads, 2) kv4_write_kernel(const StoreArgs a) {
    using Tile = Kv4Tile<D>;
    constexpr int kC = D / 8;             // chunks of 8 columns of a head
    constexpr int kWarps = kWriteThreads / 32;
    constexpr int kLoads = kC / 2;        // of a warp for one head's K or V of 16 tokens
    constexpr int kPer = 32 / kC;         // tokens a load covers
    __shared__ int s_slot[48];
    __shared__ uint32_t s_full;
    __shared__ __align__(16) uint8_t s_tile[kWarps][9 * D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = (int)blockIdx.x * PKV_BLOCK_SIZE;
    pdl_launch_dependents();
    pdl_wait();
    if (tid < 48) {
        const int t = t0 - 15 + tid;
        s_slot[tid] = t >= 0 && t < a.num_tokens ? __ldg(a.slots + t) : -1;
    }
    __syncthreads();
    if (warp == 0) {
        bool full = false;
        if (lane < 16) {
            const int slot = s_slot[15 + lane], row = slot & 15;
            full = slot >= 0 && slot / PKV_BLOCK_SIZE < a.num_blocks;
            for (int i = 0; i < 16; ++i) full &= s_slot[15 + lane - row + i] == slot - row + i;
        }
        const uint32_t all = __ballot_sync(0xffffffffu, full);
        if (lane == 0) s_full = all;
    }
    __syncthreads();
    const uint32_t full = s_full;
    int first = -1;  // the token that a whole block starts at
    for (int j = 0; j < 16; ++j)
        if ((full >> j & 1) && (s_slot[15 + j] & 15) == 0) first = j;
    if (first >= 0) {
        uint8_t *tiles = a.pool + (long long)(s_slot[15 + first] / PKV_BLOCK_SIZE) * a.num_kv_heads * Tile::kBytes;
        const int c = lane % kC;
        for (int task = warp; task < 2 * a.num_kv_heads; task += kWarps) {
            const int h = task >> 1;
            const bool is_v = task & 1;
            const uint4 *src = (is_v ? a.v + (t0 + first) * a.v_stride : a.k + (t0 + first) * a.k_stride) + h * kC + c;
            const long long stride = is_v ? a.v_stride : a.k_stride;
            uint4 x[kLoads];
#pragma unroll
            for (int j = 0; j < kLoads; ++j) x[j] = __ldg(src + (j * kPer + lane / kC) * stride);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int row = j * kPer + lane / kC;
                uint32_t scale;
                const uint32_t codes = quantise(x[j], is_v ? a.v_inv : a.k_inv, &scale);
                // as in the tile, the scales right behind the codes
                *reinterpret_cast<uint32_t *>(s_tile[warp] + (is_v ? Tile::v_code(row, c) - Tile::kV : Tile::k_code(row, c))) = codes;
                if ((c & 1) == 0)
                    s_tile[warp][8 * D + (is_v ? Tile::v_scale(row, c >> 1) - Tile::kVScale : Tile::k_scale(row, c >> 1) - Tile::kKScale)] =
                        (uint8_t)scale;
            }
            __syncwarp();
            uint8_t *to = tiles + (long long)h * Tile::kBytes;
            const uint4 *from = reinterpret_cast<const uint4 *>(s_tile[warp]);
            for (int i = lane; i < 9 * D / 16; i += 32)
                *reinterpret_cast<uint4 *>(to + (i < D / 2 ? (is_v ? Tile::kV : 0) + 16 * i
                                                            : (is_v ? Tile::kVScale : Tile::kKScale) + 16 * (i - D / 2))) = from[i];
        }
    }
    const int chunks = a.num_kv_heads * kC;  // a multiple of 8, so the two lanes of a group stay together
    for (int j = warp; j < 16; j += kWarps) {
        const int slot = s_slot[15 + j];
        if (slot < 0 || (full >> j & 1)) continue;
        const int blk = slot / PKV_BLOCK_SIZE, row = slot % PKV_BLOCK_SIZE;
        if (blk >= a.num_blocks) {
            if (lane == 0) raise_status(a.status, PKV_DEV_BAD_SLOT);
            continue;
        }
        const long long t = t0 + j;
        uint8_t *tiles = a.pool + (long long)blk * a.num_kv_heads * Tile::kBytes;
        for (int i0 = 0; i0 < 2 * chunks; i0 += 128) {
            uint4 x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + 32 * u + lane;
                if (i < 2 * chunks)
                    x[u] = i < chunks ? __ldg(a.k + t * a.k_stride + i) : __ldg(a.v + t * a.v_stride + (i - chunks));
                else
                    x[u] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (i0 + 32 * u >= 2 * chunks) break;
                const int i = i0 + 32 * u + lane;
                const bool is_v = i >= chunks;
                uint32_t scale;
                const uint32_t codes = quantise(x[u], is_v ? a.v_inv : a.k_inv, &scale);
                if (i >= 2 * chunks) continue;
                const int ii = is_v ? i - chunks : i;
                const int h = ii / kC, c = ii % kC;
                uint8_t *tile = tiles + (long long)h * Tile::kBytes;
                *reinterpret_cast<uint32_t *>(tile + (is_v ? Tile::v_code(row, c) : Tile::k_code(row, c))) = codes;
                if ((c & 1) == 0)
                    tile[is_v ? Tile::v_scale(row, c >> 1) : Tile::k_scale(row, c >> 1)] = (uint8_t)scale;
            }
        }
    }
}

struct LoadArgs {
    const uint8_t *pool;
    const int32_t *slots;
    int num_tokens, num_kv_heads, num_blocks;
    float k_scale, v_scale;
    uint4 *k, *v;
    int32_t *status;
};

__device__ __forceinline__ uint32_t to_bf16x2(__half2 x, float s) {
    const float2 f = __half22float2(x);
    return pack_bf16x2(f.x * s, f.y * s);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const LoadArgs a) {
    using Tile = Kv4Tile<D>;
    constexpr int kC = D / 8;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int chunks = a.num_kv_heads * kC;
    for (long long t = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5; t < a.num_tokens;
         t += (long long)gridDim.x * kThreads / 32) {
        const int slot = __ldg(a.slots + t);
        if (slot < 0) continue;
        const int blk = slot / PKV_BLOCK_SIZE, row = slot % PKV_BLOCK_SIZE;
        if (blk >= a.num_blocks) {
            if (lane == 0) raise_status(a.status, PKV_DEV_BAD_SLOT);
            continue;
        }
        const uint8_t *tiles = a.pool + (long long)blk * a.num_kv_heads * Tile::kBytes;
        for (int i0 = 0; i0 < 2 * chunks; i0 += 128) {
            uint32_t codes[4], scale[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + 32 * j + lane;
                if (i >= 2 * chunks) continue;
                const bool is_v = i >= chunks;
                const int ii = is_v ? i - chunks : i;
                const int h = ii / kC, c = ii % kC;
                const uint8_t *tile = tiles + (long long)h * Tile::kBytes;
                codes[j] = *reinterpret_cast<const uint32_t *>(tile + (is_v ? Tile::v_code(row, c) : Tile::k_code(row, c)));
                scale[j] = tile[is_v ? Tile::v_scale(row, c >> 1) : Tile::k_scale(row, c >> 1)];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + 32 * j + lane;
                if (i >= 2 * chunks) continue;
                const bool is_v = i >= chunks;
                uint4 *out = is_v ? a.v : a.k;
                if (!out) continue;
                const __half2 s = kv4_scales(scale[j] * 0x101u);
                const float by = is_v ? a.v_scale : a.k_scale;
                out[t * chunks + (is_v ? i - chunks : i)] =
                    make_uint4(to_bf16x2(__hmul2(kv4_pair<0>(codes[j]), s), by), to_bf16x2(__hmul2(kv4_pair<1>(codes[j]), s), by),
                               to_bf16x2(__hmul2(kv4_pair<2>(codes[j]), s), by), to_bf16x2(__hmul2(kv4_pair<3>(codes[j]), s), by));
            }
        }
    }
}

int check_common(const void *pool, const pkv_cache_desc *desc, const int32_t *slots, int32_t num_tokens,
                 const int32_t *status, float k_scale, float v_scale) {
    if (!desc) return PKV_E_NULL;
    const int rc = check_cache_desc(*desc, /*attention=*/true);
    if (rc) return rc;
    if (num_tokens < 0 || !kv4_scale_ok(k_scale) || !kv4_scale_ok(v_scale)) return PKV_E_DIMS;
    if (num_tokens == 0) return PKV_OK;
    if (!pool || !slots) return PKV_E_NULL;
    if (!aligned(pool, 16) || !aligned(slots, 4) || !aligned(status, 4)) return PKV_E_ALIGN;
    return PKV_OK;
}

int grid_for(int num_tokens) {
    return std::max(1, std::min((num_tokens + kThreads / 32 - 1) / (kThreads / 32), 1 << 20));
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" PKV_API int paged_kv4_cache_bytes(const pkv_cache_desc *desc, size_t *bytes) {
    if (!desc || !bytes) return PKV_E_NULL;
    const int rc = check_cache_desc(*desc, /*attention=*/true);
    if (rc) return rc;
    *bytes = (size_t)desc->num_blocks * desc->num_kv_heads * 18 * desc->head_size;
    return PKV_OK;
}

extern "C" PKV_API int paged_kv4_write(const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                       const int32_t *slot_mapping, int32_t num_tokens, void *kv4_cache,
                                       const pkv_cache_desc *desc, float k_scale, float v_scale, int32_t *status,
                                       void *stream) {
    const int rc = check_common(kv4_cache, desc, slot_mapping, num_tokens, status, k_scale, v_scale);
    if (rc || num_tokens == 0) return rc;
    if (!k || !v) return PKV_E_NULL;
    if (!aligned(k, 16) || !aligned(v, 16)) return PKV_E_ALIGN;
    const int64_t row = (int64_t)desc->num_kv_heads * desc->head_size;
    if (k_stride % 8 || v_stride % 8 || (num_tokens > 1 && (k_stride < row || v_stride < row)) || k_stride < 0 ||
        v_stride < 0)
        return PKV_E_DIMS;
    const StoreArgs a{static_cast<const uint4 *>(k), static_cast<const uint4 *>(v), k_stride / 8, v_stride / 8,
                      slot_mapping, num_tokens, desc->num_kv_heads, desc->num_blocks,
                      static_cast<uint8_t *>(kv4_cache), 1.0f / k_scale, 1.0f / v_scale, status};
    const auto kernel = desc->head_size == 128 ? kv4_write_kernel<128> : kv4_write_kernel<64>;
    return launch_pdl(kernel, dim3((unsigned)(((long long)num_tokens + 15) / 16)), dim3(kWriteThreads), 0,
                      static_cast<cudaStream_t>(stream), a) == cudaSuccess
               ? PKV_OK
               : PKV_E_CUDA;
}

extern "C" PKV_API int paged_kv4_read(const void *kv4_cache, const pkv_cache_desc *desc, const int32_t *slot_mapping,
                                      int32_t num_tokens, float k_scale, float v_scale, void *k_out, void *v_out,
                                      int32_t *status, void *stream) {
    const int rc = check_common(kv4_cache, desc, slot_mapping, num_tokens, status, k_scale, v_scale);
    if (rc || num_tokens == 0) return rc;
    if (!k_out && !v_out) return PKV_E_NULL;
    if (!aligned(k_out, 16) || !aligned(v_out, 16)) return PKV_E_ALIGN;
    const LoadArgs a{static_cast<const uint8_t *>(kv4_cache), slot_mapping, num_tokens, desc->num_kv_heads,
                     desc->num_blocks, k_scale, v_scale, static_cast<uint4 *>(k_out), static_cast<uint4 *>(v_out),
                     status};
    const auto kernel = desc->head_size == 128 ? kv4_read_kernel<128> : kv4_read_kernel<64>;
    return launch_pdl(kernel, dim3(grid_for(num_tokens)), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a) ==
                   cudaSuccess
               ? PKV_OK
               : PKV_E_CUDA;
}
