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

// Eight values of a group (the other eight are in the neighbouring lane) as
// codes; *scale: the group's scale byte.
__device__ __forceinline__ uint32_t quantise(uint4 x, float inv, uint32_t *scale) {
    uint32_t top = max_bits(x);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const float want = fmaxf(__uint_as_float(top << 16) * inv / 6.0f, 0x1p-9f);
    uint16_t byte;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;" : "=h"(byte) : "f"(want));
    if (top > 0x7f80u) byte = 0x7f;  // a NaN among them: the whole group is one
    *scale = byte & 0xffu;
    const float s = __low2float(kv4_scales(byte));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = __uint_as_float(w[i] << 16) * inv, hi = __uint_as_float(w[i] & 0xffff0000u) * inv;
        codes |= codes2(lo / s, hi / s) << (8 * i);
    }
    return codes;
}

// A warp per token: K chunks (8 columns of one head each), then V chunks.
template <int D>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const StoreArgs a) {
    using Tile = Kv4Tile<D>;
    constexpr int kC = D / 8;  // chunks of a head
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int chunks = a.num_kv_heads * kC;  // a multiple of 8, so the two lanes of a group stay together
    for (long long t = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5; t < a.num_tokens;
         t += (long long)gridDim.x * kThreads / 32) {
        const int slot = __ldg(a.slots + t);
        if (slot < 0) continue;
        const int blk = slot / PKV_BLOCK_SIZE, row = slot % PKV_BLOCK_SIZE;
        if (blk >= a.num_blocks) {
            if (lane == 0) raise_status(a.status, PKV_DEV_BAD_SLOT);
            continue;
        }
        uint8_t *tiles = a.pool + (long long)blk * a.num_kv_heads * Tile::kBytes;
        for (int i0 = 0; i0 < 2 * chunks; i0 += 128) {
            uint4 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + 32 * j + lane;
                if (i < 2 * chunks)
                    x[j] = i < chunks ? __ldg(a.k + t * a.k_stride + i) : __ldg(a.v + t * a.v_stride + (i - chunks));
                else
                    x[j] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (i0 + 32 * j >= 2 * chunks) break;
                const int i = i0 + 32 * j + lane;
                const bool is_v = i >= chunks;
                uint32_t scale;
                const uint32_t codes = quantise(x[j], is_v ? a.v_inv : a.k_inv, &scale);
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
    return launch_pdl(kernel, dim3(grid_for(num_tokens)), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a) ==
                   cudaSuccess
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
