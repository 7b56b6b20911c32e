// K and V of new tokens into the 4-bit pool, and tokens of the pool back as bf16.
//
// A group of 16 columns with largest magnitude A gets the scale s = A / 6 in
// e4m3 (at least 2^-9, at most 448), a value x the e2m1 code nearest to x / s.
// Both roundings are exact, ties to even: A has 8 significant bits and a tie
// between scales times 6 at most 7, so the 32-bit quotient never crosses one it
// does not hit; the same holds for x against a tie between codes times s.
//
// Bound by, and measured (one GB300, tokens of 8 heads of 128, floor at 6685 GB/s):
// 32768 tokens written in 34 us and read back in 29 (together 63.4 in a graph,
// floor 45.8). The write moves 153 MB of DRAM bytes at 4.4 TB/s with 53 % of the issue
// slots and waits for its loads, of which 64 registers a thread hold two groups; the
// read 111 MB (the rest of its output stays in L2), 45 % of the issue slots. 2240
// tokens 7.3 us, floor 3.1; 64 tokens of 4 heads of 64 in 3.8: two launches and their
// first loads.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "kv4_format.cuh"
#include "pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct StoreArgs {
    const uint4 *k, *v;
    long long k_stride, v_stride;  // 16-byte chunks from token to token
    const int32_t *slots;
    int num_tokens, num_kv_heads, num_blocks;
    uint8_t *pool;
    float k_scale, v_scale, k_inv, v_inv;
    int32_t *status;
};

struct Group {
    uint4 x, y;  // 16 bf16 values
};

// The largest magnitude of a group as its bits (NaN above infinity above all others).
__device__ __forceinline__ uint32_t max_bits(const Group &g) {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t a = __vmaxu2(__vmaxu2(g.x.x & m, g.x.y & m), __vmaxu2(g.x.z & m, g.x.w & m));
    const uint32_t b = __vmaxu2(__vmaxu2(g.y.x & m, g.y.y & m), __vmaxu2(g.y.z & m, g.y.w & m));
    const uint32_t c = __vmaxu2(a, b);
    return max(c & 0xffffu, c >> 16);
}

__device__ __forceinline__ uint32_t codes8(float2 a, float2 b, float2 c, float2 d) {
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
    return w;
}

__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A group as 16 codes and its scale byte. Quotients x / (s * by) are x * (1 / (s *
// by)), the reciprocal to about 2^-23, corrected once by their remainder (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000", 1990), which one
// fused operation gives exactly: what is left is off by 2^-46, so that a tie (x a
// border between codes times s) comes out as that border itself, and everything
// else is 2^-8 away from one. Quotients are 8 at most. (The correction makes +0 of -0:
// code 0 for both.)
__device__ __forceinline__ uint2 quantise(const Group &g, float by, float inv, uint32_t *scale) {
    const uint32_t top = max_bits(g);
    const float most = fminf(__uint_as_float(top << 16) * inv, 3e38f);
    constexpr float kSixth = 1.0f / 6.0f;
    const float q6 = most * kSixth, want = fmaxf(fmaf(fmaf(q6, -6.0f, most), kSixth, q6), 0x1p-9f);
    uint16_t byte;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;" : "=h"(byte) : "f"(want));
    if (top > 0x7f80u) byte = 0x7f;  // a NaN among them: the whole group is one
    *scale = byte & 0xffu;
    const float s = __low2float(kv4_scales(byte)), r = reciprocal(s) * inv, sb = -s * by;
    const uint32_t w[8] = {g.x.x, g.x.y, g.x.z, g.x.w, g.y.x, g.y.y, g.y.z, g.y.w};
    float2 y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    if (byte == 0x7e7e) {
        // The largest scale (both halves hold it): values past its codes, infinite ones too,
        // become 8 times it, which is the largest code with their sign. Further out the quotient
        // would overflow where by is small, and its remainder be an infinity of the other sign.
        const float bound = 8.0f * s * by;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = make_float2(fminf(fmaxf(y[i].x, -bound), bound), fminf(fmaxf(y[i].y, -bound), bound));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 q = fmul2(y[i], make_float2(r, r));
        const float2 rem = ffma2(q, make_float2(sb, sb), y[i]);
        y[i] = ffma2(rem, make_float2(r, r), q);
    }
    return make_uint2(codes8(y[0], y[1], y[2], y[3]), codes8(y[4], y[5], y[6], y[7]));
}

// Group g's codes of a token: 8 bytes, or two times 4 a row of D / 2 bytes apart
// (V, D 64).
template <int D>
__device__ __forceinline__ void put_codes(uint8_t *tile, bool is_v, int row, int g, uint2 codes) {
    using Tile = Kv4Tile<D>;
    uint8_t *to = tile + (is_v ? Tile::v_code(row, 2 * g) : Tile::k_code(row, 2 * g));
    if (D == 64) {
        *reinterpret_cast<uint32_t *>(to) = codes.x;
        *reinterpret_cast<uint32_t *>(to + (is_v ? D / 2 : 4)) = codes.y;
    } else {
        *reinterpret_cast<uint2 *>(to) = codes;
    }
}

// One head's K or V of a whole block, by one warp: rows as they come in, codes
// and scales to shared memory, from there to the tile in 16-byte chunks.
template <int D, bool kV>
__device__ __forceinline__ void write_tile(const uint4 *src, long long stride, float by, float inv, uint8_t *to, uint8_t *mem, int lane) {
    using Tile = Kv4Tile<D>;
    constexpr int kG = D / 16, kPer = 32 / kG, kLoads = 16 / kPer;  // groups of a row, rows at a time
    constexpr int kAhead = 2;
    const int g = lane % kG;
    __syncwarp();
#pragma unroll 1
    for (int j0 = 0; j0 < kLoads; j0 += kAhead) {
        Group x[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const uint4 *at = src + ((j0 + j) * kPer + lane / kG) * stride + 2 * g;
            x[j] = Group{__ldg(at), __ldg(at + 1)};
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int row = (j0 + j) * kPer + lane / kG;
            uint32_t scale;
            const uint2 codes = quantise(x[j], by, inv, &scale);
            // the part's codes, then its scales
            put_codes<D>(mem - (kV ? Tile::kV : 0), kV, row, g, codes);
            mem[8 * D + (kV ? Tile::v_scale(row, g) - Tile::kVScale : Tile::k_scale(row, g) - Tile::kKScale)] = (uint8_t)scale;
        }
    }
    __syncwarp();
    const uint4 *from = reinterpret_cast<const uint4 *>(mem);
    for (int i = lane; i < 9 * D / 16; i += 32)
        *reinterpret_cast<uint4 *>(to + (i < D / 2 ? (kV ? Tile::kV : 0) + 16 * i : (kV ? Tile::kVScale : Tile::kKScale) + 16 * (i - D / 2))) =
            from[i];
}

// One token's K and V of `heads` heads, by one warp: a lane per group.
template <int D>
__device__ __forceinline__ void write_token(const uint4 *k, const uint4 *v, int heads, const StoreArgs &a, uint8_t *tiles, int row, int lane) {
    using Tile = Kv4Tile<D>;
    constexpr int kG = D / 16, kAhead = 2;
    const int n = heads * kG;
    for (int i0 = lane; i0 < 2 * n; i0 += 32 * kAhead) {
        Group x[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = min(i0 + 32 * j, 2 * n - 1);
            const uint4 *at = i < n ? k + 2 * i : v + 2 * (i - n);
            x[j] = Group{__ldg(at), __ldg(at + 1)};
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + 32 * j;
            if (i >= 2 * n) break;
            const bool is_v = i >= n;
            const int ii = is_v ? i - n : i, g = ii % kG;
            uint32_t scale;
            const uint2 codes = quantise(x[j], is_v ? a.v_scale : a.k_scale, is_v ? a.v_inv : a.k_inv, &scale);
            uint8_t *tile = tiles + (long long)(ii / kG) * Tile::kBytes;
            put_codes<D>(tile, is_v, row, g, codes);
            tile[is_v ? Tile::v_scale(row, g) : Tile::k_scale(row, g)] = (uint8_t)scale;
        }
    }
}

// A CTA has 16 tokens, and the block that starts among them if a run of tokens
// fills it: such blocks (prompts) are turned into whole tiles, other tokens (decode
// rows, a prompt's ends) are written code by code. Every warp finds that out for
// itself from the slots around. Tiles go through shared memory because their codes
// and scales have the lanes' order: stores of 16 bytes instead of 8 and 1 (32768
// tokens written and read back 86 us against 92), found from registers instead of
// by counting in shared memory (67.7 against 82.7).
template <int D>
__global__ void __launch_bounds__(kThreads, 4) kv4_write_kernel(const StoreArgs a) {
    using Tile = Kv4Tile<D>;
    __shared__ __align__(16) uint8_t s_tile[kWarps][9 * D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = (int)blockIdx.x * PKV_BLOCK_SIZE;
    // this CTA's heads: where tokens are few, several CTAs share theirs
    const int per = (a.num_kv_heads + (int)gridDim.y - 1) / (int)gridDim.y;
    const int h0 = (int)blockIdx.y * per, heads = min(per, a.num_kv_heads - h0);
    pdl_launch_dependents();
    pdl_wait();
    if (heads <= 0) return;
    // slots of the 16 tokens before (lane 16 is the CTA's first token), and of the 16 behind
    auto slot_of = [&](int t) { return t >= 0 && t < a.num_tokens ? __ldg(a.slots + t) : -1; };
    const int one = slot_of(t0 - 16 + lane), two = slot_of(t0 + 16 + lane);
    // bit i: the token at t0 - 16 + i has the slot after its predecessor's, in the same block
    const int before1 = __shfl_up_sync(0xffffffffu, one, 1), last = __shfl_sync(0xffffffffu, one, 31);
    const int before2 = __shfl_up_sync(0xffffffffu, two, 1);
    const uint32_t run1 = __ballot_sync(0xffffffffu, lane > 0 && one > 0 && (one & 15) && one - 1 == before1);
    const uint32_t run2 = __ballot_sync(0xffffffffu, two > 0 && (two & 15) && two - 1 == (lane ? before2 : last));
    const uint64_t run = run1 | (uint64_t)run2 << 32;
    // the CTA's tokens (lane 16 on) that belong to a whole block's run
    const int row1 = one & 15;
    const bool in_full = lane >= 16 && one >= 0 && one / PKV_BLOCK_SIZE < a.num_blocks && (run >> (lane - row1 + 1) & 0x7fff) == 0x7fff;
    const uint32_t full = __ballot_sync(0xffffffffu, in_full) >> 16;
    const uint32_t begin = __ballot_sync(0xffffffffu, in_full && row1 == 0) >> 16;
    if (begin) {  // at most one: a run of 16 has one token in row 0
        const int first = __ffs(begin) - 1;
        const int blk = __shfl_sync(0xffffffffu, one, 16 + first) / PKV_BLOCK_SIZE;
        uint8_t *tiles = a.pool + (long long)blk * a.num_kv_heads * Tile::kBytes;
        for (int task = warp; task < 2 * heads; task += kWarps) {
            const int h = h0 + (task >> 1);
            uint8_t *to = tiles + (long long)h * Tile::kBytes;
            if (task & 1)
                write_tile<D, true>(a.v + (t0 + first) * a.v_stride + h * (D / 8), a.v_stride, a.v_scale, a.v_inv, to, s_tile[warp], lane);
            else
                write_tile<D, false>(a.k + (t0 + first) * a.k_stride + h * (D / 8), a.k_stride, a.k_scale, a.k_inv, to, s_tile[warp], lane);
        }
    }
    for (int j = warp; j < 16; j += kWarps) {
        const int slot = __shfl_sync(0xffffffffu, one, 16 + j);
        if (slot < 0 || (full >> j & 1)) continue;
        const int blk = slot / PKV_BLOCK_SIZE, row = slot % PKV_BLOCK_SIZE;
        if (blk >= a.num_blocks) {
            if (lane == 0) raise_status(a.status, PKV_DEV_BAD_SLOT);
            continue;
        }
        const long long t = t0 + j;
        uint8_t *tiles = a.pool + ((long long)blk * a.num_kv_heads + h0) * Tile::kBytes;
        write_token<D>(a.k + t * a.k_stride + h0 * (D / 8), a.v + t * a.v_stride + h0 * (D / 8), heads, a, tiles, row, lane);
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

// Of one token's K or V, what a lane reads: the same 8 columns of every so many
// heads, whose places are a constant apart.
template <int D>
struct Part {
    static constexpr int kC = D / 8, kStep = 32 / kC * Kv4Tile<D>::kBytes;  // 32 lanes have 32 / kC heads
    const uint8_t *at, *at_scale;
    float by;
    uint4 *to;
    uint32_t codes[2], byte[2];

    __device__ __forceinline__ void load(int i0, int n) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (i0 + 32 * j >= n) break;
            codes[j] = *reinterpret_cast<const uint32_t *>(at + j * kStep);
            byte[j] = at_scale[j * kStep];
        }
        at += 2 * kStep;
        at_scale += 2 * kStep;
    }
    __device__ __forceinline__ void store(int i0, int n) const {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (i0 + 32 * j >= n) break;
            const float s = __low2float(kv4_scales(byte[j])) * by;
            auto pair = [&](__half2 x) {
                const float2 f = fmul2(__half22float2(x), make_float2(s, s));
                return pack_bf16x2(f.x, f.y);
            };
            to[i0 + 32 * j] = make_uint4(pair(kv4_pair<0>(codes[j])), pair(kv4_pair<1>(codes[j])), pair(kv4_pair<2>(codes[j])), pair(kv4_pair<3>(codes[j])));
        }
    }
};

// A warp per token; two pieces of K and of V of a lane on their way at a time.
template <int D>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const LoadArgs a) {
    using Tile = Kv4Tile<D>;
    constexpr int kC = D / 8;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long t = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int per = (a.num_kv_heads + (int)gridDim.y - 1) / (int)gridDim.y;
    const int h0 = (int)blockIdx.y * per, n = min(per, a.num_kv_heads - h0) * kC;
    if (t >= a.num_tokens || n <= 0) return;
    const int slot = __ldg(a.slots + t);
    if (slot < 0) return;
    const int blk = slot / PKV_BLOCK_SIZE, row = slot % PKV_BLOCK_SIZE;
    if (blk >= a.num_blocks) {
        if (lane == 0) raise_status(a.status, PKV_DEV_BAD_SLOT);
        return;
    }
    const uint8_t *tiles = a.pool + ((long long)blk * a.num_kv_heads + h0) * Tile::kBytes;
    const long long at = (t * a.num_kv_heads + h0) * kC;
    const int c = lane % kC;
    const uint8_t *tile = tiles + lane / kC * Tile::kBytes;
    Part<D> k{tile + Tile::k_code(row, c), tile + Tile::k_scale(row, c >> 1), a.k_scale, a.k + at};
    Part<D> v{tile + Tile::v_code(row, c), tile + Tile::v_scale(row, c >> 1), a.v_scale, a.v + at};
    for (int i0 = lane; i0 < n; i0 += 64) {
        if (a.k) k.load(i0, n);
        if (a.v) v.load(i0, n);
        if (a.k) k.store(i0, n);
        if (a.v) v.store(i0, n);
    }
}

int check_common(const void *pool, const pkv_cache_desc *desc, const int32_t *slots, int32_t num_tokens,
                 const int32_t *status, float k_scale, float v_scale) {
    if (!desc) return PKV_E_NULL;
    const int rc = check_cache_desc(*desc, /*attention=*/true);
    if (rc) return rc;
    if (num_tokens < 0 || num_tokens > INT32_MAX - 65536 || !kv4_scale_ok(k_scale) || !kv4_scale_ok(v_scale)) return PKV_E_DIMS;
    if (num_tokens == 0) return PKV_OK;
    if (!pool || !slots) return PKV_E_NULL;
    if (!aligned(pool, 16) || !aligned(slots, 4) || !aligned(status, 4)) return PKV_E_ALIGN;
    return PKV_OK;
}

// CTAs of so many tokens, and of a part of the heads where those leave SMs without
// four; between 8 of them and half as many as SMs a part has the work of a warp at
// least (32 groups of K and V). Written and read back, us, heads not shared / shared
// as far as that / to the last one: 16 tokens of 8 heads of 128 6.9 / 4.2 / 4.1, 200
// 7.1 / 4.8 / 5.4, 2240 15.5 / 11.3 / 11.2; 64 tokens of 4 heads of 64 4.1 / 4.1 / 3.9,
// 512 4.3 / 4.3 / 5.7, 2240 of whole blocks 5.4 / 5.3 / 4.8.
int grid_for(int num_tokens, int tokens, int heads, int head_size, dim3 *grid) {
    int sms = 0;
    const int rc = device_sms(&sms);
    if (rc) return rc;
    const unsigned x = ((unsigned)num_tokens + tokens - 1) / tokens;
    const unsigned most = x >= 8 && x < (unsigned)sms / 2 ? std::max(1, heads * head_size / 256) : heads;
    *grid = dim3(x, std::min(most, std::max(1u, 4u * sms / x)));
    return PKV_OK;
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
                      static_cast<uint8_t *>(kv4_cache), k_scale, v_scale, 1.0f / k_scale, 1.0f / v_scale, status};
    const auto kernel = desc->head_size == 128 ? kv4_write_kernel<128> : kv4_write_kernel<64>;
    dim3 grid;
    const int rg = grid_for(num_tokens, PKV_BLOCK_SIZE, desc->num_kv_heads, desc->head_size, &grid);
    if (rg) return rg;
    return launch_pdl(kernel, grid, dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a) ==
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
    if (k_out == v_out) return PKV_E_DIMS;
    if (!aligned(k_out, 16) || !aligned(v_out, 16)) return PKV_E_ALIGN;
    const LoadArgs a{static_cast<const uint8_t *>(kv4_cache), slot_mapping, num_tokens, desc->num_kv_heads,
                     desc->num_blocks, k_scale, v_scale, static_cast<uint4 *>(k_out), static_cast<uint4 *>(v_out),
                     status};
    const auto kernel = desc->head_size == 128 ? kv4_read_kernel<128> : kv4_read_kernel<64>;
    dim3 grid;
    const int rg = grid_for(num_tokens, kWarps, desc->num_kv_heads, desc->head_size, &grid);
    if (rg) return rg;
    return launch_pdl(kernel, grid, dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a) ==
                   cudaSuccess
               ? PKV_OK
               : PKV_E_CUDA;
}
