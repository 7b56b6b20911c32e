// What the two kernels of attention over the 4-bit pool share: kv4_attention.cu
// (any rows, a warp an item) and kv4_chunk.cu (requests with many rows).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kv4_plan.h"
#include "pagedkv.h"

namespace pkv {

// Counters between calls, so that a workspace that nobody prepared is noticed
// (every byte 0x5a).
constexpr int kKv4Nobody = 0x5a5a5a5a;

struct Kv4Args {
    const __nv_bfloat16 *q;
    long long q_stride;
    const uint8_t *pool;
    const int32_t *table, *lens, *qsl;
    int num_tokens, num_kv_heads, group, num_reqs, max_blocks, num_blocks;
    uint32_t group_inv;  // see kv4_over
    float scale_log2, small, v_scale;  // scale * log2(e) * k_scale is scale_log2 times small, a power of two
    __nv_bfloat16 *out;
    int *claimed;   // the workspace: items of kv4_chunk.cu taken so far;
    int *arrived;   // of each CTA, the arrivals for the item that begins there and ends in another
                    // (of each split item of kv4_chunk.cu, those of its parts);
    float4 *parts;  // and two partials: of the item that began before it, and of that one
    int chunks;     // kv4_chunk.cu runs too
    int32_t *status;
};

// x / d for x below 2^31, d at most 128 and inv = min(2^32 / d rounded up, 2^32 - 1):
// the product is off by less than 1. A third of a division's instructions.
inline uint32_t kv4_inverse(int d) { return d == 1 ? 0xffffffffu : (uint32_t)((0x100000000ull + d - 1) / d); }

#ifdef __CUDACC__
__device__ __forceinline__ int kv4_over(int x, int d, uint32_t inv) {
    int q = (int)__umulhi((uint32_t)x, inv);
    const int left = x - q * d;
    if (left < 0) --q;
    if (left >= d) ++q;
    return q;
}

// Request r's description, and the status bits of one that is skipped.
__device__ __forceinline__ Kv4Request kv4_request_of(const Kv4Args &a, int r, int rows, int *bits) {
    const int q0 = __ldg(a.qsl + r), q1 = __ldg(a.qsl + r + 1), len = __ldg(a.lens + r);
    int n = q1 - q0;
    if (q0 < 0 || n < 0 || q1 > a.num_tokens) {
        *bits |= PKV_DEV_BAD_QSL;
        n = 0;
    } else if (n > 0 && (len < n || len > (long long)a.max_blocks * PKV_BLOCK_SIZE)) {
        *bits |= PKV_DEV_BAD_LEN;
        n = 0;
    }
    return kv4_request(q0, n, len, a.group, rows);
}

// Whether the requests (`each` of them a thread) have more new tokens than there
// are: that takes bounds that descend somewhere, and their sums of items and costs
// might not fit their types. All of the CTA's threads call it; s: one each.
template <int kThreads>
__device__ __forceinline__ bool kv4_overlap(const Kv4Args &a, int each, long long *s) {
    long long n = 0;
    int none = 0;
    for (int r = threadIdx.x * each; r < min(((int)threadIdx.x + 1) * each, a.num_reqs); ++r) n += kv4_request_of(a, r, 8, &none).n;
    s[threadIdx.x] = n;
    __syncthreads();
    n = 0;
#pragma unroll 1
    for (int i = 0; i < kThreads; ++i) n += s[i];
    __syncthreads();
    return n > a.num_tokens;
}
#endif

// The chunk kernel: CTAs an SM, and floats of a part of an item (O, then m and l).
constexpr int kKv4ChunkCtas = 2;
constexpr int kv4_chunk_part(int head_size) { return kKv4ChunkRows * (head_size + 2); }

// Launches the chunk kernel in front of the other one.
int kv4_chunk_launch(const Kv4Args &a, int head_size, int sms, cudaStream_t stream);

}  // namespace pkv
