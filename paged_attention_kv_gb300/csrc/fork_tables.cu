// Rows of a block table that go on from other rows (parallel samples of a
// prompt, beam search), and the block copies that this takes ("Inside vLLM",
// page 1, "Prefix Caching": blocks of 16 that several requests' tables name).
//
// A row's full blocks are shared with the row it goes on from; a partly filled
// last block, which the row will write to, is kept by the first child and copied
// for the others. shares[b] counts the rows that hold block b beyond the first,
// so blocks that paged_build_tables hands out need no entry of their own. Rows
// that nobody goes on from give their blocks up; a block given up by its last
// holder goes back in front of the free list, in the order of rows and entries.
// Whichever row brings a count below zero, the entry with the lowest index takes
// the block (an atomic minimum on the count itself), so the order of the free
// list does not depend on the order of atomics.
//
// One cluster does it all, with a barrier between counting, claiming, giving
// back and handing out. Rows with exactly one child change no count; their entries are
// looked at where the new row is written, as those of all rows with children. A warp takes a
// row, four entries a lane at a time; as many CTAs as rows have warps, up to 16 (64
// beams with their copies 12.6 us, 14.7 in one CTA, then; a quarter of that many rows a CTA
// is no faster). Bound by its five phases, each a trip to L2 and a barrier of the
// cluster, 1.5 to 2 us together: 8.6 us for 64 rows, 11.3 for 384 (11.5 and 25.4 to 25.7
// with their copies), of which the bytes would take less than 1. The new rows are written
// while the counts are on their way.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <mutex>

#include "pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaxCtas = 16;
constexpr int kMinCtas = 8;           // that a cluster has on every device
constexpr int kFree = INT_MIN / 2;    // counts below this are claims: INT_MIN + entry
static_assert(PKV_MAX_FORK_ROWS / kMinCtas <= kThreads, "a thread has one of its CTA's rows at most");

struct ForkArgs {
    const int32_t *parents, *table, *lens;
    int rows, width, num_blocks;
    int32_t *shares, *free_blocks;
    int num_free;
    int32_t *cursor, *table_out, *lens_out, *copy_src, *copy_dst, *status;
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}

// Stores v to `at` (a shared address) of CTA `rank` of the cluster.
__device__ __forceinline__ void store_to(uint32_t at, uint32_t rank, int v) {
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.b32 [a], %2;\n\t}" ::"r"(at), "r"(rank), "r"(v)
                 : "memory");
}

// Counts seen after a cluster barrier: written by atomics, read past L1.
__device__ __forceinline__ int seen(const int32_t *p) { return __ldcg(p); }

__global__ void __launch_bounds__(kThreads) fork_tables_kernel(const ForkArgs a) {
    __shared__ int s_children[PKV_MAX_FORK_ROWS], s_first[PKV_MAX_FORK_ROWS];
    __shared__ int s_warp[32], s_total[kMaxCtas];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x, ctas = gridDim.x;  // the grid is one cluster
    const int R = a.rows;
    for (int r = tid; r < R; r += kThreads) {
        s_children[r] = 0;
        s_first[r] = INT_MAX;
    }
    pdl_wait();
    __syncthreads();
    int bits = 0;
    // the tokens of a row: 0 and flagged where its length is out of range
    auto length = [&](int r) {
        const int n = __ldg(a.lens + r);
        if (n >= 0 && n <= (long long)a.width * PKV_BLOCK_SIZE) return n;
        bits |= PKV_DEV_BAD_LEN;
        return 0;
    };
    auto parent = [&](int r) {
        const int p = __ldg(a.parents + r);
        if (p >= -1 && p < R) return p;
        bits |= PKV_DEV_BAD_PAGES;
        return -1;
    };
    // four entries a lane of a row from e0 on: -1 past `held`, flagged where no block
    constexpr int kU = 4;
    auto blocks = [&](int r, int e0, int held, int (&b)[kU]) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int e = e0 + 32 * u + lane;
            b[u] = e < held ? __ldg(a.table + (long long)r * a.width + e) : -1;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
            if (b[u] < 0 || b[u] >= a.num_blocks) {
                if (e0 + 32 * u + lane < held) bits |= PKV_DEV_BAD_BLOCK;
                b[u] = -1;
            }
    };
    for (int r = tid; r < R; r += kThreads) {
        const int p = parent(r);
        if (p >= 0) {
            atomicAdd(s_children + p, 1);
            atomicMin(s_first + p, r);
        }
    }
    const int cur = *a.cursor;
    const bool list = cur >= 0 && cur <= a.num_free;
    if (!list) bits |= PKV_DEV_BAD_PAGES;
    __syncthreads();

    // this CTA's rows, one a warp at a time; of a warp's first row the first entries are
    // read once, and their counts once in the two phases that see the same ones
    const int per = (R + ctas - 1) / ctas, r0 = min(R, rank * per), r1 = min(R, r0 + per), own = r0 + warp;
    int b_own[kU], v_own[kU];
    auto entries = [&](int r, int e0, int held, int (&b)[kU]) {
        if (r != own || e0) {
            blocks(r, e0, held, b);
            return;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) b[u] = b_own[u];
    };
    auto counts = [&](const int (&b)[kU], int (&v)[kU]) {
#pragma unroll
        for (int u = 0; u < kU; ++u) v[u] = b[u] >= 0 ? seen(a.shares + b[u]) : 0;
    };
    int gone = 0;  // rows without children that hold a block, of this thread's
    for (int r = tid; r < R; r += kThreads) gone |= s_children[r] == 0 && length(r) > 0;
    for (int r = own; r < r1; r += kThreads / 32) {
        const int c = s_children[r];
        if (c == 1) continue;
        const int n = length(r), full = n / PKV_BLOCK_SIZE, held = c ? full : (n + 15) / PKV_BLOCK_SIZE;
        if (r == own) blocks(r, 0, held, b_own);
        for (int e0 = 0; e0 < held; e0 += 32 * kU) {
            int b[kU];
            entries(r, e0, held, b);
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (b[u] >= 0) atomicAdd(a.shares + b[u], c - 1);
        }
    }
    cluster_arrive();
    // Meanwhile the new rows, but for the copies' places: every CTA numbers the copies
    // of all rows up to its own, of which a thread has one at most.
    int copies = 0, my_row = -1, my_src = -1, my_copy = -1, my_last = 0;
    for (int c0 = 0; c0 < R; c0 += kThreads) {
        const int r = c0 + tid;
        const int p = r < R ? parent(r) : -1;
        const int n = p >= 0 ? length(p) : 0;
        const int last = n / PKV_BLOCK_SIZE;
        const bool part = n % PKV_BLOCK_SIZE && s_first[p] != r;
        const int src = part ? __ldg(a.table + (long long)p * a.width + last) : -1;
        const bool copy = src >= 0 && src < a.num_blocks;  // no block stays as it is, in all children
        const uint32_t all = __ballot_sync(0xffffffffu, copy);
        __syncthreads();
        if (lane == 0) s_warp[warp] = __popc(all);
        __syncthreads();
        const int sum = __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0);
        const int sums = __reduce_add_sync(0xffffffffu, s_warp[lane]);
        if (r >= r0 && r < r1) {
            my_row = r;
            my_last = last;
            if (copy) {
                my_copy = copies + sum + __popc(all & ((1u << lane) - 1));
                my_src = src;
            }
            a.lens_out[r] = n;
        }
        copies += sums;
    }
    for (int r = own; r < r1; r += kThreads / 32) {
        const int p = parent(r), held = p >= 0 ? (length(p) + 15) / PKV_BLOCK_SIZE : 0;
        const int32_t *line = a.table + (long long)max(p, 0) * a.width;
        int32_t *to = a.table_out + (long long)r * a.width;
        for (int e0 = 0; e0 < a.width; e0 += 32 * kU) {
            int b[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int e = e0 + 32 * u + lane;
                b[u] = e < held ? __ldg(line + e) : -1;
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int e = e0 + 32 * u + lane;
                if (e < held && (b[u] < 0 || b[u] >= a.num_blocks)) bits |= PKV_DEV_BAD_BLOCK;
                if (e < a.width) to[e] = b[u];
            }
        }
    }
    cluster_wait();
    int given = 0;  // blocks that go back
    if (__syncthreads_or(gone)) {  // of all rows, so all CTAs agree
        for (int r = own; r < r1; r += kThreads / 32) {
            if (s_children[r]) continue;
            const int held = (length(r) + 15) / PKV_BLOCK_SIZE;
            for (int e0 = 0; e0 < held; e0 += 32 * kU) {
                int b[kU], v[kU];
                entries(r, e0, held, b);
                counts(b, v);
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    if (v[u] == -1 || v[u] < kFree) atomicMin(a.shares + b[u], INT_MIN + (r * a.width + e0 + 32 * u + lane));
                    else if (v[u] < -1) bits |= PKV_DEV_BAD_PAGES;  // given up more often than held
                }
            }
        }
        cluster_sync();
        // blocks that this CTA's rows give back
        int mine = 0;
        for (int r = own; r < r1; r += kThreads / 32) {
            if (s_children[r]) continue;
            const int held = (length(r) + 15) / PKV_BLOCK_SIZE;
            int got = 0;
            for (int e0 = 0; e0 < held; e0 += 32 * kU) {
                int b[kU], v[kU];
                entries(r, e0, held, b);
                counts(b, v);
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    got += v[u] == INT_MIN + (r * a.width + e0 + 32 * u + lane);
                    if (r == own && e0 == 0) v_own[u] = v[u];
                }
            }
            got = __reduce_add_sync(0xffffffffu, got);
            if (lane == 0) s_first[r] = got;  // a row without children has no first one
            mine += got;
        }
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        if (warp == 0) {
            const int sum = __reduce_add_sync(0xffffffffu, s_warp[lane]);
            if (lane < ctas) store_to(smem_u32(s_total + rank), lane, sum);
        }
        cluster_sync();
        int before = 0;
        for (int i = 0; i < ctas; ++i) {
            if (i < rank) before += s_total[i];
            given += s_total[i];
        }
        if (!list) given = 0;
        if (given > cur && list) bits |= PKV_DEV_BAD_PAGES;  // more than were ever taken
        const int base = list ? cur - given : 0;             // where the first one goes
        // every row's place: a sum over the CTA's rows before it (at most a thread each)
        {
            const int r = r0 + tid, n = r < r1 && !s_children[r] ? s_first[r] : 0;
            int v = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, v, d);
                if (lane >= d) v += o;
            }
            if (lane == 31) s_warp[warp] = v;
            __syncthreads();
            int sum = lane < warp ? s_warp[lane] : 0;
            sum = __reduce_add_sync(0xffffffffu, sum);
            if (r < r1 && !s_children[r]) s_first[r] = before + sum + v - n;
        }
        __syncthreads();
        for (int r = own; r < r1; r += kThreads / 32) {
            if (s_children[r]) continue;
            const int held = (length(r) + 15) / PKV_BLOCK_SIZE;
            int at = base + s_first[r];
            for (int e0 = 0; e0 < held; e0 += 32 * kU) {
                int b[kU], v[kU];
                entries(r, e0, held, b);
                if (r == own && e0 == 0) {
#pragma unroll
                    for (int u = 0; u < kU; ++u) v[u] = v_own[u];
                } else {
                    counts(b, v);
                }
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const bool take = v[u] == INT_MIN + (r * a.width + e0 + 32 * u + lane);
                    const uint32_t all = __ballot_sync(0xffffffffu, take);
                    if (take) {
                        const int to = at + __popc(all & ((1u << lane) - 1));
                        if (list && to >= 0) a.free_blocks[to] = b[u];
                    }
                    if (take || (v[u] < 0 && v[u] >= kFree)) a.shares[b[u]] = 0;
                    at += __popc(all);
                }
            }
        }
        cluster_sync();
    }
    // the copies' places
    const int from = list ? max(cur - given, 0) : 0;
    if (my_row >= 0) {
        int dst = -1;
        if (my_copy >= 0) {
            const int k = from + my_copy;
            if (list && k < a.num_free) {
                dst = __ldcg(a.free_blocks + k);
                if (dst < 0 || dst >= a.num_blocks) {
                    dst = -1;
                    bits |= PKV_DEV_BAD_BLOCK;
                }
            } else {
                bits |= PKV_DEV_NO_BLOCKS;
            }
            a.table_out[(long long)my_row * a.width + my_last] = dst;
        }
        a.copy_src[my_row] = dst < 0 ? -1 : my_src;
        a.copy_dst[my_row] = dst;
    }
    if (rank == 0 && tid == 0 && list) *a.cursor = from + min(copies, a.num_free - from);
    if (bits) raise_status(a.status, bits);
}

constexpr int kCopyThreads = 256;

struct CopyArgs {
    uint4 *pools[PKV_MAX_POOLS];
    const int32_t *src, *dst;
    long long vecs;  // 16-byte chunks of a block
    int num_pairs, num_blocks, splits;
    int32_t *status;
};

// A CTA copies one part of one block of one pool, in parts of a pass each, four at
// most: 64 beams 12.6 us against 13.7 with two, 384 samples (12 pools, 130 MB moved) 26.7
// against 28.1 with eight smaller ones.
__global__ void __launch_bounds__(kCopyThreads) copy_blocks_kernel(const __grid_constant__ CopyArgs a) {
    constexpr int kUnroll = 4;
    pdl_launch_dependents();
    pdl_wait();
    const int i = blockIdx.x / a.splits, part = blockIdx.x % a.splits;
    const int s = __ldg(a.src + i), d = __ldg(a.dst + i);
    if (s < 0 || d < 0) return;
    if (s >= a.num_blocks || d >= a.num_blocks) {
        if (threadIdx.x == 0 && part == 0 && blockIdx.y == 0) raise_status(a.status, PKV_DEV_BAD_BLOCK);
        return;
    }
    uint4 *pool = a.pools[blockIdx.y];
    const uint4 *from = pool + s * a.vecs;
    uint4 *to = pool + d * a.vecs;
    const long long end = a.vecs;
    for (long long base = (long long)part * kCopyThreads * kUnroll + threadIdx.x; base < end;
         base += (long long)a.splits * kCopyThreads * kUnroll) {
        uint4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (base + u * kCopyThreads < end) v[u] = __ldcs(from + base + u * kCopyThreads);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (base + u * kCopyThreads < end) to[base + u * kCopyThreads] = v[u];
    }
}

// The largest cluster this device takes, 16 or the 8 that every one takes.
std::mutex g_mu;
int g_cluster[64];

int largest_cluster(int *ctas) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_E_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_cluster[dev]) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kMaxCtas);
        cfg.blockDim = dim3(kThreads);
        int n = 0;
        if (cudaFuncSetAttribute(fork_tables_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
            cudaOccupancyMaxPotentialClusterSize(&n, fork_tables_kernel, &cfg) != cudaSuccess)
            return PKV_E_CUDA;
        g_cluster[dev] = n >= kMaxCtas ? kMaxCtas : kMinCtas;
    }
    *ctas = g_cluster[dev];
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" PKV_API int paged_fork_tables(const int32_t *parents, int32_t num_rows, const int32_t *block_table,
                                         int32_t max_blocks_per_req, const int32_t *seq_lens, int32_t num_blocks,
                                         int32_t *shares, int32_t *free_blocks, int32_t num_free, int32_t *free_cursor,
                                         int32_t *block_table_out, int32_t *seq_lens_out, int32_t *copy_src,
                                         int32_t *copy_dst, int32_t *status, void *stream) {
    if (num_rows < 0 || num_rows > PKV_MAX_FORK_ROWS || max_blocks_per_req < 0 || num_free < 0 || num_blocks <= 0)
        return PKV_E_DIMS;
    if (num_blocks > INT32_MAX / PKV_BLOCK_SIZE || max_blocks_per_req > INT32_MAX / PKV_BLOCK_SIZE ||
        (long long)num_rows * max_blocks_per_req > (1 << 29) || num_free > INT32_MAX - 65536)
        return PKV_E_DIMS;
    if (num_rows == 0) return PKV_OK;
    if (!parents || !seq_lens || !shares || !free_cursor || !seq_lens_out || !copy_src || !copy_dst ||
        (num_free > 0 && !free_blocks) || (max_blocks_per_req > 0 && (!block_table || !block_table_out)))
        return PKV_E_NULL;
    if (!aligned(parents, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(shares, 4) ||
        !aligned(free_blocks, 4) || !aligned(free_cursor, 4) || !aligned(block_table_out, 4) ||
        !aligned(seq_lens_out, 4) || !aligned(copy_src, 4) || !aligned(copy_dst, 4) || !aligned(status, 4))
        return PKV_E_ALIGN;
    if (block_table_out == block_table || seq_lens_out == seq_lens) return PKV_E_DIMS;
    const ForkArgs a{parents, block_table, seq_lens, num_rows, max_blocks_per_req, num_blocks, shares, free_blocks,
                     num_free, free_cursor, block_table_out, seq_lens_out, copy_src, copy_dst, status};
    // a warp a row, as far as a cluster goes
    int ctas = 1;
    while (ctas < kMinCtas && ctas * (kThreads / 32) < num_rows) ctas *= 2;
    if (ctas * (kThreads / 32) < num_rows) {
        const int rc = largest_cluster(&ctas);
        if (rc) return rc;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fork_tables_kernel, a) == cudaSuccess ? PKV_OK : PKV_E_CUDA;
}

extern "C" PKV_API int paged_copy_blocks(void *const *pools, int32_t num_pools, int64_t block_bytes, int32_t num_blocks,
                                         const int32_t *src, const int32_t *dst, int32_t num_pairs, int32_t *status,
                                         void *stream) {
    if (num_pools < 0 || num_pools > PKV_MAX_POOLS || num_pairs < 0 || num_pairs > INT32_MAX / 64 || num_blocks <= 0 ||
        block_bytes <= 0 || block_bytes % 16)
        return PKV_E_DIMS;
    if (num_pools == 0 || num_pairs == 0) return PKV_OK;
    if (!pools || !src || !dst) return PKV_E_NULL;
    if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(status, 4)) return PKV_E_ALIGN;
    CopyArgs a{};
    for (int i = 0; i < num_pools; ++i) {
        if (!pools[i]) return PKV_E_NULL;
        if (!aligned(pools[i], 16)) return PKV_E_ALIGN;
        a.pools[i] = static_cast<uint4 *>(pools[i]);
    }
    a.src = src;
    a.dst = dst;
    a.vecs = block_bytes / 16;
    a.num_pairs = num_pairs;
    a.num_blocks = num_blocks;
    a.splits = (int)std::min<long long>(4, std::max<long long>(1, a.vecs / (kCopyThreads * 4)));
    a.status = status;
    return launch_pdl(copy_blocks_kernel, dim3(num_pairs * a.splits, num_pools), dim3(kCopyThreads), 0,
                      static_cast<cudaStream_t>(stream), a) == cudaSuccess
               ? PKV_OK
               : PKV_E_CUDA;
}
