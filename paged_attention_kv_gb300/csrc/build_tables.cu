// A step's metadata from its requests' lengths: new blocks handed out in
// request order, block-table rows extended, sequence lengths, query starts,
// positions and slots ("Inside vLLM", page 1, "Scheduler": allocate_slots
// gives each request the blocks of 16 that its new tokens need; "Run forward
// pass", step 2, builds the tables and the slot mapping).
//
// Request r with L0 tokens of context and n new ones ends at L1 = L0 + n and
// takes ceil(L1 / 16) - ceil(L0 / 16) new blocks; both prefix sums (tokens,
// blocks) come from one scan. Every CTA scans all requests (a kilobyte or two
// from L2), which costs less than handing the result on, and then fills its
// share of the tokens; the new token at a block's first position also writes
// the block-table entry, so no entry is written twice. Where the lengths or the
// cursor are updated in place, rank 0 writes them once every CTA has read them:
// the grid is then one cluster, with a cluster barrier per kThreads requests.
// Otherwise nothing is read that another CTA writes, and the CTAs are as many as
// the rows want. Bound by its launch and the round trips to memory one behind
// another (lengths, free ids, rows): 4.3 us back to back for 256 decode
// requests, 4.6 us for 200 prompts of 103k tokens together, 6.2 us for 700 of
// 138k (in place, where 16 SMs write all rows, 9.7 to 11.5).
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

struct TableArgs {
    const int32_t *query_lens, *context_lens, *free_blocks, *cursor;
    int num_reqs, max_blocks_per_req, num_free, num_tokens, num_blocks;
    int32_t *block_table, *seq_lens, *qsl, *positions, *slots, *cursor_out, *status;
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Tokens and blocks summed side by side, each clamped to its cap: one more
// than the step's rows, one more than the ids left. A sum at its cap refuses
// its request whatever its exact value, and clamped sums of counts are still
// associative, so 32 bits do for any lengths.
struct Sums {
    uint32_t tok, blk;
};

__device__ __forceinline__ Sums add(Sums a, Sums b, Sums cap) {
    return {min(a.tok + b.tok, cap.tok), min(a.blk + b.blk, cap.blk)};
}

__device__ __forceinline__ Sums shift(Sums v, int d) {
    return {__shfl_up_sync(0xffffffffu, v.tok, d), __shfl_up_sync(0xffffffffu, v.blk, d)};
}

// Inclusive sums over the warp; *before: the exclusive ones.
__device__ __forceinline__ Sums warp_scan(Sums v, Sums cap, int lane, Sums *before) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Sums o = shift(v, d);
        if (lane >= d) v = add(v, o, cap);
    }
    *before = shift(v, 1);
    if (lane == 0) *before = {0, 0};
    return v;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) build_tables_kernel(const TableArgs a) {
    constexpr int kWarps = kThreads / 32;
    __shared__ Sums s_warp[kWarps];
    __shared__ int s_start[kThreads + 1];  // first row of each request of the pass, at most num_tokens
    __shared__ int s_len[kThreads];        // context before the step; -1: the request is refused
    __shared__ int s_base[kThreads];       // its first new id in free_blocks
    __shared__ uint32_t s_taken;           // ids handed out so far
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = blockIdx.x;  // the grid is one cluster, or no CTA waits for another
    const int T = a.num_tokens;
    if (tid == 0) s_taken = 0;
    // No early trigger: kernels of this library that read the tables ahead
    // of their own wait must not start before this one has finished.
    pdl_wait();
    const int cur = a.cursor ? *a.cursor : 0;
    const uint32_t avail = cur >= 0 && cur <= a.num_free ? a.num_free - cur : 0;
    const Sums cap{(uint32_t)T + 1, avail + 1};
    Sums carry{0, 0};
    int bits = 0;
    for (int r0 = 0; r0 == 0 || r0 < a.num_reqs; r0 += kThreads) {
        const int r = r0 + tid;
        const bool in = r < a.num_reqs;
        int n = in ? __ldg(a.query_lens + r) : 0;
        const int L0 = in ? a.context_lens[r] : 0;  // may be written below: not through the read-only path
        if (n < 0) {
            n = 0;
            bits |= PKV_DEV_BAD_QSL;
        }
        const long long L1 = (long long)L0 + n;
        bool refused = L0 < 0 || L1 > (long long)a.max_blocks_per_req * PKV_BLOCK_SIZE;
        if (refused) bits |= PKV_DEV_BAD_LEN;
        const uint32_t need = refused ? 0 : (uint32_t)((L1 + 15) / 16 - (L0 + 15LL) / 16);
        Sums before;
        const Sums v = warp_scan({min((uint32_t)n, cap.tok), min(need, cap.blk)}, cap, lane, &before);
        if (lane == 31) s_warp[warp] = v;
        __syncthreads();
        // every warp adds up the warps before it, each lane one warp's sums
        Sums base;
        const Sums upto = warp_scan(lane < kWarps ? s_warp[lane] : Sums{0, 0}, cap, lane, &base);
        base = {__shfl_sync(0xffffffffu, base.tok, warp), __shfl_sync(0xffffffffu, base.blk, warp)};
        base = add(carry, base, cap);
        const Sums first = add(base, before, cap), end = add(base, v, cap);
        carry = add(carry, {__shfl_sync(0xffffffffu, upto.tok, 31), __shfl_sync(0xffffffffu, upto.blk, 31)}, cap);
        // Requests whose rows do not fit the step, or whose blocks are not
        // there, get nothing. The sums only grow, so a refusal never changes
        // what the requests before it got.
        if (n > 0 && end.tok > (uint32_t)T) {
            refused = true;
            bits |= PKV_DEV_BAD_QSL;
        }
        if (need > 0 && end.blk > avail) {
            refused = true;
            bits |= PKV_DEV_NO_BLOCKS;
        }
        s_start[tid] = (int)min(first.tok, (uint32_t)T);
        s_len[tid] = refused ? -1 : L0;
        s_base[tid] = refused ? 0 : cur + (int)first.blk;
        if (tid == kThreads - 1) s_start[kThreads] = (int)min(end.tok, (uint32_t)T);
        const uint32_t got = __reduce_max_sync(0xffffffffu, refused || need == 0 ? 0u : end.blk);
        if (lane == 0 && got) atomicMax(&s_taken, got);
        __syncthreads();
        cluster_arrive();  // this CTA has read the pass's lengths (and the cursor)

        const int t0 = s_start[0], t1 = s_start[kThreads];
        const bool wide = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15) == 0;
        for (int g = (t0 >> 2) + (int)rank * kThreads + tid; g < ((t1 + 3) >> 2);
             g += (int)(gridDim.x * kThreads)) {
            int pos[4], slot[4];
            int j = -1, nxt = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 4 * g + e;
                pos[e] = slot[e] = -1;
                if (t < t0 || t >= t1) continue;
                if (j < 0 || t >= nxt) {
                    // the last request of the pass that starts at or before t
                    int lo = j < 0 ? 0 : j, hi = kThreads;
                    if (j >= 0 && (j + 2 >= kThreads || s_start[j + 2] > t)) {
                        lo = j + 1;  // the next one, as among decode requests
                    } else {
                        while (hi - lo > 1) {
                            const int mid = (lo + hi) >> 1;
                            if (s_start[mid] <= t) lo = mid; else hi = mid;
                        }
                    }
                    j = lo;
                    nxt = s_start[j + 1];
                }
                const int len = s_len[j];
                if (len < 0) continue;
                const int p = len + (t - s_start[j]);
                const int b = p / PKV_BLOCK_SIZE, fresh = b - (len + 15) / 16;
                int32_t *entry = a.block_table + (long long)(r0 + j) * a.max_blocks_per_req + b;
                int id = fresh >= 0 ? __ldg(a.free_blocks + s_base[j] + fresh) : *entry;
                if (id < 0 || id >= a.num_blocks) {
                    bits |= PKV_DEV_BAD_BLOCK;
                    id = -1;
                }
                if (p % PKV_BLOCK_SIZE == 0) *entry = id;
                pos[e] = p;
                slot[e] = id < 0 ? -1 : id * PKV_BLOCK_SIZE + p % PKV_BLOCK_SIZE;
            }
            if (wide && 4 * g >= t0 && 4 * g + 3 < t1) {
                *reinterpret_cast<int4 *>(a.slots + 4 * g) = make_int4(slot[0], slot[1], slot[2], slot[3]);
                if (a.positions)
                    *reinterpret_cast<int4 *>(a.positions + 4 * g) = make_int4(pos[0], pos[1], pos[2], pos[3]);
                continue;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 4 * g + e;
                if (t < t0 || t >= t1) continue;
                a.slots[t] = slot[e];
                if (a.positions) a.positions[t] = pos[e];
            }
        }
        __syncwarp();
        cluster_wait();
        if (rank == 0 && in) {
            a.seq_lens[r] = refused ? L0 : (int)L1;
            a.qsl[r + 1] = (int)min(end.tok, (uint32_t)T);
        }
        __syncthreads();
    }
    // rows behind the last request
    for (long long t = (long long)min(carry.tok, (uint32_t)T) + (long long)rank * kThreads + tid; t < T;
         t += gridDim.x * kThreads) {
        a.slots[t] = -1;
        if (a.positions) a.positions[t] = -1;
    }
    if (rank == 0 && tid == 0) {
        a.qsl[0] = 0;
        if (a.cursor_out) *a.cursor_out = cur + (int)s_taken;
    }
    if (bits) raise_status(a.status, bits);
    __threadfence();
}

// Rows a CTA fills at four a thread; as many CTAs as are at work at once, 1024
// threads an SM, take the rows in turn.
constexpr int kRowsPerThread = 4;

int ctas_for(int rows, int threads, int most) {
    const int per = threads * kRowsPerThread;
    return std::min(most, std::max(1, (rows + per - 1) / per));
}

// The largest cluster this device takes, 16 or the 8 that every one takes.
std::mutex g_mu;
int g_cluster[64];

int large_cluster(int *ctas) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_E_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_cluster[dev]) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(1024);
        int n = 0;
        if (cudaFuncSetAttribute(build_tables_kernel<1024>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
                cudaSuccess ||
            cudaOccupancyMaxPotentialClusterSize(&n, build_tables_kernel<1024>, &cfg) != cudaSuccess)
            return PKV_E_CUDA;
        g_cluster[dev] = n >= 16 ? 16 : 8;
    }
    *ctas = g_cluster[dev];
    return PKV_OK;
}

template <int kThreads>
cudaError_t launch(const TableArgs &a, int ctas, int cluster, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, build_tables_kernel<kThreads>, a);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" PKV_API int paged_build_tables(const int32_t *query_lens, const int32_t *context_lens, int32_t num_reqs,
                                          const int32_t *free_blocks, int32_t num_free, const int32_t *free_cursor,
                                          int32_t num_tokens, int32_t num_blocks, int32_t *block_table,
                                          int32_t max_blocks_per_req, int32_t *seq_lens, int32_t *query_start_loc,
                                          int32_t *positions, int32_t *slot_mapping, int32_t *free_cursor_out,
                                          int32_t *status, void *stream) {
    if (num_reqs < 0 || num_tokens < 0 || num_free < 0 || max_blocks_per_req < 0 || num_blocks <= 0)
        return PKV_E_DIMS;
    if (num_blocks > INT32_MAX / PKV_BLOCK_SIZE || max_blocks_per_req > INT32_MAX / PKV_BLOCK_SIZE ||
        num_tokens > INT32_MAX - 65536 || num_reqs > INT32_MAX - 65536 || num_free > INT32_MAX - 65536)
        return PKV_E_DIMS;
    if (!query_start_loc || (num_tokens > 0 && !slot_mapping) || (num_free > 0 && !free_blocks)) return PKV_E_NULL;
    if (num_reqs > 0 && (!query_lens || !context_lens || !seq_lens || (max_blocks_per_req > 0 && !block_table)))
        return PKV_E_NULL;
    if (!aligned(query_lens, 4) || !aligned(context_lens, 4) || !aligned(free_blocks, 4) || !aligned(free_cursor, 4) ||
        !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) || !aligned(positions, 4) ||
        !aligned(slot_mapping, 4) || !aligned(free_cursor_out, 4) || !aligned(status, 4))
        return PKV_E_ALIGN;
    const TableArgs a{query_lens,  context_lens, free_blocks, free_cursor,  num_reqs, max_blocks_per_req, num_free,
                      num_tokens,  num_blocks,   block_table, seq_lens,     query_start_loc, positions, slot_mapping,
                      free_cursor_out, status};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // CTAs of 256 threads start sooner and meet sooner than those of 1024 (256
    // decode requests: 4.4 against 5.4 us; 2304 rows of 196 requests: 3 CTAs of
    // 256 4.7 us, one of 1024 6.0), but more requests than threads make the scan
    // go round again (700 prompts, 138k rows: 10.4 against 6.2 us).
    const bool small = num_reqs <= 256;
    cudaError_t err;
    if (seq_lens != context_lens && (!free_cursor || free_cursor_out != free_cursor)) {
        int sms = 0;
        const int rc = device_sms(&sms);
        if (rc) return rc;
        err = small ? launch<256>(a, ctas_for(num_tokens, 256, 4 * sms), 1, st)
                    : launch<1024>(a, ctas_for(num_tokens, 1024, sms), 1, st);
    } else if (small && num_tokens <= 8 * 256 * kRowsPerThread) {
        const int ctas = ctas_for(num_tokens, 256, 8);  // a cluster that every device takes
        err = launch<256>(a, ctas, ctas, st);
    } else {
        // One CTA while its scan, not the rows, takes the time; beyond, as
        // many as a cluster takes (700 prompts: 13.9 us with 8 CTAs, 9.7 with 16).
        int ctas = 1;
        if (num_tokens > 1024 * kRowsPerThread) {
            const int rc = large_cluster(&ctas);
            if (rc) return rc;
        }
        err = launch<1024>(a, ctas, ctas, st);
    }
    return err == cudaSuccess ? PKV_OK : PKV_E_CUDA;
}
