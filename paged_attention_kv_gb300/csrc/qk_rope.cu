// What a layer does to its projections before attention, in one pass: a
// root-mean-square norm of each q and k head, the rotation of the head's
// first columns by the token's position, and the KV write ("Inside vLLM",
// page 1, "Run forward pass": the forward pass computes q, k and v of the
// new tokens and populates their KVs in paged memory).
//
//   y = x * rsqrt(mean(x^2) + eps) * w          (no weight: y = x)
//   (a, b) -> (a cos - b sin, b cos + a sin)    pair f of the rotary columns,
//                                               angle at the token's position
//                                               on the axis that f belongs to
//
// All of it in 32 bits from the bf16 inputs, rounded to bf16 once. HBM-bound
// for many tokens: q and k are read and written once, v goes straight to the
// pool. A head is held by kLanes lanes, each with two 16-byte chunks that are
// half the rotary columns apart, so that either pairing of the columns stays
// within a lane; a warp stays with one token, so that positions, cosines and
// sines are read once for all the heads it takes. Two steps of heads are in
// flight ahead of the one at work; the arithmetic is on packed pairs (the
// scalar form was bound by instruction issue: 158 against 147 us then).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "rope_plan.h"

namespace pkv {
namespace {

// 24 warps an SM: 80 registers hold a warp's two heads in flight without much
// spilling (32768 tokens of 32/8 heads x 128 columns: 147 us in blocks of 256
// threads; with 16 warps 168, with 32, at 64 registers, 169). Small blocks, since
// a block's place is free for the next only when its last warp is done (64
// threads: 144 us, 2240 tokens 12.4 -> 11.9).
constexpr int kThreads = 64, kBlocksPerSm = 12;

struct RopeArgs {
    const __nv_bfloat16 *q, *k, *v, *q_weight, *k_weight;
    long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;  // elements from token to token
    __nv_bfloat16 *q_out, *k_out, *cache;
    const int32_t *positions, *slots;
    const float *cos_sin;
    int num_slots;
    int num_tokens, num_q_heads, num_kv_heads, head_size, rotary, num_axes, num_positions;
    int section_end[PKV_MAX_ROPE_AXES];  // axis a has the pairs [section_end[a - 1], section_end[a])
    int parts;                           // warps that share a token's heads
    float eps, inv_d;
    int32_t *status;
};

__device__ __forceinline__ int axis_of(const RopeArgs &a, int f) {
    int x = 0;
#pragma unroll
    for (int i = 0; i < PKV_MAX_ROPE_AXES - 1; ++i) x += i < a.num_axes - 1 && f >= a.section_end[i];
    return x;
}

// Eight bf16 values as four pairs of floats, and back.
__device__ __forceinline__ void unpack8(uint4 v, float2 (&x)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
    return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y),
                      pack_bf16x2(x[3].x, x[3].y));
}

template <int kLanes, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) qk_rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int kHeads = 32 / kLanes;  // heads a warp holds at once
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, j = lane % kLanes;
    const long long unit = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const long long t = unit / a.parts;
    const int part = (int)(unit - t * a.parts);
    if (t >= a.num_tokens) return;
    const int D = a.head_size, half = a.rotary / 2;
    const bool active = j < D / 16, turned = j < a.rotary / 16;
    // this lane's two chunks of every head
    const int c0 = turned ? j : a.rotary / 8 + 2 * (j - a.rotary / 16);
    const int c1 = turned ? j + a.rotary / 16 : c0 + 1;
    const int Hq = a.num_q_heads, Hkv = a.num_kv_heads;
    const int heads = Hq + Hkv + (a.cache ? Hkv : 0);
    const int row = D / 8;  // 16-byte chunks of a head
    const uint4 zero = make_uint4(0, 0, 0, 0);
    struct Head {
        uint4 x0, x1;
    };
    // Not through the read-only path: the outputs may be the inputs. (A warp
    // reads a head before it writes it, and no other warp touches it.)
    const __nv_bfloat16 *qt = a.q + t * a.q_stride, *kt = a.k + t * a.k_stride - Hq * D,
                        *vt = a.v + t * a.v_stride - (Hq + Hkv) * D;
    auto load = [&](int h) {
        Head r{zero, zero};
        if (active && h < heads) {
            const uint4 *src = reinterpret_cast<const uint4 *>((h < Hq ? qt : h < Hq + Hkv ? kt : vt) + h * D);
            r.x0 = src[c0];
            r.x1 = src[c1];
        }
        return r;
    };
    pdl_wait();
    // The first heads are on their way before the position and what hangs on
    // it are looked up.
    const int step = a.parts * kHeads;
    int h = part * kHeads + lane / kLanes;
    Head cur = load(h), next = load(h + step);

    // The token's positions; a negative one is padding, one past the table
    // is reported. Either way the token's rows are left as they are.
    int pos[PKV_MAX_ROPE_AXES];
    bool pad = false, bad = false;
#pragma unroll
    for (int x = 0; x < PKV_MAX_ROPE_AXES; ++x) {
        pos[x] = x < a.num_axes ? __ldg(a.positions + (long long)x * a.num_tokens + t) : 0;
        pad |= pos[x] < 0;
        bad |= pos[x] >= a.num_positions;
    }
    int slot = a.cache ? __ldg(a.slots + t) : -1;
    if (pad || bad) {
        if (!pad && part == 0 && lane == 0) raise_status(a.status, PKV_DEV_BAD_POS);
        return;
    }
    if (slot >= a.num_slots) {
        if (part == 0 && lane == 0) raise_status(a.status, PKV_DEV_BAD_SLOT);
        slot = -1;
    }
    // Cosines and sines of this lane's eight pairs, f0 .. f0 + 3 and f1 .. f1 + 3.
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cs[e] = 1.f;
        sn[e] = 0.f;
    }
    if (turned) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int f = kInterleaved ? (g ? c1 : c0) * 4 : j * 8 + g * 4;
            const int x0 = axis_of(a, f);
            if (axis_of(a, f + 3) == x0) {
                int p = pos[0];
#pragma unroll
                for (int x = 1; x < PKV_MAX_ROPE_AXES; ++x) p = x == x0 ? pos[x] : p;
                const float *at = a.cos_sin + (long long)p * a.rotary + f;
                const float4 c = __ldg(reinterpret_cast<const float4 *>(at));
                const float4 s = __ldg(reinterpret_cast<const float4 *>(at + half));
                cs[4 * g] = c.x; cs[4 * g + 1] = c.y; cs[4 * g + 2] = c.z; cs[4 * g + 3] = c.w;
                sn[4 * g] = s.x; sn[4 * g + 1] = s.y; sn[4 * g + 2] = s.z; sn[4 * g + 3] = s.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int xe = axis_of(a, f + e);
                    int p = pos[0];
#pragma unroll
                    for (int x = 1; x < PKV_MAX_ROPE_AXES; ++x) p = x == xe ? pos[x] : p;
                    const float *at = a.cos_sin + (long long)p * a.rotary + f + e;
                    cs[4 * g + e] = __ldg(at);
                    sn[4 * g + e] = __ldg(at + half);
                }
            }
        }
    }
    const long long tile = (long long)PKV_BLOCK_SIZE * row;
    uint4 *kv_row = reinterpret_cast<uint4 *>(a.cache) +
                    (slot >= 0 ? (long long)(slot / PKV_BLOCK_SIZE) * 2 * Hkv * tile + slot % PKV_BLOCK_SIZE * row : 0);
    // The warp's heads: all lanes go round equally often (the norms' sums
    // cross lanes), those past the last head with zeros.
    for (int base = part * kHeads; base < heads; base += step, h += step) {
        const Head in = cur;
        cur = next;
        next = load(h + 2 * step);
        const bool live = active && h < heads;
        if (h >= Hq + Hkv) {
            if (live && slot >= 0) {
                uint4 *dst = kv_row + (h - Hq) * tile;  // V's heads lie behind K's
                dst[c0] = in.x0;
                dst[c1] = in.x1;
            }
        }
        float2 x0[4], x1[4];
        unpack8(in.x0, x0);
        unpack8(in.x1, x1);
        if (a.q_weight || a.k_weight) {
            float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) s2 = ffma2(x0[e], x0[e], ffma2(x1[e], x1[e], s2));
            float ss = s2.x + s2.y;
#pragma unroll
            for (int d = kLanes / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
            const __nv_bfloat16 *w = h < Hq ? a.q_weight : a.k_weight;
            if (w && active) {
                const float rs = rsqrtf(fmaf(ss, a.inv_d, a.eps));
                const float2 rs2 = make_float2(rs, rs);
                float2 w0[4], w1[4];
                unpack8(__ldg(reinterpret_cast<const uint4 *>(w) + c0), w0);
                unpack8(__ldg(reinterpret_cast<const uint4 *>(w) + c1), w1);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x0[e] = fmul2(fmul2(x0[e], rs2), w0[e]);
                    x1[e] = fmul2(fmul2(x1[e], rs2), w1[e]);
                }
            }
        }
        if (!live || h >= Hq + Hkv) continue;
        if (turned) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 p = x0[e], r = x1[e];
                if (kInterleaved) {  // columns 2e and 2e + 1 of a chunk
                    x0[e] = make_float2(p.x * cs[e] - p.y * sn[e], p.y * cs[e] + p.x * sn[e]);
                    x1[e] = make_float2(r.x * cs[4 + e] - r.y * sn[4 + e], r.y * cs[4 + e] + r.x * sn[4 + e]);
                } else {             // the same column of both chunks
                    const float2 c = make_float2(cs[2 * e], cs[2 * e + 1]), s = make_float2(sn[2 * e], sn[2 * e + 1]);
                    x0[e] = ffma2(r, make_float2(-s.x, -s.y), fmul2(p, c));
                    x1[e] = ffma2(p, s, fmul2(r, c));
                }
            }
        }
        const uint4 y0 = pack8(x0), y1 = pack8(x1);
        if (h < Hq) {
            uint4 *dst = reinterpret_cast<uint4 *>(a.q_out + t * a.q_out_stride) + h * row;
            dst[c0] = y0;
            dst[c1] = y1;
        } else {
            if (a.k_out) {
                uint4 *dst = reinterpret_cast<uint4 *>(a.k_out + t * a.k_out_stride) + (h - Hq) * row;
                dst[c0] = y0;
                dst[c1] = y1;
            }
            if (slot >= 0) {
                uint4 *dst = kv_row + (h - Hq) * tile;
                dst[c0] = y0;
                dst[c1] = y1;
            }
        }
    }
}

template <int kLanes>
cudaError_t launch(const RopeArgs &a, bool interleaved, cudaStream_t st) {
    const long long units = (long long)a.num_tokens * a.parts;
    const int warps = kThreads / 32;
    const dim3 grid((unsigned)((units + warps - 1) / warps));
    return interleaved ? launch_pdl(qk_rope_kernel<kLanes, true>, grid, dim3(kThreads), 0, st, a)
                       : launch_pdl(qk_rope_kernel<kLanes, false>, grid, dim3(kThreads), 0, st, a);
}

bool stride_ok(long long stride, long long width, int tokens) {
    return stride % 8 == 0 && (tokens <= 1 || stride >= width) && stride < (1LL << 32);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" PKV_API int paged_qk_norm_rope(const pkv_rope_desc *d, const void *q, const void *k, const void *v,
                                          int32_t num_tokens, const void *q_weight, const void *k_weight,
                                          const int32_t *positions, const float *cos_sin, void *q_out, void *k_out,
                                          const int32_t *slot_mapping, void *kv_cache, int32_t num_blocks,
                                          int32_t *status, void *stream) {
    if (!d) return PKV_E_NULL;
    if (d->head_size <= 0 || d->head_size % 16 != 0 || d->head_size > 256) return PKV_E_HEAD_SIZE;
    if (num_tokens < 0 || d->num_q_heads <= 0 || d->num_kv_heads <= 0 || d->num_q_heads > 4096 ||
        d->num_kv_heads > 4096)
        return PKV_E_DIMS;
    if (d->rotary_dim < 16 || d->rotary_dim % 16 != 0 || d->rotary_dim > d->head_size || d->num_positions <= 0)
        return PKV_E_DIMS;
    if (d->num_axes < 1 || d->num_axes > PKV_MAX_ROPE_AXES || !(d->eps >= 0.f)) return PKV_E_DIMS;
    RopeArgs a{};
    int end = 0;
    for (int x = 0; x < d->num_axes; ++x) {
        const int n = d->num_axes == 1 ? d->rotary_dim / 2 : d->axis_pairs[x];
        if (n < 0 || n > d->rotary_dim / 2) return PKV_E_DIMS;
        end += n;
        a.section_end[x] = end;
    }
    if (end != d->rotary_dim / 2) return PKV_E_DIMS;
    const long long wq = (long long)d->num_q_heads * d->head_size, wkv = (long long)d->num_kv_heads * d->head_size;
    if (!stride_ok(d->q_stride, wq, num_tokens) || !stride_ok(d->k_stride, wkv, num_tokens) ||
        !stride_ok(d->q_out_stride, wq, num_tokens) || (k_out && !stride_ok(d->k_out_stride, wkv, num_tokens)) ||
        (kv_cache && !stride_ok(d->v_stride, wkv, num_tokens)))
        return PKV_E_DIMS;
    if (kv_cache && (num_blocks <= 0 || num_blocks > INT32_MAX / PKV_BLOCK_SIZE)) return PKV_E_DIMS;
    if (num_tokens == 0) return PKV_OK;
    if (!q || !k || !positions || !cos_sin || !q_out || (kv_cache && (!v || !slot_mapping))) return PKV_E_NULL;
    if (!k_out && !kv_cache) return PKV_E_NULL;
    // in place: a token's rows are where they were
    if (num_tokens > 1 && ((q_out == q && d->q_out_stride != d->q_stride) ||
                           (k_out == k && d->k_out_stride != d->k_stride)))
        return PKV_E_DIMS;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) ||
        !aligned(cos_sin, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(kv_cache, 16) ||
        !aligned(positions, 4) || !aligned(slot_mapping, 4) || !aligned(status, 4))
        return PKV_E_ALIGN;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.q_weight = static_cast<const __nv_bfloat16 *>(q_weight);
    a.k_weight = static_cast<const __nv_bfloat16 *>(k_weight);
    a.q_stride = d->q_stride;
    a.k_stride = d->k_stride;
    a.v_stride = d->v_stride;
    a.q_out_stride = d->q_out_stride;
    a.k_out_stride = d->k_out_stride;
    a.q_out = static_cast<__nv_bfloat16 *>(q_out);
    a.k_out = static_cast<__nv_bfloat16 *>(k_out);
    a.cache = static_cast<__nv_bfloat16 *>(kv_cache);
    a.positions = positions;
    a.slots = slot_mapping;
    a.cos_sin = cos_sin;
    a.num_slots = num_blocks * PKV_BLOCK_SIZE;
    a.num_tokens = num_tokens;
    a.num_q_heads = d->num_q_heads;
    a.num_kv_heads = d->num_kv_heads;
    a.head_size = d->head_size;
    a.rotary = d->rotary_dim;
    a.num_axes = d->num_axes;
    a.num_positions = d->num_positions;
    a.eps = d->eps;
    a.inv_d = 1.f / (float)d->head_size;
    a.status = status;
    const int lanes = d->head_size <= 64 ? 4 : d->head_size <= 128 ? 8 : 16;
    const int heads = d->num_q_heads + (kv_cache ? 2 : 1) * d->num_kv_heads, at_once = 32 / lanes;
    int sms = 0;
    const int rc = device_sms(&sms);
    if (rc) return rc;
    a.parts = rope_parts(num_tokens, (heads + at_once - 1) / at_once, (long long)sms * kBlocksPerSm * (kThreads / 32));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t err = lanes == 4 ? launch<4>(a, d->interleaved != 0, st)
                            : lanes == 8 ? launch<8>(a, d->interleaved != 0, st)
                                         : launch<16>(a, d->interleaved != 0, st);
    return err == cudaSuccess ? PKV_OK : PKV_E_CUDA;
}
