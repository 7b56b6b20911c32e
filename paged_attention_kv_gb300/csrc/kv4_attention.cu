// Causal attention with grouped heads over the 4-bit pool (kv4_format.cuh), for
// a ragged batch of decode tokens and chunks.
//
// For a row (query token, head) with keys j = 0 .. p:
//     out = sum_j softmax_j(scale q . K_j) V_j,  K_j = k_scale * codes * scales
// A warp works alone. It takes an item's blocks of 16 keys two at a time through
// its own ring of bulk copies, turns the codes into fp16 fragments in registers
// (exactly: six significant bits), and runs both products transposed, S^T (16
// keys x 8 rows) = K Q^T and O^T (D x 8 rows) += V^T P^T, on mma.sync m16n8k16,
// so that the 4 to 8 rows of a decode token's head group fill the N side and K
// and V are made once for up to four such groups of rows. An item is (request,
// tile of 8 kMaxNt rows, kv head) and its cost a number of keys; all items in a
// row are cut into equal shares, one a warp (kv4_plan.h), neighbouring shares in
// one CTA. An item that lies in several shares leaves one partial (m, l, O) a
// share, in the layout of the fragments: the first of its warps in a CTA joins
// those of the CTA, through shared memory, and where it lies in several CTAs,
// all warps of the last of them to arrive join theirs, always in order, so that
// the result does not depend on timing. Every CTA adds the requests' costs up
// itself: one launch.
//
// Softmax: scores stay unscaled; a row's reference m is the largest score of its
// first two blocks, and moves only when a score passes it by 2^10 (p then still
// fits fp16), so that two blocks cost one vote and no exchange between lanes. p is
// 2^x in 32 bits, rounded to fp16 (2^-11 of each) for the product with V; sums are
// held in 32 bits.
//
// Bound by, and measured (us in a graph, one GB300; bytes over the copy bandwidth
// of 6685 GB/s as the floor):
//   256 decode requests of 512 to 4096 keys, 32 heads on 8 of 128: 94.1, floor 78.3.
//     525 MB of DRAM reads, 6.3 TB/s while all warps work (copies alone, without the
//     products: 88 us in all); 10 us of prologue, items' starts, joins and ends. 57 % of
//     the issue slots.
//   the same with 4 tokens each: 133.5, floor 80. Three warps a scheduler, as many as
//     registers allow, wait for one another's chains (48 % of the issue slots); 105 KB
//     of code pass through the instruction cache, and items' starts and ends wait for it.
//   64 decode requests of 128 to 2048 keys, 4 heads of 64: 12.8, floor 2.3: a chain of
//     1.3 us for the sums of all costs, 1 for a warp's share, 1 to the first keys, 3
//     of them, and joins. Two requests of 17 and 40 keys: 5.3. Instructions that run
//     once come from L2 and are waited for, hence the votes,
//     approximate quotients and few branches where each warp finds its share.
//   3 requests of 30000 to 100000 keys: 34.1, floor 21.1.
// Chosen against: one block at a time with 14 or 16 warps (16 rows 149 to 168 us against
// 143 then; 8 rows 110 against 99), scores a pair ahead of the values (103 against 97:
// registers), 8 rows with 16 warps of 128 registers (103 against 99), 32 rows with 10
// warps (spills), pieces joined by all of a CTA's warps (64 requests 17.8 against 15.3).
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "kv4_args.h"
#include "kv4_format.cuh"
#include "kv4_plan.h"
#include "pagedkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_short_wait.cuh"

namespace pkv {
namespace {

// Warps of a CTA (one CTA an SM), and copies of two blocks that a warp has in
// flight, by the rows of a tile.
template <int kMaxNt>
constexpr int kWarps = kMaxNt == 4 ? 8 : 12;
template <int D, int kMaxNt>
constexpr int kStages = (D == 64 ? 2 : 1) * 3;

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) { return as_u32(__floats2half2_rn(lo, hi)); }

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
        : "memory");
}

// A row's reference before it sees any key: its sums are 0 then, whatever they are
// multiplied by, and no score is below it.
constexpr float kNoKey = -FLT_MAX;
// The factor that what was taken against reference m has against `to`.
__device__ __forceinline__ float against(float m, float to, float mul) { return fast_exp2((m - to) * mul); }

template <int D, int kNt>
constexpr int kQBytes = kNt * (D / 16) * 2 * 32 * 4;  // q's fragments of 8 kNt rows

// What a lane (4 g + t) reads of a tile: K of two tokens, V of two pairs of tokens.
template <int D>
struct Lane {
    static constexpr int kW = D / 32;  // words of codes of each

    static __device__ __forceinline__ void load_k(uint32_t tile, int lane, uint32_t (&k)[2][kW], uint32_t &scales) {
        if constexpr (D == 128) {
            lds(k[0], tile + 16 * lane);
            lds(k[1], tile + 4 * D + 16 * lane);
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(scales) : "r"(tile + 16 * D + 4 * lane));
        } else {
            lds(k[0], tile + 8 * lane);
            lds(k[1], tile + 4 * D + 8 * lane);
            asm volatile("{\n\t.reg .b16 s;\n\tld.shared.b16 s, [%1];\n\tcvt.u32.u16 %0, s;\n\t}" : "=r"(scales) : "r"(tile + 16 * D + 2 * lane));
        }
    }
    static __device__ __forceinline__ void load_v(uint32_t tile, int lane, uint32_t (&v)[2][kW], uint32_t &scales) {
        lds(v[0], tile + 8 * D + 4 * kW * lane);
        lds(v[1], tile + 12 * D + 4 * kW * lane);
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(scales) : "r"(tile + 17 * D + (D == 128 ? 4 * lane : 16 * (lane >> 3) + 4 * (lane & 3))));
    }
    static __device__ __forceinline__ void lds(uint32_t (&w)[4], uint32_t at) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
    }
    static __device__ __forceinline__ void lds(uint32_t (&w)[2], uint32_t at) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
    }
};

// Where a pair of blocks lies among its item's rows.
struct Span {
    int key0;    // position of the first block's first key
    int limit0;  // keys that the tile's first row sees
    int end;     // keys that its last row sees
    int row0, tok0, group;  // tok0: row0 / group
    uint32_t inv;

    // keys of the pair that row `row` of the tile sees (at most 32 count)
    __device__ __forceinline__ int sees(int row) const { return limit0 + kv4_over(row0 + row, group, inv) - tok0 - key0; }
};

// A whole warp's state for one item of up to 8 kNt rows. Of O^T a lane holds,
// for rows 8 n + 2 t and 8 n + 2 t + 1, the D / 8 columns from D / 8 * g on. With
// 16 rows or more q's fragments lie in shared memory: registers are full of O.
template <int D, int kNt>
struct Item {
    static constexpr int kK = D / 16;  // steps of 16 columns
    static constexpr int kW = Lane<D>::kW;
    static constexpr bool kQShared = kNt >= 2;
    float o[kNt][kK][4];
    float2 m[kNt], l[kNt], mul[kNt];
    uint32_t q[kQShared ? 1 : kNt][kQShared ? 1 : kK][2];
    uint32_t q_at;  // shared address, this lane's

    // q rows as they are; zero past `rows`. The loads go out before anything waits for
    // the block ids.
    using Rows = uint4[kNt][D / 32];
    static __device__ __forceinline__ void read_q(const Kv4Args &a, int token0, int row0, int rows, int head, Rows &w, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
            const int row = 8 * n + g;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) w[n][i] = make_uint4(0, 0, 0, 0);
            if (row < rows) {
                const int rr = row0 + row, tok = kv4_over(rr, a.group, a.group_inv);
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    a.q + (long long)(token0 + tok) * a.q_stride + (long long)(head * a.group + rr - tok * a.group) * D) + t * (D / 32);
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
                    asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[n][i].x), "=r"(w[n][i].y), "=r"(w[n][i].z), "=r"(w[n][i].w)
                                 : "l"(src + i));
            }
        }
    }
    // As fp16 fragments, each row scaled by a power of two to lie in (-4, 4); mul takes
    // that back.
    __device__ __forceinline__ void begin(const Kv4Args &a, int rows, const Rows &all, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
            const int row = 8 * n + g;
            const uint4 (&w)[D / 32] = all[n];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t mk = 0x7fff7fffu;
                const uint32_t x = __vmaxu2(__vmaxu2(w[i].x & mk, w[i].y & mk), __vmaxu2(w[i].z & mk, w[i].w & mk));
                top = max(top, max(x & 0xffffu, x >> 16));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // exponent of the largest value; a row that is not finite keeps its values
            int e = (int)(top >> 7);
            e = e == 255 ? 127 : min(max(e, 1), 253);
            const float down = __uint_as_float((uint32_t)(254 - e) << 23), up = __uint_as_float((uint32_t)e << 23);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                uint32_t f[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = pack_f16x2(__uint_as_float(x[j] << 16) * down, __uint_as_float(x[j] & 0xffff0000u) * down);
                if constexpr (kQShared) {
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(q_at + 512 * (n * kW + i)), "r"(f[0]), "r"(f[1]), "r"(f[2]), "r"(f[3])
                                 : "memory");
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) q[n][2 * i + j / 2][j & 1] = f[j];
                }
            }
            // neither 0 nor infinite: masked scores times it have to stay -inf, and 0 has to stay 0
            const float f = row < rows ? fminf(fmaxf(up * a.small * a.scale_log2, 0x1p-126f), 0x1p127f) : 1.0f;
            mul[n] = make_float2(__shfl_sync(0xffffffffu, f, 8 * t), __shfl_sync(0xffffffffu, f, 8 * t + 4));
            m[n] = make_float2(kNoKey, kNoKey);
            l[n] = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < kK; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[n][i][c] = 0.0f;
        }
    }

    // The row's reference becomes the largest score so far.
    static __device__ __forceinline__ void move(float &m, float &l, float mul, float top, float *f) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float to = fmaxf(m, top);
        *f = against(m, to, mul);
        m = to;
        l *= *f;
    }
    __device__ __forceinline__ void move_references(const float (&s)[2][kNt][4]) {
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
            float fx, fy;
            move(m[n].x, l[n].x, mul[n].x, fmaxf(fmaxf(s[0][n][0], s[0][n][2]), fmaxf(s[1][n][0], s[1][n][2])), &fx);
            move(m[n].y, l[n].y, mul[n].y, fmaxf(fmaxf(s[0][n][1], s[0][n][3]), fmaxf(s[1][n][1], s[1][n][3])), &fy);
#pragma unroll
            for (int i = 0; i < kK; ++i) {
                o[n][i][0] *= fx;
                o[n][i][1] *= fy;
                o[n][i][2] *= fx;
                o[n][i][3] *= fy;
            }
        }
    }
    // Scores to exponents of 2 against the references; returns the largest.
    __device__ __forceinline__ float exponents(const float (&s)[2][kNt][4], float (&e)[2][kNt][4]) const {
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const float2 x = fmul2(fadd2(make_float2(s[b][n][0], s[b][n][1]), make_float2(-m[n].x, -m[n].y)), mul[n]);
                const float2 y = fmul2(fadd2(make_float2(s[b][n][2], s[b][n][3]), make_float2(-m[n].x, -m[n].y)), mul[n]);
                e[b][n][0] = x.x, e[b][n][1] = x.y, e[b][n][2] = y.x, e[b][n][3] = y.y;
                top = fmax3(top, fmax3(x.x, x.y, y.x), y.y);
            }
        }
        return top;
    }

    // Scores of the two blocks at `tile` and behind it.
    __device__ __forceinline__ void scores(uint32_t tile, float (&s)[2][kNt][4], int lane) const {
        {
            uint32_t k[2][2][kW], ks[2];
            Lane<D>::load_k(tile, lane, k[0], ks[0]);
            Lane<D>::load_k(tile + Kv4Tile<D>::kBytes, lane, k[1], ks[1]);
            // scales: tokens g and g + 8, one or two groups of this lane's quarter
            __half2 sc[2][2][2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if constexpr (D == 128) {
                    const __half2 x = kv4_scales(ks[b]), y = kv4_scales(ks[b] >> 16);
                    sc[b][0][0] = __low2half2(x), sc[b][0][1] = __high2half2(x);
                    sc[b][1][0] = __low2half2(y), sc[b][1][1] = __high2half2(y);
                } else {
                    const __half2 x = kv4_scales(ks[b]);
                    sc[b][0][0] = sc[b][0][1] = __low2half2(x);
                    sc[b][1][0] = sc[b][1][1] = __high2half2(x);
                }
#pragma unroll
                for (int n = 0; n < kNt; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[b][n][c] = 0.0f;
            }
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const int p = w * 2 / kW;
                uint32_t f[2][2][4];  // of each block: two steps
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint32_t x = k[b][0][w], y = k[b][1][w];
                    f[b][0][0] = as_u32(__hmul2(kv4_pair<0>(x), sc[b][0][p])), f[b][0][1] = as_u32(__hmul2(kv4_pair<0>(y), sc[b][1][p]));
                    f[b][0][2] = as_u32(__hmul2(kv4_pair<1>(x), sc[b][0][p])), f[b][0][3] = as_u32(__hmul2(kv4_pair<1>(y), sc[b][1][p]));
                    f[b][1][0] = as_u32(__hmul2(kv4_pair<2>(x), sc[b][0][p])), f[b][1][1] = as_u32(__hmul2(kv4_pair<2>(y), sc[b][1][p]));
                    f[b][1][2] = as_u32(__hmul2(kv4_pair<3>(x), sc[b][0][p])), f[b][1][3] = as_u32(__hmul2(kv4_pair<3>(y), sc[b][1][p]));
                }
#pragma unroll
                for (int n = 0; n < kNt; ++n) {
                    uint32_t qf[4];
                    if constexpr (kQShared) {
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(qf[0]), "=r"(qf[1]), "=r"(qf[2]), "=r"(qf[3])
                                     : "r"(q_at + 512 * (n * kW + w)));
                    } else {
                        qf[0] = q[n][2 * w][0], qf[1] = q[n][2 * w][1], qf[2] = q[n][2 * w + 1][0], qf[3] = q[n][2 * w + 1][1];
                    }
#pragma unroll
                    for (int b = 0; b < 2; ++b) mma_f16(s[b][n], f[b][0], qf[0], qf[1]);
#pragma unroll
                    for (int b = 0; b < 2; ++b) mma_f16(s[b][n], f[b][1], qf[2], qf[3]);
                }
            }
        }
    }

    // Their probabilities, as fragments for the product with V. masked: some row does
    // not see all of their keys. One copy of everything: what runs once an item comes
    // from L2, and is waited for.
    __device__ __forceinline__ void probabilities(float (&s)[2][kNt][4], bool masked, bool first, const Span &at, uint32_t (&p)[2][kNt][2], int lane) {
        const int g = lane >> 2, t = lane & 3;
        float e[2][kNt][4];
        if (masked) {
#pragma unroll
            for (int n = 0; n < kNt; ++n) {
                // never past the last row's keys: rows of padding would see more, and the
                // second block may be missing
                const int end = at.end - at.key0, x = min(at.sees(8 * n + 2 * t), end), y = min(at.sees(8 * n + 2 * t + 1), end);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (16 * b + g >= x) s[b][n][0] = -INFINITY;
                    if (16 * b + g >= y) s[b][n][1] = -INFINITY;
                    if (16 * b + g + 8 >= x) s[b][n][2] = -INFINITY;
                    if (16 * b + g + 8 >= y) s[b][n][3] = -INFINITY;
                }
            }
        }
        const float top = exponents(s, e);
        if (__any_sync(0xffffffffu, top > 10.0f) || first) {
            move_references(s);
            exponents(s, e);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int n = 0; n < kNt; ++n) {
                float x[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) x[c] = fast_exp2(e[b][n][c]);
                l[n] = fadd2(l[n], fadd2(make_float2(x[0], x[1]), make_float2(x[2], x[3])));
                p[b][n][0] = movmatrix_trans(pack_f16x2(x[0], x[1]));
                p[b][n][1] = movmatrix_trans(pack_f16x2(x[2], x[3]));
            }
    }

    // O += V P; between(): called when the tiles are read.
    template <typename Between>
    __device__ __forceinline__ void values(uint32_t tile, bool masked, const Span &at, const uint32_t (&p)[2][kNt][2], Between between, int lane) {
        uint32_t v[2][2][kW], vs[2];
        Lane<D>::load_v(tile, lane, v[0], vs[0]);
        Lane<D>::load_v(tile + Kv4Tile<D>::kBytes, lane, v[1], vs[1]);
        __syncwarp();
        between();
        if (masked) {
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                uint32_t x = b ? vs[1] : vs[0];
                guard(x, b, at, lane);
                if (b) vs[1] = x;
                else vs[0] = x;
            }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const __half2 va = kv4_scales(vs[b]), vb = kv4_scales(vs[b] >> 16);  // tokens 2 t, 2 t + 1 and 8 on
#pragma unroll
            for (int w = 0; w < kW / 2; ++w) {
                // low and high codes of two tokens side by side
                constexpr int kH = kW / 2;
                const uint32_t a0 = v[b][0][w], a1 = v[b][0][w + kH], b0 = v[b][1][w], b1 = v[b][1][w + kH];
                const uint32_t lo = 0x0f0f0f0fu;
                const uint32_t ae = (a0 & lo) | ((a1 << 4) & ~lo), ao = ((a0 >> 4) & lo) | (a1 & ~lo);
                const uint32_t be = (b0 & lo) | ((b1 << 4) & ~lo), bo = ((b0 >> 4) & lo) | (b1 & ~lo);
                pv<0>(4 * w, ae, ao, be, bo, va, vb, p[b]);
                pv<1>(4 * w + 1, ae, ao, be, bo, va, vb, p[b]);
                pv<2>(4 * w + 2, ae, ao, be, bo, va, vb, p[b]);
                pv<3>(4 * w + 3, ae, ao, be, bo, va, vb, p[b]);
            }
        }
    }
    template <int kB>
    __device__ __forceinline__ void pv(int i, uint32_t ae, uint32_t ao, uint32_t be, uint32_t bo, __half2 va, __half2 vb,
                                       const uint32_t (&p)[kNt][2]) {
        const uint32_t f[4] = {as_u32(__hmul2(kv4_pair<kB>(ae), va)), as_u32(__hmul2(kv4_pair<kB>(ao), va)),
                               as_u32(__hmul2(kv4_pair<kB>(be), vb)), as_u32(__hmul2(kv4_pair<kB>(bo), vb))};
#pragma unroll
        for (int n = 0; n < kNt; ++n) mma_f16(o[n][i], f, p[n][0], p[n][1]);
    }

    // A partial, 32 lanes side by side: O, then (m, l) and mul of each 8 rows.
    static constexpr int kVecs = kNt * (kK + 2);
    __device__ __forceinline__ void store(float4 *to, int lane) const {
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
#pragma unroll
            for (int i = 0; i < kK; ++i) to[(n * kK + i) * 32 + lane] = make_float4(o[n][i][0], o[n][i][1], o[n][i][2], o[n][i][3]);
            to[(kNt * kK + n) * 32 + lane] = make_float4(m[n].x, m[n].y, l[n].x, l[n].y);
            to[(kNt * (kK + 1) + n) * 32 + lane] = make_float4(mul[n].x, mul[n].y, 0.0f, 0.0f);
        }
    }
    static __device__ __forceinline__ void factors(float m, float n, float mul, float *to, float *f, float *g) {
        *to = fmaxf(m, n);
        *f = against(m, *to, mul);
        *g = against(n, *to, mul);
    }
    struct Loaded {
        float4 o[kK], st;
    };
    static __device__ __forceinline__ void load(const float4 *from, int n, Loaded &x, int lane) {  // a partial's 8 rows n
#pragma unroll
        for (int i = 0; i < kK; ++i) x.o[i] = from[(n * kK + i) * 32 + lane];
        x.st = from[(kNt * kK + n) * 32 + lane];
    }
    __device__ __forceinline__ void join(int n, const Loaded &x) {
        float fx, fy, gx, gy;
        factors(m[n].x, x.st.x, mul[n].x, &m[n].x, &fx, &gx);
        factors(m[n].y, x.st.y, mul[n].y, &m[n].y, &fy, &gy);
        l[n] = make_float2(l[n].x * fx + x.st.z * gx, l[n].y * fy + x.st.w * gy);
#pragma unroll
        for (int i = 0; i < kK; ++i) {
            o[n][i][0] = o[n][i][0] * fx + x.o[i].x * gx;
            o[n][i][1] = o[n][i][1] * fy + x.o[i].y * gy;
            o[n][i][2] = o[n][i][2] * fx + x.o[i].z * gx;
            o[n][i][3] = o[n][i][3] * fy + x.o[i].w * gy;
        }
    }

    // V scales of tokens that no row sees become zero, and those that are no
    // number too: the rows that see their token become NaN here, in this lane's
    // columns, the others must not.
    __device__ __forceinline__ void guard(uint32_t &vs, int blk, const Span &at, int lane) {
        const int t = lane & 3, end = at.end - at.key0 - 16 * blk;
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tok = 8 * (i >> 1) + 2 * t + (i & 1);
            if (tok >= end) {
                vs &= ~(0xffu << (8 * i));
            } else if ((vs >> (8 * i) & 0x7fu) == 0x7fu) {
                vs &= ~(0xffu << (8 * i));
                bad |= 1u << tok;
            }
        }
        if (!__any_sync(0xffffffffu, bad != 0)) return;
        bad |= __shfl_xor_sync(0xffffffffu, bad, 1);  // the four lanes of one g: the same columns
        bad |= __shfl_xor_sync(0xffffffffu, bad, 2);
        const float nan = __uint_as_float(0x7fffffffu);
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int lim = at.sees(8 * n + 2 * t + c) - 16 * blk;
                const uint32_t sees = lim >= 16 ? 0xffffu : lim <= 0 ? 0u : (1u << lim) - 1;
                if (bad & sees)
#pragma unroll
                    for (int i = 0; i < kK; ++i) o[n][i][c] = o[n][i][c + 2] = nan;
            }
        }
    }
};

// A warp's ring of pairs of tiles.
template <int D, int kStg>
struct Ring {
    uint32_t buf, bar;              // shared addresses
    uint32_t take, take_parity;     // the next pair to be read
    uint32_t put;                   // the next one to be copied
    uint32_t out;                   // pairs on their way
    static constexpr uint32_t kPair = 2 * Kv4Tile<D>::kBytes;

    __device__ __forceinline__ uint32_t tile() const { return buf + take * kPair; }
    __device__ __forceinline__ uint32_t taking() const { return bar + 8 * take; }
    __device__ __forceinline__ void taken() {
        --out;
        if (++take == kStg) {
            take = 0;
            take_parity ^= 1;
        }
    }
    // Two lanes start a copy each, or say that there is none.
    __device__ __forceinline__ void start(int which, bool there, const uint8_t *src) {
        const uint32_t b = bar + 8 * put;
        if (which == 0 || which == 1) {
            if (there) {
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(b), "r"(Kv4Tile<D>::kBytes) : "memory");
                bulk_copy(buf + put * kPair + which * Kv4Tile<D>::kBytes, src, Kv4Tile<D>::kBytes, b);
            } else {
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(b) : "memory");
            }
        }
        ++out;
        if (++put == kStg) put = 0;
    }
};

struct Where {
    int r, i, h;      // request, tile, kv head
    Kv4Request q;
    long long start;  // the item's first position
};

// Of what another SM wrote. Volatile: such loads go out together, before their
// values are used.
__device__ __forceinline__ float4 far_load(const float4 *from) {
    float4 x;
    asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "l"(from) : "memory");
    return x;
}

// An item of which this CTA was the last to leave its part.
struct Far {
    int rows, nt;  // 0: none; the partials are of 8 nt rows
    int row0, token0, head;
    int first, last;  // the item's shares
};

// What an item's warps have in common, and this warp's place among the CTA's.
struct Team {
    int warp, cta, shares;  // shares of this CTA, one a warp
    int first, last;        // the item's shares
    bool begun, cut;        // it began in a share before this one, it ends in one behind
    Kv4Shares sh;
    float4 *area;           // a partial of each warp
    uint32_t q;             // shared address of this warp's q fragments (16 rows or more)
    volatile int *abort;
    bool met;               // this warp has been at the CTA's barrier
    Far *far;               // of the CTA: the item begun before it, the one that goes on behind it
    int *any_far;           // it has parts of such
};

template <int D, int kMaxNt>
struct Kernel {
    static constexpr int kStg = kStages<D, kMaxNt>;
    static constexpr int kW = kWarps<kMaxNt>;
    static constexpr int kRows = 8 * kMaxNt;
    static constexpr size_t kRing = (size_t)kW * kStg * 2 * Kv4Tile<D>::kBytes;
    static constexpr int kPart = Item<D, kMaxNt>::kVecs * 32;  // float4 of a partial
    // With 16 rows or more shared memory holds q's fragments, and the warps' partials
    // lie in the workspace (12 times 16 rows of them, or 8 times 32).
    static constexpr bool kAreaShared = kMaxNt == 1;
    static constexpr size_t kSmem = kRing + (size_t)kW * (kAreaShared ? kPart * 16 : kQBytes<D, kMaxNt>);

    // Blocks [b0, b1) of an item; false: a wait gave up.
    template <int kNt>
    static __device__ bool run(const Kv4Args &a, Ring<D, kStg> &ring, const Where &w, const Kv4Tiling &tl, int b0, int b1,
                               Team &team, int lane) {
        Item<D, kNt> it;
        it.q_at = team.q + 16 * lane;
        const int row0 = w.i * kRows, rows = tl.rows;
        const int32_t *ids = a.table + (long long)w.r * a.max_blocks;
        const uint8_t *heads = a.pool + (long long)w.h * Kv4Tile<D>::kBytes;
        const long long block_bytes = (long long)a.num_kv_heads * Kv4Tile<D>::kBytes;
        int bits = 0;
        // ids are looked up 32 at a time, the next 32 ahead; a lane copies its own block
        int have = b0 + lane < b1 ? __ldg(ids + b0 + lane) : 0;
        int next = b0 + 32 + lane < b1 ? __ldg(ids + b0 + 32 + lane) : 0;
        typename Item<D, kNt>::Rows q_rows;
        Item<D, kNt>::read_q(a, w.q.q0, row0, rows, w.h, q_rows, lane);
        int put = b0;  // next pair to copy
        auto start = [&]() {
            const int at = (put - b0) & 31;
            if (at == 0 && put > b0) {
                have = next;
                next = put + 32 + lane < b1 ? __ldg(ids + put + 32 + lane) : 0;
            }
            const bool bad = have < 0 || have >= a.num_blocks;
            if (bad) bits = PKV_DEV_BAD_BLOCK;
            ring.start(lane - at, put + lane - at < b1, heads + (bad ? 0 : have) * block_bytes);
            put += 2;
        };
#pragma unroll 1
        for (int i = 0; i < kStg && put < b1; ++i) start();
        it.begin(a, rows, q_rows, lane);
        if (Item<D, kNt>::kQShared) __syncwarp();
        const int tok0 = kv4_over(row0, a.group, a.group_inv);
        Span at{16 * b0, w.q.len - w.q.n + tok0 + 1, min(tl.keys, 16 * b1), row0, tok0, a.group, a.group_inv};
        auto between = [&]() {
            if (put < b1) start();
        };
#pragma unroll 1
        for (int b = b0; b < b1; b += 2, at.key0 += 32) {
            if (!warp_wait(ring.taking(), ring.take_parity, team.abort)) return false;
            const uint32_t tile = ring.tile();
            ring.taken();
            const bool masked = at.key0 + 32 > at.limit0 || b + 1 >= b1;
            float s[2][kNt][4];
            uint32_t p[2][kNt][2];
            it.scores(tile, s, lane);
            it.probabilities(s, masked, b == b0, at, p, lane);
            it.values(tile, masked, at, p, between, lane);
        }
        if (__any_sync(0xffffffffu, bits != 0) && lane == 0) raise_status(a.status, PKV_DEV_BAD_BLOCK);
        hand_over<kNt>(a, it, w, row0, rows, team, lane);
        return true;
    }

    // An item's end in this share: its output, or this share's part of it.
    template <int kNt>
    static __device__ __forceinline__ void hand_over(const Kv4Args &a, Item<D, kNt> &it, const Where &w, int row0, int rows,
                                                     Team &team, int lane) {
        const int base = team.cta * team.sh.per_cta;
        const bool leads = !team.begun || team.warp == 0;  // it has the first of the item's pieces in this CTA
        const bool far = team.first < base || team.last >= base + team.shares;
        if (leads && far && lane == 0) *team.any_far = 1;
        if (leads && team.cut) {
            team.met = true;
            __syncthreads();
            if (*team.abort) return;
            const int upto = min(team.last - base, team.shares - 1);
            for (int i = team.warp + 1; i <= upto; ++i)
#pragma unroll
                for (int g = 0; g < kNt; ++g) {
                    typename Item<D, kNt>::Loaded x;
                    Item<D, kNt>::load(team.area + i * kPart, g, x, lane);
                    it.join(g, x);
                }
        }
        if (!leads || far) {  // for the first of its warps in this CTA; or for another CTA
            const int c0 = team.first / team.sh.per_cta, n = team.last / team.sh.per_cta - c0 + 1;
            it.store(leads ? a.parts + ((size_t)2 * team.cta + (team.cta == c0)) * kPart : team.area + team.warp * kPart, lane);
            if (!leads) return;
            __syncwarp();
            if (lane == 0) {
                int seen;
                // releases this warp's partial, and takes the others' in
                asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(seen) : "l"(a.arrived + c0) : "memory");
                seen -= kKv4Nobody;
                if (seen == n - 1) {
                    atomicExch(a.arrived + c0, kKv4Nobody);
                    team.far[team.cta == c0] = Far{rows, kNt, row0, w.q.q0, w.h, team.first, team.last};
                }
                if (seen < 0 || seen >= n) raise_status(a.status, PKV_DEV_BAD_WORKSPACE);
            }
            return;
        }
        output<kNt>(a, it, w, row0, rows, lane);
    }

    // The parts of an item that several CTAs left, by all warps of the last of them:
    // one of the D / 16 steps of 8 rows at a time, kAhead parts on their way.
    static __device__ __forceinline__ void join_far(const Kv4Args &a, const Far &j, int per_cta, int warp, int lane) {
        constexpr int kK = D / 16, kAhead = 4;
        const int g = lane >> 2, t = lane & 3;
        const int c0 = j.first / per_cta, count = j.last / per_cta - c0 + 1;
        const float4 *lead = a.parts + ((size_t)2 * c0 + 1) * kPart + lane;
        auto part = [&](int c) { return lead + (c ? (size_t)(2 * c - 1) * kPart : 0); };
#pragma unroll 1
        for (int unit = warp; unit < j.nt * kK; unit += kW) {
            const int n = unit / kK, at = (j.nt * kK + n) * 32;
            const float4 mul = __ldcg(lead + at + 32 * j.nt);
            float mx = -INFINITY, my = -INFINITY, lx = 0.0f, ly = 0.0f;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
            for (int k0 = 0; k0 < count; k0 += kAhead) {
                float4 st[kAhead], x[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const float4 *from = part(min(k0 + k, count - 1));
                    st[k] = far_load(from + at);
                    x[k] = far_load(from + unit * 32);
                }
                float tx = mx, ty = my;
#pragma unroll
                for (int k = 0; k < kAhead; ++k) tx = fmaxf(tx, st[k].x), ty = fmaxf(ty, st[k].y);
                const float fx = against(mx, tx, mul.x), fy = against(my, ty, mul.y);
                mx = tx, my = ty;
                lx *= fx, ly *= fy;
                o = make_float4(o.x * fx, o.y * fy, o.z * fx, o.w * fy);
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const bool live = k0 + k < count;
                    const float gx = live ? against(st[k].x, tx, mul.x) : 0.0f, gy = live ? against(st[k].y, ty, mul.y) : 0.0f;
                    lx += st[k].z * gx, ly += st[k].w * gy;
                    o = make_float4(o.x + x[k].x * gx, o.y + x[k].y * gy, o.z + x[k].z * gx, o.w + x[k].w * gy);
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = c ? ly : lx;
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const int row = 8 * n + 2 * t + c;
                if (row >= j.rows) continue;
                const float f = __fdividef(a.v_scale, l);
                const int rr = j.row0 + row, tok = kv4_over(rr, a.group, a.group_inv);
                *reinterpret_cast<uint32_t *>(a.out + ((long long)(j.token0 + tok) * a.num_kv_heads * a.group + j.head * a.group + rr - tok * a.group) * D +
                                              D / 8 * g + 2 * (unit - n * kK)) = c ? pack_bf16x2(o.y * f, o.w * f) : pack_bf16x2(o.x * f, o.z * f);
            }
        }
    }

    template <int kNt>
    static __device__ __forceinline__ void output(const Kv4Args &a, Item<D, kNt> &it, const Where &w, int row0, int rows, int lane) {
        constexpr int kC = D / 8;  // columns a lane holds
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = c ? it.l[n].y : it.l[n].x;
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const int row = 8 * n + 2 * t + c;
                if (row >= rows) continue;
                const float f = __fdividef(a.v_scale, l);
                const int rr = row0 + row, tok = kv4_over(rr, a.group, a.group_inv);
                uint4 *to = reinterpret_cast<uint4 *>(
                    a.out + ((long long)(w.q.q0 + tok) * a.num_kv_heads * a.group + w.h * a.group + rr - tok * a.group) * D + kC * g);
#pragma unroll
                for (int i = 0; i < kC / 8; ++i)
                    to[i] = make_uint4(pack_bf16x2(it.o[n][4 * i][c] * f, it.o[n][4 * i][c + 2] * f),
                                       pack_bf16x2(it.o[n][4 * i + 1][c] * f, it.o[n][4 * i + 1][c + 2] * f),
                                       pack_bf16x2(it.o[n][4 * i + 2][c] * f, it.o[n][4 * i + 2][c + 2] * f),
                                       pack_bf16x2(it.o[n][4 * i + 3][c] * f, it.o[n][4 * i + 3][c + 2] * f));
            }
        }
    }
};

template <int D, int kMaxNt>
__global__ void __launch_bounds__(32 * kWarps<kMaxNt>, 1) kv4_attention_kernel(const Kv4Args a) {
    using K = Kernel<D, kMaxNt>;
    constexpr int kThreads = 32 * K::kW;
    extern __shared__ __align__(128) uint8_t s_mem[];  // rings, then a partial of each warp
    __shared__ __align__(8) uint64_t s_bar[K::kW * K::kStg];
    __shared__ long long s_sum[kThreads], s_warp[K::kW];
    __shared__ int s_abort, s_most[K::kW], s_any_far;
    __shared__ Far s_far[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
    for (int i = tid; i < K::kW * K::kStg; i += kThreads) mbar_init(s_bar + i, 2);
    if (tid == 0) s_abort = s_any_far = s_far[0].rows = s_far[1].rows = 0;
    mbar_fence_init();
    pdl_launch_dependents();
    pdl_wait();

    // The costs of all requests: `each` of them a thread, in order; of those that the
    // chunk kernel may have, apart.
    const int each = (a.num_reqs + kThreads - 1) / kThreads;
    long long sum = 0, theirs = 0;
    bool skip = false;  // they are the chunk kernel's
    int bits = 0;
    {
        int most = 0;
        long long units = 0, items = 0;
        for (int r = tid * each; r < min((tid + 1) * each, a.num_reqs); ++r) {
            const Kv4Request q = kv4_request_of(a, r, K::kRows, &bits);
            const long long cost = kv4_cost(q, a.num_kv_heads, q.tiles);
            if (kMaxNt == 4 && a.chunks && kv4_is_chunk(q, a.group)) {
                theirs += cost;
                const Kv4Request c = kv4_request(q.q0, q.n, q.len, a.group, kKv4ChunkRows);
                units += kv4_chunk_units(c, a.num_kv_heads);
                items += (long long)c.tiles * a.num_kv_heads;
                most = max(most, kv4_chunk_tiles(q.len));
            } else {
                sum += cost;
            }
        }
        if (cta == 0 && bits) raise_status(a.status, bits);
        if (kMaxNt == 4 && a.chunks) {
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                units += __shfl_xor_sync(0xffffffffu, units, d);
                items += __shfl_xor_sync(0xffffffffu, items, d);
                most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
            }
            if (lane == 0) {
                s_warp[warp] = units;
                s_sum[warp] = items;
                s_most[warp] = most;
            }
            __syncthreads();
            units = items = most = 0;
            for (int i = 0; i < K::kW; ++i) {
                units += s_warp[i];
                items += s_sum[i];
                most = max(most, s_most[i]);
            }
            __syncthreads();
            skip = kv4_use_chunks(units, most, kv4_splits(items, gridDim.x));
        }
        if (!skip) sum += theirs;
    }
    auto request = [&](int r) {
        int none = 0;
        Kv4Request q = kv4_request_of(a, r, K::kRows, &none);
        if (kMaxNt == 4 && skip && kv4_is_chunk(q, a.group)) q.tiles = 0;
        return q;
    };
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
    }
    if (lane == 31) s_warp[warp] = sum;
    s_sum[tid] = sum;  // of its warp's requests
    if (__syncthreads_or(bits & PKV_DEV_BAD_QSL)) {
        if (kv4_overlap<kThreads>(a, each, s_sum)) return;
        s_sum[tid] = sum;
        __syncthreads();
    }
    long long total = 0;
#pragma unroll
    for (int i = 0; i < K::kW; ++i) total += s_warp[i];

    Team team;
    team.sh = kv4_shares(total, (int)gridDim.x, K::kW, kv4_least(K::kRows), a.num_reqs, a.num_kv_heads);
    team.warp = warp;
    team.cta = cta;
    team.shares = min(team.sh.per_cta, team.sh.count - cta * team.sh.per_cta);
    team.area = K::kAreaShared ? reinterpret_cast<float4 *>(s_mem + K::kRing)
                               : a.parts + (size_t)2 * gridDim.x * K::kPart + (size_t)cta * K::kW * K::kPart;
    team.q = smem_u32(s_mem + K::kRing) + warp * kQBytes<D, kMaxNt>;
    team.abort = &s_abort;
    team.met = false;
    team.far = s_far;
    team.any_far = &s_any_far;
    if (team.shares <= 0) return;
    if (warp < team.shares) {
        const int share = cta * team.sh.per_cta + warp;
        const long long from = team.sh.begin(share);
        Where w;
        {
            // the thread whose requests `from` lies in: its warp, then by a vote the lane
            long long first = 0;
            int run = 0;
#pragma unroll
            for (int i = 0; i < K::kW - 1; ++i)
                if (first + s_warp[i] <= from && run == i) {
                    first += s_warp[i];
                    ++run;
                }
            const int in = __ffs(__ballot_sync(0xffffffffu, first + s_sum[run * 32 + lane] > from)) - 1;
            if (in) first += s_sum[run * 32 + in - 1];
            const int lo = run * 32 + in;
            for (w.r = lo * each;; ++w.r) {  // of its requests, the one that `from` lies in
                w.q = request(w.r);
                const long long cost = kv4_cost(w.q, a.num_kv_heads, w.q.tiles);
                if (from < first + cost) break;
                first += cost;
            }
            kv4_locate(w.q, a.num_kv_heads, from - first, &w.i, &w.h, &w.start);
            w.start += first;
        }
        Ring<D, K::kStg> ring{smem_u32(s_mem) + (uint32_t)warp * K::kStg * Ring<D, K::kStg>::kPair, smem_u32(s_bar + warp * K::kStg), 0, 0, 0, 0};
        while (true) {
            const Kv4Tiling tl = kv4_tile(w.q, w.i, a.group, K::kRows);
            const long long cost = kv4_item_cost(w.q, w.i);
            const Kv4Piece p = kv4_piece(team.sh, share, w.start, cost, tl.blocks);
            if (p.b0 < p.b1) {
                team.begun = p.begun, team.cut = p.cut, team.first = p.first, team.last = p.last;
                bool ok;
                if (kMaxNt == 1 || tl.rows <= 8) ok = K::template run<1>(a, ring, w, tl, p.b0, p.b1, team, lane);
                else if (kMaxNt == 2 || tl.rows <= 16) ok = K::template run<kMaxNt >= 2 ? 2 : 1>(a, ring, w, tl, p.b0, p.b1, team, lane);
                else ok = K::template run<kMaxNt>(a, ring, w, tl, p.b0, p.b1, team, lane);
                if (!ok) {
                    // nothing may still be on its way into this SM's memory when the CTA ends
                    int never = 0;
                    for (; ring.out; ring.taken())
                        if (!warp_wait(ring.taking(), ring.take_parity, &never)) break;
                    if (lane == 0) raise_status(a.status, PKV_DEV_TIMEOUT);
                    break;
                }
            }
            if (!p.more) break;
            w.start += cost;
            if (++w.h == a.num_kv_heads) {
                w.h = 0;
                if (++w.i == w.q.tiles) {
                    w.i = 0;
                    do {
                        w.q = request(++w.r);
                    } while (w.q.tiles == 0);  // one follows: positions up to `to` belong to requests
                }
            }
        }
    }
    if (!team.met) __syncthreads();
    if (!s_any_far) return;
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < 2; ++k)
        if (s_far[k].rows) K::join_far(a, s_far[k], team.sh.per_cta, warp, lane);
}

// Places in the workspace, for any batch and form (the chunk kernel has left its
// parts before the other one begins).
size_t parts_at(int sms) { return (((size_t)sms + 1) * sizeof(int) + 255) / 256 * 256; }
size_t workspace_bytes(int sms, int head_size) {
    const size_t chunks = (size_t)kKv4ChunkCtas * sms * kv4_chunk_part(head_size) * sizeof(float);
    return parts_at(sms) + std::max(chunks, (size_t)sms * sizeof(float4) * (head_size == 128 ? 2 * Kernel<128, 4>::kPart + kWarps<4> * Kernel<128, 4>::kPart
                                                                            : 2 * Kernel<64, 4>::kPart + kWarps<4> * Kernel<64, 4>::kPart));
}

std::mutex g_mu;
bool g_ready[64][2][3];

template <int D, int kMaxNt>
int launch(const Kv4Args &a, int sms, int which, cudaStream_t st) {
    using K = Kernel<D, kMaxNt>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_E_CUDA;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        if (!g_ready[dev][D == 128][which]) {
            if (cudaFuncSetAttribute(kv4_attention_kernel<D, kMaxNt>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)K::kSmem) != cudaSuccess)
                return PKV_E_CUDA;
            g_ready[dev][D == 128][which] = true;
        }
    }
    if (launch_pdl(kv4_attention_kernel<D, kMaxNt>, dim3(sms), dim3(32 * K::kW), K::kSmem, st, a) != cudaSuccess)
        return PKV_E_CUDA;
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" PKV_API int paged_kv4_attention_workspace_bytes(const pkv_cache_desc *desc, size_t *bytes) {
    if (!desc || !bytes) return PKV_E_NULL;
    const int rc = check_cache_desc(*desc, /*attention=*/true);
    if (rc) return rc;
    int sms = 0;
    const int rs = device_sms(&sms);
    if (rs) return rs;
    *bytes = workspace_bytes(sms, desc->head_size);
    return PKV_OK;
}

extern "C" PKV_API int paged_kv4_attention_init(const pkv_cache_desc *desc, void *workspace, size_t workspace_size,
                                                void *stream) {
    if (!desc) return PKV_E_NULL;
    const int rc = check_cache_desc(*desc, /*attention=*/true);
    if (rc) return rc;
    if (!workspace) return PKV_E_NULL;
    if (!aligned(workspace, 16)) return PKV_E_ALIGN;
    int sms = 0;
    const int rs = device_sms(&sms);
    if (rs) return rs;
    if (workspace_size < workspace_bytes(sms, desc->head_size)) return PKV_E_WORKSPACE;
    return cudaMemsetAsync(workspace, kKv4Nobody & 0xff, parts_at(sms), static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_E_CUDA;
}

extern "C" PKV_API int paged_kv4_attention(const void *q, int64_t q_stride, int32_t num_tokens, int32_t num_q_heads,
                                           const void *kv4_cache, const pkv_cache_desc *desc,
                                           const int32_t *block_table, int32_t num_reqs, int32_t max_blocks_per_req,
                                           const int32_t *seq_lens, const int32_t *query_start_loc,
                                           int32_t max_query_len, float scale, float k_scale, float v_scale, void *out,
                                           void *workspace, size_t workspace_size, int32_t *status, void *stream) {
    if (!desc) return PKV_E_NULL;
    const int rc = check_cache_desc(*desc, /*attention=*/true);
    if (rc) return rc;
    if (num_tokens < 0 || num_reqs < 0 || max_blocks_per_req < 0 || max_query_len < 0) return PKV_E_DIMS;
    if (max_blocks_per_req > INT32_MAX / PKV_BLOCK_SIZE || num_reqs > INT32_MAX - 65536) return PKV_E_DIMS;
    if (num_q_heads <= 0 || num_q_heads % desc->num_kv_heads) return PKV_E_GQA;
    const int group = num_q_heads / desc->num_kv_heads;
    if (group > 128 || (long long)num_tokens * group > INT32_MAX - 1024) return PKV_E_DIMS;
    if (!(scale > 0.0f && scale <= 1e30f) || !kv4_scale_ok(k_scale) || !kv4_scale_ok(v_scale)) return PKV_E_DIMS;
    if (q_stride % 8 || q_stride < 0 || (num_tokens > 1 && q_stride < (int64_t)num_q_heads * desc->head_size))
        return PKV_E_DIMS;
    if (num_tokens == 0 || num_reqs == 0) return PKV_OK;
    if (!q || !kv4_cache || !block_table || !seq_lens || !query_start_loc || !out || !workspace) return PKV_E_NULL;
    if (!aligned(q, 16) || !aligned(kv4_cache, 16) || !aligned(out, 16) || !aligned(workspace, 16) ||
        !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) || !aligned(status, 4))
        return PKV_E_ALIGN;
    if (out == q) return PKV_E_DIMS;
    int sms = 0;
    const int rs = device_sms(&sms);
    if (rs) return rs;
    if (workspace_size < workspace_bytes(sms, desc->head_size)) return PKV_E_WORKSPACE;
    // Below 2^-126 the product would keep few bits or none, but with q near the largest values
    // there are scores of any size: 2^96 of it goes to q's powers of two then.
    const double product = scale * 1.4426950408889634 * k_scale;
    const bool tiny = product < 0x1p-126;
    const float small = tiny ? 0x1p-96f : 1.0f;
    const float scale_log2 = tiny ? (float)(product * 0x1p96) : scale * 1.4426950408889634f * k_scale;
    if (!std::isfinite(scale_log2)) return PKV_E_DIMS;
    // rows that the longest request has of a kv head
    const long long rows = (long long)(max_query_len ? max_query_len : num_tokens) * group;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const Kv4Args a{static_cast<const __nv_bfloat16 *>(q), q_stride, static_cast<const uint8_t *>(kv4_cache), block_table,
                    seq_lens, query_start_loc, num_tokens, desc->num_kv_heads, group, num_reqs, max_blocks_per_req,
                    desc->num_blocks, kv4_inverse(group), scale_log2, small, v_scale, static_cast<__nv_bfloat16 *>(out),
                    reinterpret_cast<int *>(ws), reinterpret_cast<int *>(ws) + 1, reinterpret_cast<float4 *>(ws + parts_at(sms)),
                    rows >= 64, status};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a.chunks) {
        const int rl = kv4_chunk_launch(a, desc->head_size, sms, st);
        if (rl) return rl;
    }
    if (desc->head_size == 128)
        return rows <= 8 ? launch<128, 1>(a, sms, 0, st) : rows <= 16 ? launch<128, 2>(a, sms, 1, st) : launch<128, 4>(a, sms, 2, st);
    return rows <= 8 ? launch<64, 1>(a, sms, 0, st) : rows <= 16 ? launch<64, 2>(a, sms, 1, st) : launch<64, 4>(a, sms, 2, st);
}
