// The 4-bit KV pool: its tile layout and the conversions to and from it.
//
// A value is an e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) times the
// e4m3 scale of its 16 columns, and times the call's k_scale or v_scale, a
// power of two. Code times scale has six significant bits at most and lies in
// [2^-10, 2688] or is zero, so it is exact in fp16 and in bf16.
//
// One (block, kv head) is a tile of 18 * D bytes: K codes (8 D), V codes (8 D),
// K scales (D), V scales (D). Every part but the first is in the order in which
// the lanes of a warp want it as fragments of m16n8k16 (lane 4 g + t, g < 8, t
// < 4), so that a warp reads a part with one or two loads, lane by lane, and
// nothing has to be moved between lanes. A byte of codes holds an even column
// (low four bits) and the next one of one token, so that a token is written
// without touching another's bits.
//   K codes   [token][D / 2]; lane (g, t): tokens g and g + 8, columns of the
//             t-th quarter (the sum over columns does not care for their order)
//   V codes   [half][g][t][e][D / 16]: token 8 half + 2 t + e, the g-th eighth
//             of the columns
//   K scales  [g][t][half][D / 64]: token 8 half + g, groups of the t-th quarter
//   V scales  [group][t][half][e]: token 8 half + 2 t + e
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "pkv_device.cuh"

namespace pkv {

template <int D>
struct Kv4Tile {
    static constexpr int kBytes = 18 * D;
    static constexpr int kV = 8 * D, kKScale = 16 * D, kVScale = 17 * D;

    // Byte offsets of a token's row: the codes of columns 8 c .. 8 c + 7 (four
    // bytes) and the scale of columns 16 g .. 16 g + 15.
    __host__ __device__ static constexpr int k_code(int row, int c) { return row * (D / 2) + 4 * c; }
    __host__ __device__ static constexpr int v_code(int row, int c) {
        // D 128: an eighth is two such chunks; D 64: one
        return kV + (row >> 3) * (4 * D) + (D == 128 ? c >> 1 : c) * (D / 2) + ((row >> 1) & 3) * (D / 8) +
               (row & 1) * (D / 16) + (D == 128 ? (c & 1) * 4 : 0);
    }
    __host__ __device__ static constexpr int k_scale(int row, int g) {
        return kKScale + (row & 7) * (D / 8) + g / (D / 64) * (D / 32) + (row >> 3) * (D / 64) + g % (D / 64);
    }
    __host__ __device__ static constexpr int v_scale(int row, int g) {
        return kVScale + g * 16 + ((row >> 1) & 3) * 4 + (row >> 3) * 2 + (row & 1);
    }
};

// Both codes of byte kByte of w as fp16.
template <int kByte>
__device__ __forceinline__ __half2 kv4_pair(uint32_t w) {
    uint32_t h;
    if constexpr (kByte == 0)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(h) : "r"(w));
    else if constexpr (kByte == 1)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(w));
    else if constexpr (kByte == 2)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(h) : "r"(w));
    else
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(h) : "r"(w));
    return *reinterpret_cast<__half2 *>(&h);
}

// Two scales (the low 16 bits of w) as fp16.
__device__ __forceinline__ __half2 kv4_scales(uint32_t w) {
    uint32_t h;
    asm("{\n\t.reg .b16 s;\n\tcvt.u16.u32 s, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, s;\n\t}" : "=r"(h) : "r"(w));
    return *reinterpret_cast<__half2 *>(&h);
}

// A power of two that the pool's scales are multiplied by.
inline bool kv4_scale_ok(float s) {
    if (!(s >= 0x1p-60f && s <= 0x1p60f)) return false;
    uint32_t bits;
    __builtin_memcpy(&bits, &s, 4);
    return (bits & 0x7fffff) == 0;
}

}  // namespace pkv
