// The format of a cache in 4 bits: a row (block, KV head, offset) has 64 bytes, K
// then V, element 2i in the low half of byte i, and four bf16 scales, of the 32
// elements 0 to 31 and 32 to 63 of K, then of V.  A half-byte c stands for (c - 8)
// times its scale.
//
// A scale has four significant bits and c - 8 three, so that every value is a
// bf16 number: what is read needs no rounding, and one multiply-add of bf16 pairs
// makes it, (128 + c) s - 136 s with 128 + c the bf16 number 0x4300 | c: 136 s = 17 * 8 s
// has eight significant bits, so has the result, and the sum is rounded once.
#pragma once
#include "rc_internal.cuh"

namespace rc {

constexpr int kKv4Row = 64;            // bytes of K and V of a row
constexpr int kKv4Scales = 4;          // their scales
constexpr uint32_t kKv4MostScale = 0x7180u;     // 2^100 as bf16

// A pair of scales as they count: without a sign, of four significant bits, and at
// most 2^100 (which takes infinities and NaN in, so that no value is either).
__device__ __forceinline__ uint32_t kv4_scales(uint32_t two) {
    return __vminu2(two & 0x7FF07FF0u, kKv4MostScale | kKv4MostScale << 16);
}

// (a0 * b0 + c0, a1 * b1 + c1) of bf16 pairs, and their product
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// -136 times a pair of scales
__device__ __forceinline__ uint32_t kv4_offsets(uint32_t two) { return mul_bf16x2(two, 0xC308C308u); }

// Half-bytes i and i + 4 of a word as the bf16 numbers 128 + c.
__device__ __forceinline__ uint32_t kv4_pair(uint32_t word, int i) {
    return ((word >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
}

}  // namespace rc
