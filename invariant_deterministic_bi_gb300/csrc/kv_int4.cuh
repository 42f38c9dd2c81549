// kv_int4.cuh -- the 4-bit formats: codes, scales and their expansion to bf16.
//
// A code is u = n + 8 for an integer n in -7..7 (cache) or any u in 0..15
// (weights). As bf16, the bits 0x4300 | u are the number 128 + u exactly (its
// unit in the last place is 1), so one shift and one three-input logic
// operation turn two codes of a 32-bit word into a bf16 pair, with no
// conversion instruction:  (w >> 4q) & 0x000F000F | 0x43004300.
//
// A cache scale s has four significant bits. Then 136 s = 17 * 8 s has at most
// eight, so c = -136 s is a bf16 number, and
//   fma(128 + u, s, c) = (u - 8) s
// rounds nothing: (u - 8) s has at most 3 + 4 bits. A cached value is therefore
// one fused multiply-add on a pair, and it is a bf16 number exactly: attention
// over the 4-bit cache multiplies the same operands as attention over a bf16
// cache holding those values.
//
// Cache row of one token and KV head: 64 bytes of codes, 4 bf16 scales (one per
// 32 dimensions). Dimension d = 32 i + 8 q + r (i, q in 0..3, r in 0..7) is
// nibble q of the row's 16-bit word number
//   K:  8 (r / 2) + 2 i + r % 2        V:  4 r + i
// so that the lanes of a warp find their operands of the tensor-core products
// in contiguous bytes: lane (row g, column pair c) of q.k takes the 16 bytes
// r / 2 = c (all eight 16-dimension steps), lane (row g, column pair c) of p.v
// the 8 bytes r = g (its row of all eight 16-dimension tiles).
#pragma once
#include <cstdint>

namespace bi {

constexpr int kI4Row = 64;                     // code bytes of a cache row
constexpr int kI4Scales = 4;                   // scales of a cache row
constexpr int kI4Group = 32;                   // dimensions that share a scale
constexpr uint32_t kBf16x2_m136 = 0xC308C308u; // (-136, -136)

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
// (128 + u, 128 + u') of nibble Q of the word's two halves.
template <int Q>
__device__ __forceinline__ uint32_t i4_pair(uint32_t w) {
    return ((w >> (4 * Q)) & 0x000F000Fu) | 0x43004300u;
}
// The four pairs (u - 8) s of a word of eight codes; s2 the halves' scales,
// c2 = -136 s2.
__device__ __forceinline__ void i4_expand(uint32_t w, uint32_t s2, uint32_t c2, uint32_t (&v)[4]) {
    v[0] = fma_bf16x2(i4_pair<0>(w), s2, c2);
    v[1] = fma_bf16x2(i4_pair<1>(w), s2, c2);
    v[2] = fma_bf16x2(i4_pair<2>(w), s2, c2);
    v[3] = fma_bf16x2(i4_pair<3>(w), s2, c2);
}
// Both halves = the low (hi = 0) or high (hi = 1) 16 bits of w.
template <int HI>
__device__ __forceinline__ uint32_t dup16(uint32_t w) { return __byte_perm(w, 0, HI ? 0x3232 : 0x1010); }
// (low halves of a and b) or (high halves): a's in the low half.
template <int HI>
__device__ __forceinline__ uint32_t zip16(uint32_t a, uint32_t b) { return __byte_perm(a, b, HI ? 0x7632 : 0x5410); }

}  // namespace bi
