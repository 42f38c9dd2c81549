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
// Cache row of one token and KV head: 64 bytes of codes in four 16-byte
// segments, one for each group of 32 dimensions, and 4 bf16 scales. Dimension
// d = 32 i + 8 q + r (i, q in 0..3, r in 0..7) is nibble q of 16-bit word r of
// segment i. That is the layout ldmatrix wants of both operands: of eight
// tokens' segments i it gives lane (g, c) the word 2c, 2c + 1 of token g (keys:
// dimension pairs of token g), or transposed the words g of tokens 2c, 2c + 1
// (values: token pairs of dimension g), each time four operand pairs in one
// register. Segment i stands at place i ^ (offset / 2 % 4), offset the token's
// place in its block: eight consecutive tokens' segments i then lie in all the
// shared-memory banks, also when a block is copied there as it is.
#pragma once
#include <cstdint>

namespace bi {

constexpr int kI4Row = 64;                     // code bytes of a cache row
constexpr int kI4Scales = 4;                   // scales of a cache row
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
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w >> (4 * Q)), "r"(0x000F000Fu), "r"(0x43004300u));
    return d;
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

// Whether a group with this scale holds numbers (else its values are NaN).
__device__ __forceinline__ bool i4_finite(uint16_t scale) { return (scale & 0x7F80u) != 0x7F80u; }

// Place of segment i in the code row of a token at this offset of its block.
__device__ __forceinline__ int i4_place(int i, int offset) { return i ^ ((offset >> 1) & 3); }

}  // namespace bi
