// attn_common.cuh -- what the attention kernels over the bf16 and the 4-bit
// cache share: the chunk size, the tensor-core products and the chunk merge.
// One definition of each keeps their results the same bits.
#pragma once
#include <cstdint>

#include "bi_ptx.cuh"

namespace bi {

constexpr int kD = 128;
constexpr int kChunk = 128;                    // tokens per chunk: fixed, by position
// Over the 4-bit cache: the maximum of a chunk of which a row sees no token in
// the cache (its blocks lie outside). The least number, so that the chunk's sums,
// which are 0, leave every other chunk's weight as it is, whatever its scores;
// with -inf its exponentials would be NaN, as they have to be where the scores of
// tokens in the cache are all -inf (bi_attention_decode gives NaN there).
constexpr float kNoScore = -0x1.fffffep127f;

// 16-byte global -> shared copy; src_bytes = 0 writes 16 zero bytes and reads nothing.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
// The same with 8 bytes.
__device__ __forceinline__ void cp_async_8(uint32_t dst, const void *src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// D += A B on the tensor cores, one warp: A 16x16 bf16 (row-major fragment
// a0..a3), B 16x8 bf16 (column fragment b0, b1), D 16x8 fp32.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four 8x8 bf16 matrices from shared memory, transposed (lanes 8i..8i+7 give
// the 16-byte rows of matrix i).
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3,
                                                  uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(addr));
}
// Four 8x8 bf16 matrices from shared memory (lanes 8i..8i+7 give the 16-byte
// rows of matrix i); lane (g, c) receives row g, columns 2c and 2c+1 of each.
__device__ __forceinline__ void ldmatrix_x4(uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(addr));
}
// (p0, p1) = hi + lo, hi and lo packed bf16 pairs (round to nearest even);
// hi + lo carries 16 significant bits of each p.
__device__ __forceinline__ void split_bf16x2(float p0, float p1, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16x2(__float_as_uint(p0), __float_as_uint(p1));
    const float h0 = __uint_as_float(hi << 16), h1 = __uint_as_float(hi & 0xFFFF0000u);
    lo = pack_bf16x2(__float_as_uint(p0 - h0), __float_as_uint(p1 - h1));
}

// Merge one chunk's (m_c, l_c, o_c) into the running (m, l, o) of a query
// row, in chunk order: m' = max(m, m_c); o = o e^{m - m'} + o_c e^{m_c - m'},
// l likewise (the first chunk finds m = -inf, l = o = 0). Decode and extend
// attention both merge through this one definition.
__device__ __forceinline__ void merge_factors(float m, float m_c, float &m_new, float &alpha, float &beta) {
    m_new = fmaxf(m, m_c);
    alpha = expf(__fsub_rn(m, m_new));
    beta = expf(__fsub_rn(m_c, m_new));
}
__device__ __forceinline__ float merge_value(float run, float chunk, float alpha, float beta) {
    return __fmaf_rn(chunk, beta, __fmul_rn(run, alpha));
}

}  // namespace bi
