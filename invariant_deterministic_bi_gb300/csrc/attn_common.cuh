// attn_common.cuh -- what the attention kernels over the bf16 and the 4-bit
// cache share: the chunk size, the tensor-core products and the chunk merge.
// One definition of each keeps their results the same bits.
#pragma once
#include <cstdint>
#include <type_traits>

#include "bi_ptx.cuh"

namespace bi {

constexpr int kD = 128;
constexpr int kChunk = 128;                    // tokens per chunk: fixed, by position
constexpr int kRowBytes = kD * 2;              // one token's K (or V) row of one KV head
constexpr int kTileBytes = kChunk * kRowBytes; // 32 KB
constexpr int kHalfTile = kChunk * 128;        // one 64-dimension half of a K or V tile (128-byte swizzle)
// Over the 4-bit cache and with a window: the maximum of a chunk of which a row sees
// no token in the cache (its blocks lie outside). The least number, so that the chunk's sums,
// which are 0, leave every other chunk's weight as it is, whatever its scores;
// with -inf its exponentials would be NaN, as they have to be where the scores of
// tokens in the cache are all -inf (bi_attention_decode gives NaN there).
constexpr float kNoScore = -0x1.fffffep127f;

// Byte offset of 16-byte piece x (0..15) of token row t in a swizzled K or V tile.
__device__ __forceinline__ int kv_piece(int t, int x) {
    return (x >> 3) * kHalfTile + t * 128 + (((x & 7) ^ (t & 7)) << 4);
}

// Sliding window: a token at position p sees the tokens j <= p with j > p - window
// or j < sinks. For the earliest of some tokens (its length n, n - window = from)
// and all after it: first tokens [0, first), then from `lo` on; of the chunks,
// the `ns` that hold first tokens before lo's chunk c0, then c0 and the rest.
struct Seen {
    int first, lo, ns, c0;
    __device__ __forceinline__ Seen(int from, int sinks) {
        lo = max(0, from);
        first = min(sinks, lo);
        c0 = lo / kChunk;
        ns = min((first + kChunk - 1) / kChunk, c0);
    }
    __device__ __forceinline__ int chunks(int n) const { return ns + (n + kChunk - 1) / kChunk - c0; }
    __device__ __forceinline__ int start(int i) const { return (i < ns ? i : c0 + i - ns) * kChunk; }   // of the i-th chunk
    __device__ __forceinline__ bool has(int j) const { return j < first || j >= lo; }
};

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

// bar.sync on the named barrier (1 + grp) of consumer group grp's GW warps
template <int GW>
__device__ __forceinline__ void group_sync(int grp) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * GW) : "memory");
}
// the same barrier with an OR vote over the group's threads
template <int GW>
__device__ __forceinline__ bool group_sync_or(int grp, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(pred)), "r"(1 + grp), "n"(32 * GW)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ bool finite_pair(uint32_t x) { return (x & 0x7F80u) != 0x7F80u && (x & 0x7F800000u) != 0x7F800000u; }

// The merge of a query row's chunk records (m, l, o[kD]) in chunk order by a CTA
// of kD threads, one per dimension: the output's bf16 bits. The first tile's values
// are loaded by the caller: o of dimension threadIdx.x, and (m, l) of record threadIdx.x.
// Chunks in tiles of 32. Every thread issues the tile's o loads of its
// dimension d at once; meanwhile warp 0 loads the tile's (m_c, l_c), one
// chunk per lane: the running maximum before chunk c is a prefix maximum
// (exact in any order: a shuffle scan), and chunk c's merge factors
// depend only on it and m_c, so each lane computes its chunk's factors.
// Then each thread merges its o values in chunk order: the same
// operations, in the same order, as a sequential walk over the chunks.
constexpr int kMergeTile = 32;
struct MergeTile {
    float fa[kMergeTile], fb[kMergeTile], fl[kMergeTile];   // alpha, beta and l of the tile's chunks
};
__device__ __forceinline__ uint16_t merge_records(const float *w, int nc, const float (&first)[kMergeTile], float mc0, float lc0,
                                                  MergeTile &t) {
    const int d = threadIdx.x;
    float o = 0.0f, l = 0.0f, m_run = -INFINITY;           // m_run: warp 0's copy of the running maximum
    // merge chunks c0 .. c0 + nt - 1 (their o values in ov; (m_c, l_c) of
    // chunk c0 + d in warp 0's lane d)
    auto merge_tile = [&](const float (&ov)[kMergeTile], int nt, float mc, float lc) {
        __syncthreads();                                   // previous tile fully consumed
        if (d < 32) {
            mc = d < nt ? mc : -INFINITY;
            lc = d < nt ? lc : 0.0f;
            float incl = mc;                               // max(m_c0 .. m_c) over the tile
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float v = __shfl_up_sync(0xffffffffu, incl, off);
                if (d >= off) incl = fmaxf(incl, v);
            }
            float before = __shfl_up_sync(0xffffffffu, incl, 1);
            before = d == 0 ? m_run : fmaxf(m_run, before);   // running maximum before chunk c0 + d
            float mn, a, bt;
            merge_factors(before, mc, mn, a, bt);
            if (d < nt) {
                t.fa[d] = a;
                t.fb[d] = bt;
                t.fl[d] = lc;
            }
            m_run = fmaxf(m_run, __shfl_sync(0xffffffffu, incl, 31));
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < kMergeTile; ++c) {
            if (c < nt) {
                o = merge_value(o, ov[c], t.fa[c], t.fb[c]);
                l = merge_value(l, t.fl[c], t.fa[c], t.fb[c]);
            }
        }
    };
    merge_tile(first, min(kMergeTile, nc), mc0, lc0);
    for (int c0 = kMergeTile; c0 < nc; c0 += kMergeTile) {
        const int nt = min(kMergeTile, nc - c0);
        const float *oc = w + static_cast<int64_t>(c0) * (kD + 2) + 2 + d;
        float ov[kMergeTile];                                   // in flight while warp 0 prepares the factors
#pragma unroll
        for (int c = 0; c < kMergeTile; ++c) ov[c] = c < nt ? oc[static_cast<int64_t>(c) * (kD + 2)] : 0.0f;
        const float *wc = w + static_cast<int64_t>(c0 + d) * (kD + 2);
        const float mc = d < nt ? wc[0] : -INFINITY;       // read by warp 0 only
        const float lc = d < nt ? wc[1] : 0.0f;
        merge_tile(ov, nt, mc, lc);
    }
    return static_cast<uint16_t>(pack_bf16x2(__float_as_uint(__fdiv_rn(o, l)), 0u) & 0xFFFFu);
}

}  // namespace bi
