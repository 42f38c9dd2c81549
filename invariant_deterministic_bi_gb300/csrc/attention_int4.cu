// attention_int4.cu -- decode attention over the paged 4-bit K/V cache.
//
// The result is bi_attention_decode's over a bf16 cache that holds the same
// values, bit for bit: the values are bf16 numbers exactly (kv_int4.cuh), the
// 128-token chunks, the tensor-core chains (ascending dimension steps for q.k,
// ascending token steps with p's high part before its low part for p.v), the
// order of each sum and the chunk merge are the same. What differs is the work
// split: a chunk of one KV head is 18 KB here, not 64 KB, and its codes are
// expanded in registers, so one warp computes one chunk on its own, without a
// barrier. The products are taken transposed, tokens (or dimensions) as the 16
// rows and the up to eight query heads of the KV head as the 8 columns: half
// the tensor-core work of 16 query rows of which at most eight exist.
//   q.k: A = 16 tokens x 16 dimensions of K, B = q^T. A lane's operands of all
//        eight steps are 16 contiguous bytes of each of its two rows.
//   p.v: A = 16 dimensions x 16 tokens of V (the pairs joined from two tokens'
//        words), B = p: the scores' fragment transposed by movmatrix.
#include "attn_common.cuh"
#include "bi_internal.h"
#include "bi_ptx.cuh"
#include "kv_int4.cuh"

namespace bi {
namespace {

constexpr int kWarps = 4;                      // items in flight per CTA, one a warp
constexpr uint32_t kNoRow = 0xFFFFFFFFu;

struct DecodeI4Params {
    KvInt4 c;
    const uint16_t *Q;       // [B][Hq][D]
    const int32_t *table;    // [B][max_blocks]
    const int32_t *lens;     // [B]
    float *ws;               // [B][Hq][chunks][kD + 2]
    int64_t batch;
    int32_t max_blocks, Hq, chunks, max_len;
    float scale;
    unsigned *status;
};

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

template <int G>
__global__ void __launch_bounds__(32 * kWarps)
attn_decode_int4_kernel(const DecodeI4Params p) {
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, cq = lane & 3;               // fragment row group, column pair
    const int64_t items = p.batch * p.c.Hkv * static_cast<int64_t>(p.chunks);
    const int64_t ws_head = static_cast<int64_t>(p.chunks) * (kD + 2);   // next query head's record
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * kWarps + warp; it < items;
         it += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int g = static_cast<int>(it % p.c.Hkv);
        const int64_t r = it / p.c.Hkv;
        const int c = static_cast<int>(r % p.chunks);
        const int64_t b = r / p.chunks;
        const int L = p.lens[b];
        if (L < 1 || L > p.max_len || L > static_cast<int64_t>(p.max_blocks) * p.c.bs) {
            if (lane == 0 && c == 0 && g == 0) atomicOr(p.status, kDevBadOffsets);
            continue;
        }
        const int n = min(kChunk, L - c * kChunk);
        if (n <= 0) continue;
        // cache rows of tokens lane, lane + 32, lane + 64, lane + 96
        uint32_t row[4];
        bool bad = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            row[k] = kNoRow;
            const int t = lane + 32 * k;
            if (t < n) {
                const int j = c * kChunk + t;
                const int64_t blk = p.table[b * p.max_blocks + j / p.c.bs];
                if (blk >= 0 && blk < p.c.num_blocks)
                    row[k] = static_cast<uint32_t>((blk * p.c.Hkv + g) * p.c.bs + j % p.c.bs);
                else
                    bad = true;
            }
        }
        if (bad) atomicOr(p.status, kDevBadOffsets);
        const uint16_t *q = p.Q + (b * p.Hq + g * G + (gq < G ? gq : 0)) * kD + 2 * cq;
        uint32_t qb[kD / 16][2];
#pragma unroll
        for (int ks = 0; ks < kD / 16; ++ks) {
            qb[ks][0] = gq < G ? *reinterpret_cast<const uint32_t *>(q + 16 * ks) : 0u;
            qb[ks][1] = gq < G ? *reinterpret_cast<const uint32_t *>(q + 16 * ks + 8) : 0u;
        }
        // scores: s[mt][e], token 16 mt + gq + 8 (e / 2), head 2 cq + e % 2
        float s[kChunk / 16][4];
#pragma unroll
        for (int mt = 0; mt < kChunk / 16; ++mt) {
            uint32_t kw[2][4], sc[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t rr = __shfl_sync(0xffffffffu, row[mt >> 1], 16 * (mt & 1) + 8 * h + gq);
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                uint2 x = make_uint2(0u, 0u);
                if (rr != kNoRow) {
                    w = *reinterpret_cast<const uint4 *>(p.c.kc + static_cast<int64_t>(rr) * kI4Row + 16 * cq);
                    x = *reinterpret_cast<const uint2 *>(p.c.ks + static_cast<int64_t>(rr) * kI4Scales);
                }
                kw[h][0] = w.x, kw[h][1] = w.y, kw[h][2] = w.z, kw[h][3] = w.w;
                sc[h][0] = x.x, sc[h][1] = x.y;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][e] = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {                  // 32 dimensions: one scale, two 16-dimension steps
                uint32_t a[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t s2 = i & 1 ? dup16<1>(sc[h][i >> 1]) : dup16<0>(sc[h][i >> 1]);
                    i4_expand(kw[h][i], s2, mul_bf16x2(s2, kBf16x2_m136), a[h]);
                }
                mma_16816(s[mt], a[0][0], a[1][0], a[0][1], a[1][1], qb[2 * i][0], qb[2 * i][1]);
                mma_16816(s[mt], a[0][2], a[1][2], a[0][3], a[1][3], qb[2 * i + 1][0], qb[2 * i + 1][1]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = __shfl_sync(0xffffffffu, row[mt >> 1], 16 * (mt & 1) + 8 * h + gq) != kNoRow;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    s[mt][2 * h + e] = in ? __fmul_rn(s[mt][2 * h + e], p.scale) : -INFINITY;
            }
        }
        // per head: the maximum, the exponentials, and their sum in the bf16 kernels' order: tokens
        // L, L + 32, L + 64, L + 96 in turn (mt = L / 16 % 2 + 0, 2, 4, 6), then a butterfly over
        // L xor 16 (mt), 8 (the fragment's half), 4, 2, 1 (lanes)
        float m[2], l[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m[e] = kNoScore;
#pragma unroll
            for (int mt = 0; mt < kChunk / 16; ++mt) m[e] = fmaxf(m[e], fmaxf(s[mt][e], s[mt][2 + e]));
#pragma unroll
            for (int o = 16; o >= 4; o >>= 1) m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], o));
        }
#pragma unroll
        for (int mt = 0; mt < kChunk / 16; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][e] = expf(s[mt][e] - m[e & 1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float col[2][2];                               // [mt % 2][half]
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    col[o][h] = ((s[o][2 * h + e] + s[o + 2][2 * h + e]) + s[o + 4][2 * h + e]) + s[o + 6][2 * h + e];
            l[e] = (col[0][0] + col[1][0]) + (col[0][1] + col[1][1]);
#pragma unroll
            for (int o = 16; o >= 4; o >>= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], o);
        }
        float *ws = p.ws + ((b * p.Hq + g * G) * p.chunks + c) * static_cast<int64_t>(kD + 2);
        if (!BI_IN_BOUNDS(b < p.batch && c < p.chunks, p.status)) break;
        if (gq == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (2 * cq + e < G) {
                    ws[(2 * cq + e) * ws_head] = m[e];
                    ws[(2 * cq + e) * ws_head + 1] = l[e];
                }
        }
        // p as B fragments (high and low bf16 parts): the score fragment is [token][head], B wants
        // lane (head gq, tokens 2 cq, 2 cq + 1)
        uint32_t ph[kChunk / 16][2], pl[kChunk / 16][2];
#pragma unroll
        for (int mt = 0; mt < kChunk / 16; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t hi, lo;
                split_bf16x2(s[mt][2 * h], s[mt][2 * h + 1], hi, lo);
                ph[mt][h] = transpose_8x8(hi);
                pl[mt][h] = transpose_8x8(lo);
            }
        // values: o[j][e], dimension 16 j + gq + 8 (e / 2), head 2 cq + e % 2
        float o[kD / 16][4];
#pragma unroll
        for (int j = 0; j < kD / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < kChunk / 16; ++ks) {
            uint32_t vw[4][2], sc[4][2];                   // tokens 2 cq, + 1, + 8, + 9 of the step
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t rr = __shfl_sync(0xffffffffu, row[ks >> 1], 16 * (ks & 1) + 2 * cq + (k & 1) + 8 * (k >> 1));
                uint2 w = make_uint2(0u, 0u), x = make_uint2(0u, 0u);
                if (rr != kNoRow) {
                    w = *reinterpret_cast<const uint2 *>(p.c.vc + static_cast<int64_t>(rr) * kI4Row + 8 * gq);
                    x = *reinterpret_cast<const uint2 *>(p.c.vs + static_cast<int64_t>(rr) * kI4Scales);
                }
                vw[k][0] = w.x, vw[k][1] = w.y;
                sc[k][0] = x.x, sc[k][1] = x.y;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {                  // 32 dimensions: tiles 2 i and 2 i + 1
                uint32_t a[2][4];                          // [token pair][nibble]
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t s2 = i & 1 ? zip16<1>(sc[2 * k][i >> 1], sc[2 * k + 1][i >> 1])
                                              : zip16<0>(sc[2 * k][i >> 1], sc[2 * k + 1][i >> 1]);
                    const uint32_t w = i & 1 ? zip16<1>(vw[2 * k][i >> 1], vw[2 * k + 1][i >> 1])
                                             : zip16<0>(vw[2 * k][i >> 1], vw[2 * k + 1][i >> 1]);
                    i4_expand(w, s2, mul_bf16x2(s2, kBf16x2_m136), a[k]);
                }
                mma_16816(o[2 * i], a[0][0], a[0][1], a[1][0], a[1][1], ph[ks][0], ph[ks][1]);
                mma_16816(o[2 * i + 1], a[0][2], a[0][3], a[1][2], a[1][3], ph[ks][0], ph[ks][1]);
                mma_16816(o[2 * i], a[0][0], a[0][1], a[1][0], a[1][1], pl[ks][0], pl[ks][1]);
                mma_16816(o[2 * i + 1], a[0][2], a[0][3], a[1][2], a[1][3], pl[ks][0], pl[ks][1]);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (2 * cq + e < G) {
                float *w = ws + (2 * cq + e) * ws_head + 2 + gq;
#pragma unroll
                for (int j = 0; j < kD / 16; ++j) {
                    w[16 * j] = o[j][e];
                    w[16 * j + 8] = o[j][2 + e];
                }
            }
    }
}

template <int G>
bi_status launch_decode(int64_t items, const DecodeI4Params &p, cudaStream_t s) {
    const int64_t ctas = (items + kWarps - 1) / kWarps;
    return launch_pdl(attn_decode_int4_kernel<G>, dim3(static_cast<unsigned>(ctas < 0x7FFFFFFF ? ctas : 0x7FFFFFFF)),
                      dim3(32 * kWarps), 0, s, p);
}

}  // namespace

bi_status launch_attention_decode_int4(const void *Q, const KvInt4 &c, const int32_t *table, int32_t max_blocks,
                                       const int32_t *lens, int64_t B, int32_t Hq, int32_t max_len, float scale,
                                       void *workspace, void *O, cudaStream_t s) {
    DecodeI4Params p{};
    p.c = c;
    p.Q = static_cast<const uint16_t *>(Q);
    p.table = table;
    p.lens = lens;
    p.ws = static_cast<float *>(workspace);
    p.batch = B;
    p.max_blocks = max_blocks;
    p.Hq = Hq;
    p.chunks = static_cast<int32_t>((static_cast<int64_t>(max_len) + kChunk - 1) / kChunk);
    p.max_len = max_len;
    p.scale = scale;
    p.status = device_status_word();
    const int64_t items = B * c.Hkv * static_cast<int64_t>(p.chunks);
    bi_status st = BI_ERR_UNSUPPORTED;
    switch (Hq / c.Hkv) {
        case 1: st = launch_decode<1>(items, p, s); break;
        case 2: st = launch_decode<2>(items, p, s); break;
        case 4: st = launch_decode<4>(items, p, s); break;
        case 8: st = launch_decode<8>(items, p, s); break;
        default: break;
    }
    if (st != BI_OK) return st;
    return launch_attention_combine(workspace, lens, max_blocks, c.bs, B, Hq, max_len, O, s);
}

}  // namespace bi
