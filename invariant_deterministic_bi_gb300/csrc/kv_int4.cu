// kv_int4.cu -- the paged 4-bit K/V cache: append (quantise) and read.
//
// Per row of 128 dimensions and group of 32: amax = max |x|,
//   s = the smallest number with four significant bits >= amax / 7, kept in
//       [2^-100, 2^120] (a group that holds an infinity or a NaN: s = NaN),
//   n = clamp(x / s rounded to an integer, ties to even, -7, 7),  code n + 8,
// on the exact quotients. Half a warp takes one row: lane (i, q) holds the
// eight dimensions 32 i + 8 q + r as one 16-byte load, the four lanes of a
// group share its maximum by two shuffles, and their codes, each at nibble q,
// are joined by or-shuffles into the segment's words (layout: kv_int4.cuh).
// The two half warps take the K and the V row of the same token and head, and
// a warp one or four heads of a token.
//
// 512 bytes in and 144 out per token and KV head (append), the reverse (read).
// Measured (8 heads): 8155 tokens 26 us for both (3.3 TB/s each; append is bound by
// its about 110 instructions a row pair as much as by memory), 64 tokens 3.7 us.
#include "bi_internal.h"
#include "bi_ptx.cuh"
#include "kv_int4.cuh"

namespace bi {
namespace {

constexpr int kRowDims = 128;
constexpr int kThreads = 256;

struct RowsParams {
    KvInt4 c;
    const int64_t *slots;    // [T]
    uint16_t *K, *V;         // [T] tokens of [Hkv][128], ldk / ldv elements apart (append reads, read writes)
    int64_t ldk, ldv, T;
    int32_t per_token;       // warps a token: its heads, HEADS a warp
    unsigned *status;
};

// What a warp does: token t's heads g .. g + HEADS - 1, whose cache rows are row + k * bs (row < 0: the slot is
// padding or outside the cache), at this offset of their block.
struct Work {
    int64_t t, row;
    int g, offset;
};
template <int HEADS>
__device__ __forceinline__ bool find_work(const RowsParams &p, int64_t w, Work &x) {
    if (w >= p.T * p.per_token) return false;
    x.t = p.per_token == 1 ? w : w / p.per_token;
    x.g = static_cast<int>(w - x.t * p.per_token) * HEADS;
    const int64_t slot = p.slots[x.t];
    x.row = -1, x.offset = 0;
    if (slot >= 0 && slot < p.c.num_blocks * p.c.bs) {      // (slots of a cache are below 2^32)
        const uint32_t blk = static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.c.bs);
        x.offset = static_cast<int>(static_cast<uint32_t>(slot) - blk * static_cast<uint32_t>(p.c.bs));
        x.row = (static_cast<int64_t>(blk) * p.c.Hkv + x.g) * p.c.bs + x.offset;
    } else if (slot != -1) {
        atomicOr(p.status, kDevBadOffsets);
    }
    return true;
}

// Quantises half a warp's row: the lane's eight values in `xw`; the row's word of the lane (segment i, word q) and
// the group's scale.
__device__ __forceinline__ void quantise(const uint32_t (&xw)[4], int q, uint32_t &word, uint32_t &scale) {
    // the group's largest magnitude, as bf16 bits (a NaN or infinity compares above every number)
    uint32_t am = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) am = max(am, max(xw[k] & 0x7FFFu, (xw[k] >> 16) & 0x7FFFu));
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
    const float amax = __uint_as_float(am << 16);
    // amax / 7 is a four-bit number or further from one than its rounding to
    // fp32, so rounding the fp32 quotient up is rounding the quotient up
    float s = fminf(fmaxf(__fdiv_rn(amax, 7.0f), 0x1p-100f), 0x1p120f);
    s = __uint_as_float((__float_as_uint(s) + 0xFFFFFu) & ~0xFFFFFu);
    const bool finite = am < 0x7F80u;
    // 1 / s in two parts: x hi + x lo then rounds to x / s where that is a tie (a number of few bits), and stays on
    // its side of the nearest tie elsewhere (x has 8 bits, s four)
    const float hi = finite ? __frcp_rn(s) : 0.0f, lo = finite ? __fmul_rn(__fmaf_rn(-s, hi, 1.0f), hi) : 0.0f;
    const float cap = amax > 0x1.cp122f && finite ? 0x1.cp122f : INFINITY;   // 7 * 2^120: saturates
    uint32_t code[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t m[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float x = fminf(fmaxf(__uint_as_float(e ? xw[k] & 0xFFFF0000u : xw[k] << 16), -cap), cap);
            // 1.5 * 2^23 + 8 + the quotient: rounded to an integer (ties to even), its code in the low bits
            m[e] = __float_as_uint(__fadd_rn(__fmaf_rn(x, hi, __fmul_rn(x, lo)), 12582920.0f));
        }
        code[k] = ((finite ? zip16<0>(m[0], m[1]) : 0x00080008u) & 0x000F000Fu) << (4 * q);
    }
    // the four lanes of the group have a nibble of each of the segment's words; lane q keeps word q
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        code[k] |= __shfl_xor_sync(0xffffffffu, code[k], 1);
        code[k] |= __shfl_xor_sync(0xffffffffu, code[k], 2);
    }
    word = q == 0 ? code[0] : q == 1 ? code[1] : q == 2 ? code[2] : code[3];
    scale = finite ? __float_as_uint(s) >> 16 : 0x7FFFu;
}

template <int HEADS>
__global__ void __launch_bounds__(kThreads)
kv_int4_append_kernel(const RowsParams p) {
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    const int lane = threadIdx.x & 31, is_v = lane >> 4, i = (lane >> 2) & 3, q = lane & 3;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    Work x;
    for (int64_t w = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5); find_work<HEADS>(p, w, x); w += warps) {
        if (x.row < 0) continue;                           // the whole warp: one token
        const uint16_t *src = (is_v ? p.V + x.t * p.ldv : p.K + x.t * p.ldk) + x.g * kRowDims + 32 * i + 8 * q;
        uint4 in[HEADS];
#pragma unroll
        for (int k = 0; k < HEADS; ++k)
            if (x.g + k < p.c.Hkv) in[k] = *reinterpret_cast<const uint4 *>(src + k * kRowDims);
        uint8_t *codes = is_v ? p.c.vc : p.c.kc;
        uint16_t *scales = is_v ? p.c.vs : p.c.ks;
#pragma unroll
        for (int k = 0; k < HEADS; ++k) {
            if (x.g + k >= p.c.Hkv) break;
            const uint32_t xw[4] = {in[k].x, in[k].y, in[k].z, in[k].w};
            uint32_t word, scale;
            quantise(xw, q, word, scale);
            const int64_t row = x.row + static_cast<int64_t>(k) * p.c.bs;
            if (!BI_IN_BOUNDS(row < p.c.num_blocks * p.c.Hkv * p.c.bs, p.status)) continue;
            *reinterpret_cast<uint32_t *>(codes + row * kI4Row + i4_place(i, x.offset) * 16 + 4 * q) = word;
            if (q == 0) scales[row * kI4Scales + i] = static_cast<uint16_t>(scale);
        }
    }
}

template <int HEADS>
__global__ void __launch_bounds__(kThreads)
kv_int4_read_kernel(const RowsParams p) {
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    const int lane = threadIdx.x & 31, is_v = lane >> 4, i = (lane >> 2) & 3, q = lane & 3;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    Work x;
    for (int64_t w = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5); find_work<HEADS>(p, w, x); w += warps) {
        const uint8_t *codes = is_v ? p.c.vc : p.c.kc;
        const uint16_t *scales = is_v ? p.c.vs : p.c.ks;
        uint4 seg[HEADS];
        uint32_t sc[HEADS];
#pragma unroll
        for (int k = 0; k < HEADS; ++k) {
            seg[k] = make_uint4(0u, 0u, 0u, 0u), sc[k] = 0u;   // (all zeros expand to 0)
            const int64_t row = x.row + static_cast<int64_t>(k) * p.c.bs;
            if (x.row >= 0 && x.g + k < p.c.Hkv && BI_IN_BOUNDS(row < p.c.num_blocks * p.c.Hkv * p.c.bs, p.status)) {
                seg[k] = *reinterpret_cast<const uint4 *>(codes + row * kI4Row + i4_place(i, x.offset) * 16);
                sc[k] = scales[row * kI4Scales + i];
            }
        }
        uint16_t *dst = (is_v ? p.V + x.t * p.ldv : p.K + x.t * p.ldk) + x.g * kRowDims + 32 * i + 8 * q;
#pragma unroll
        for (int k = 0; k < HEADS; ++k) {
            if (x.g + k >= p.c.Hkv) break;
            const uint32_t s2 = sc[k] | (sc[k] << 16), c2 = mul_bf16x2(s2, kBf16x2_m136);
            const uint32_t cw[4] = {seg[k].x, seg[k].y, seg[k].z, seg[k].w};
            uint32_t out[4];
#pragma unroll
            for (int a = 0; a < 4; ++a) out[a] = fma_bf16x2(i4_pair<0>(cw[a] >> (4 * q)), s2, c2);
            *reinterpret_cast<uint4 *>(dst + k * kRowDims) = make_uint4(out[0], out[1], out[2], out[3]);
        }
    }
}

// Four heads a warp keep more loads in flight; one a warp has the shorter way through. Measured with
// eight heads: 64 tokens append + read 3.9 us with one, 5.1 with four; 8155 tokens 48 us and 25 us.
template <typename One, typename Four>
bi_status launch_rows(One one, Four four, RowsParams p, cudaStream_t s) {
    int dev = 0;
    const DeviceInfo *info = nullptr;
    const bi_status st = current_device(&dev, &info);
    if (st != BI_OK) return st;
    const bool few = p.T * p.c.Hkv < 32 * static_cast<int64_t>(info->sm_count);
    p.per_token = few ? p.c.Hkv : (p.c.Hkv + 3) / 4;
    const int64_t ctas = (p.T * p.per_token + kThreads / 32 - 1) / (kThreads / 32), cap = static_cast<int64_t>(info->sm_count) * 32;
    const dim3 grid(static_cast<unsigned>(ctas < cap ? ctas : cap));
    return few ? launch_pdl(one, grid, dim3(kThreads), 0, s, p) : launch_pdl(four, grid, dim3(kThreads), 0, s, p);
}

}  // namespace

bi_status launch_kv_int4_append(const KvInt4 &c, const int64_t *slots, const void *K, int64_t ldk, const void *V,
                                int64_t ldv, int64_t T, cudaStream_t s) {
    RowsParams p{c, slots, static_cast<uint16_t *>(const_cast<void *>(K)), static_cast<uint16_t *>(const_cast<void *>(V)),
                 ldk, ldv, T, 0, device_status_word()};
    return launch_rows(kv_int4_append_kernel<1>, kv_int4_append_kernel<4>, p, s);
}

bi_status launch_kv_int4_read(const KvInt4 &c, const int64_t *slots, void *K, int64_t ldk, void *V, int64_t ldv,
                              int64_t T, cudaStream_t s) {
    RowsParams p{c, slots, static_cast<uint16_t *>(K), static_cast<uint16_t *>(V), ldk, ldv, T, 0, device_status_word()};
    return launch_rows(kv_int4_read_kernel<1>, kv_int4_read_kernel<4>, p, s);
}

}  // namespace bi
