// kv_int4.cu -- the paged 4-bit K/V cache: append (quantise) and read.
//
// Per row of 128 dimensions and group of 32: amax = max |x|,
//   s = the smallest number with four significant bits >= amax / 7, kept in
//       [2^-100, 2^120] (a group that holds an infinity or a NaN: s = NaN),
//   n = clamp(x / s rounded to an integer, ties to even, -7, 7),  code n + 8,
// on the exact quotients. Half a warp takes one row: lane (i, q) holds the
// eight dimensions 32 i + 8 q + r as one 16-byte load, the four lanes of a
// group share its maximum by two shuffles, and their codes, each at nibble q,
// are transposed by two shuffles into the segment's words (layout: kv_int4.cuh).
// The two half warps take the K and the V row of the same token and head, and
// a warp one or four heads of a token.
//
// 512 bytes in and 144 out per token and KV head (append), the reverse (read).
// Measured (8 heads): 8155 tokens 19.5 us for both (4.4 TB/s; append by its 124 instructions
// a row pair, 60 % of the issue slots, as much as by memory), 64 tokens 3.2 us.
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
    unsigned *status;
};

// Where token t is held: the cache row of its head 0 (a head's rows are bs apart; -1: the slot is padding or outside
// the cache), at this offset of its block.
struct Place {
    int64_t row;
    int offset;
};
__device__ __forceinline__ Place find(const RowsParams &p, int64_t t) {
    const int64_t slot = p.slots[t];
    Place x{-1, 0};
    if (slot >= 0 && slot < p.c.num_blocks * p.c.bs) {      // (slots of a cache are below 2^32)
        const uint32_t blk = static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.c.bs);
        x.offset = static_cast<int>(static_cast<uint32_t>(slot) - blk * static_cast<uint32_t>(p.c.bs));
        x.row = static_cast<int64_t>(blk) * p.c.Hkv * p.c.bs + x.offset;
    } else if (slot != -1) {
        atomicOr(p.status, kDevBadOffsets);
    }
    return x;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// The bits of a where mask is set, else those of b.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t pick(uint32_t a, uint32_t b) { return (a & MASK) | (b & ~MASK); }

// Quantises half a warp's row: the lane's eight values in `xw`; the row's word of the lane (segment i, word q) and
// the group's scale.
__device__ __forceinline__ void quantise(const uint32_t (&xw)[4], int q, uint32_t &word, uint32_t &scale) {
    // the group's largest magnitude, as bf16 bits (a NaN or infinity compares above every number)
    uint32_t am = max_u16x2(max_u16x2(xw[0] & 0x7FFF7FFFu, xw[1] & 0x7FFF7FFFu), max_u16x2(xw[2] & 0x7FFF7FFFu, xw[3] & 0x7FFF7FFFu));
    am = max_u16x2(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = max_u16x2(am, __shfl_xor_sync(0xffffffffu, am, 2));
    am = max(am << 16, am & 0xFFFF0000u);
    const float amax = __uint_as_float(am);
    // amax times 1/7 rounded down: amax / 7 is a four-bit number, then this is it or just below, or more than 2^-8 away
    // from one, so rounding this up to four bits is rounding the quotient up
    float s = fminf(fmaxf(__fmul_rn(amax, 0x1.249248p-3f), 0x1p-100f), 0x1p120f);
    s = __uint_as_float((__float_as_uint(s) + 0xFFFFFu) & ~0xFFFFFu);
    const bool finite = am < 0x7F800000u;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));   // (1 / s within 2^-23 of itself)
    float x[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[2 * k] = __uint_as_float(xw[k] << 16), x[2 * k + 1] = __uint_as_float(xw[k] & 0xFFFF0000u);
    if (amax > 0x1.cp122f) {                               // 7 * 2^120: saturates
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = fminf(fmaxf(x[k], -0x1.cp122f), 0x1.cp122f);
    }
    // x r + 1.5 * 2^13, rounded to a multiple of 2^-10, has the quotient x / s where that is a tie, and is on the
    // quotient's side of the nearest tie elsewhere (x has 8 bits and s four: no other quotient is within 2^-10 of a tie);
    // then 1.5 * 2^23 + 8 + the quotient rounds it to an integer (ties to even), its code in the low bits
    uint32_t z[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        z[k] = zip16<0>(__float_as_uint(__fadd_rn(__fmaf_rn(x[2 * k], r, 12288.0f), 12570632.0f)),
                        __float_as_uint(__fadd_rn(__fmaf_rn(x[2 * k + 1], r, 12288.0f), 12570632.0f)));
    // nibble k of each half: the code pair for word k. The group's four lanes transpose these: lane q keeps nibble q
    // of each lane's, at that lane's nibble, first by bytes (lanes q ^ 2), then within them (q ^ 1)
    uint32_t w = pick<0x0FFF0FFFu>(pick<0x00FF00FFu>(pick<0x000F000Fu>(z[0], z[1] << 4), z[2] << 8), z[3] << 12);
    w = finite ? w : 0x88888888u;
    uint32_t o = __shfl_xor_sync(0xffffffffu, w, 2);
    w = __byte_perm(w, o, q & 2 ? 0x3715 : 0x6240);
    o = __shfl_xor_sync(0xffffffffu, w, 1);
    word = q & 1 ? pick<0xF0F0F0F0u>(w, o >> 4) : pick<0x0F0F0F0Fu>(w, o << 4);
    scale = finite ? __float_as_uint(s) >> 16 : 0x7FFFu;
}

// Warps take tokens (grid x) and HEADS heads (grid y).
template <int HEADS>
__global__ void __launch_bounds__(kThreads)
kv_int4_append_kernel(const RowsParams p) {
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    const int lane = threadIdx.x & 31, is_v = lane >> 4, i = (lane >> 2) & 3, q = lane & 3;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32), next = static_cast<int64_t>(p.c.bs) * kI4Row;
    for (int64_t t = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5); t < p.T; t += warps) {
        const Place x = find(p, t);
        if (x.row < 0) continue;                           // the whole warp: one token
        for (int g = blockIdx.y * HEADS; g < p.c.Hkv; g += gridDim.y * HEADS) {
            const uint16_t *src = (is_v ? p.V + t * p.ldv : p.K + t * p.ldk) + g * kRowDims + 32 * i + 8 * q;
            uint4 in[HEADS];
#pragma unroll
            for (int k = 0; k < HEADS; ++k)
                if (g + k < p.c.Hkv) in[k] = *reinterpret_cast<const uint4 *>(src + k * kRowDims);
            const int64_t row = x.row + static_cast<int64_t>(g) * p.c.bs;
            uint8_t *codes = (is_v ? p.c.vc : p.c.kc) + row * kI4Row + i4_place(i, x.offset) * 16 + 4 * q;
            uint16_t *scales = (is_v ? p.c.vs : p.c.ks) + row * kI4Scales + i;
#pragma unroll
            for (int k = 0; k < HEADS; ++k, codes += next, scales += next / (kI4Row / kI4Scales)) {
                if (g + k >= p.c.Hkv) break;
                const uint32_t xw[4] = {in[k].x, in[k].y, in[k].z, in[k].w};
                uint32_t word, scale;
                quantise(xw, q, word, scale);
                if (!BI_IN_BOUNDS(row + static_cast<int64_t>(k) * p.c.bs < p.c.num_blocks * p.c.Hkv * p.c.bs, p.status)) continue;
                *reinterpret_cast<uint32_t *>(codes) = word;
                if (q == 0) *scales = static_cast<uint16_t>(scale);
            }
        }
    }
}

template <int HEADS>
__global__ void __launch_bounds__(kThreads)
kv_int4_read_kernel(const RowsParams p) {
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    const int lane = threadIdx.x & 31, is_v = lane >> 4, i = (lane >> 2) & 3, q = lane & 3;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32), next = static_cast<int64_t>(p.c.bs) * kI4Row;
    for (int64_t t = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5); t < p.T; t += warps) {
        const Place x = find(p, t);
        for (int g = blockIdx.y * HEADS; g < p.c.Hkv; g += gridDim.y * HEADS) {
            const int64_t row = x.row + static_cast<int64_t>(g) * p.c.bs;
            const uint8_t *codes = (is_v ? p.c.vc : p.c.kc) + row * kI4Row + i4_place(i, x.offset) * 16;
            const uint16_t *scales = (is_v ? p.c.vs : p.c.ks) + row * kI4Scales + i;
            uint4 seg[HEADS];
            uint32_t sc[HEADS];
#pragma unroll
            for (int k = 0; k < HEADS; ++k, codes += next, scales += next / (kI4Row / kI4Scales)) {
                seg[k] = make_uint4(0u, 0u, 0u, 0u), sc[k] = 0u;   // (all zeros expand to 0)
                if (x.row >= 0 && g + k < p.c.Hkv &&
                    BI_IN_BOUNDS(row + static_cast<int64_t>(k) * p.c.bs < p.c.num_blocks * p.c.Hkv * p.c.bs, p.status)) {
                    seg[k] = *reinterpret_cast<const uint4 *>(codes);
                    sc[k] = *scales;
                }
            }
            uint16_t *dst = (is_v ? p.V + t * p.ldv : p.K + t * p.ldk) + g * kRowDims + 32 * i + 8 * q;
#pragma unroll
            for (int k = 0; k < HEADS; ++k) {
                if (g + k >= p.c.Hkv) break;
                const uint32_t s2 = sc[k] | (sc[k] << 16), c2 = mul_bf16x2(s2, kBf16x2_m136);
                const uint32_t cw[4] = {seg[k].x, seg[k].y, seg[k].z, seg[k].w};
                uint32_t out[4];
#pragma unroll
                for (int a = 0; a < 4; ++a) out[a] = fma_bf16x2(i4_pair<0>(cw[a] >> (4 * q)), s2, c2);
                *reinterpret_cast<uint4 *>(dst + k * kRowDims) = make_uint4(out[0], out[1], out[2], out[3]);
            }
        }
    }
}

// Four heads a warp keep more loads in flight; one a warp has the shorter way through. Append + read, eight heads,
// one / four: 64 tokens 3.2 / 4.0 us, 256 3.6 / 4.0, 608 5.4 / 4.1, 8155 29.9 / 19.3.
template <typename One, typename Four>
bi_status launch_rows(One one, Four four, RowsParams p, cudaStream_t s) {
    int dev = 0;
    const DeviceInfo *info = nullptr;
    const bi_status st = current_device(&dev, &info);
    if (st != BI_OK) return st;
    const bool few = p.T * p.c.Hkv < 32 * static_cast<int64_t>(info->sm_count);
    const int64_t x = (p.T + kThreads / 32 - 1) / (kThreads / 32), y = few ? p.c.Hkv : (p.c.Hkv + 3) / 4;
    const int64_t cap = static_cast<int64_t>(info->sm_count) * 32;
    const dim3 grid(static_cast<unsigned>(x < cap ? x : cap), static_cast<unsigned>(y < 64 ? y : 64));
    return few ? launch_pdl(one, grid, dim3(kThreads), 0, s, p) : launch_pdl(four, grid, dim3(kThreads), 0, s, p);
}

}  // namespace

bi_status launch_kv_int4_append(const KvInt4 &c, const int64_t *slots, const void *K, int64_t ldk, const void *V,
                                int64_t ldv, int64_t T, cudaStream_t s) {
    RowsParams p{c, slots, static_cast<uint16_t *>(const_cast<void *>(K)), static_cast<uint16_t *>(const_cast<void *>(V)),
                 ldk, ldv, T, device_status_word()};
    return launch_rows(kv_int4_append_kernel<1>, kv_int4_append_kernel<4>, p, s);
}

bi_status launch_kv_int4_read(const KvInt4 &c, const int64_t *slots, void *K, int64_t ldk, void *V, int64_t ldv,
                              int64_t T, cudaStream_t s) {
    RowsParams p{c, slots, static_cast<uint16_t *>(K), static_cast<uint16_t *>(V), ldk, ldv, T, device_status_word()};
    return launch_rows(kv_int4_read_kernel<1>, kv_int4_read_kernel<4>, p, s);
}

}  // namespace bi
