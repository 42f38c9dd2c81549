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
// The two half warps take the K and the V row of the same token and head.
//
// Both kernels are bound by memory: 512 bytes in and 144 out per token and KV
// head (append), the reverse (read).
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

// Cache row of token t's slot for head g; -1: padding (slot -1) or a slot outside the cache.
__device__ __forceinline__ int64_t slot_row(const RowsParams &p, int64_t t, int g) {
    const int64_t slot = p.slots[t];
    if (slot < 0 || slot >= p.c.num_blocks * p.c.bs) {
        if (slot != -1) atomicOr(p.status, kDevBadOffsets);
        return -1;
    }
    return (slot / p.c.bs * p.c.Hkv + g) * p.c.bs + slot % p.c.bs;
}

__global__ void __launch_bounds__(kThreads)
kv_int4_append_kernel(const RowsParams p) {
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    const int lane = threadIdx.x & 31, is_v = lane >> 4, i = (lane >> 2) & 3, q = lane & 3;
    const int64_t pairs = p.T * p.c.Hkv;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t w = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5); w < pairs; w += warps) {
        const int64_t t = w / p.c.Hkv;
        const int g = static_cast<int>(w % p.c.Hkv);
        const int64_t row = slot_row(p, t, g);
        if (row < 0) continue;                             // the whole warp: one (token, head)
        const uint16_t *src = (is_v ? p.V + t * p.ldv : p.K + t * p.ldk) + g * kRowDims + 32 * i + 8 * q;
        const uint4 x4 = *reinterpret_cast<const uint4 *>(src);
        const uint32_t xw[4] = {x4.x, x4.y, x4.z, x4.w};
        // the group's largest magnitude, as bf16 bits (a NaN or infinity compares above every number)
        uint32_t am = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) am = max(am, max(xw[k] & 0x7FFFu, (xw[k] >> 16) & 0x7FFFu));
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
        // amax / 7 is a four-bit number or further from one than its rounding to
        // fp32, so rounding the fp32 quotient up is rounding the quotient up
        float s = fminf(fmaxf(__fdiv_rn(__uint_as_float(am << 16), 7.0f), 0x1p-100f), 0x1p120f);
        s = __uint_as_float((__float_as_uint(s) + 0xFFFFFu) & ~0xFFFFFu);
        const bool finite = am < 0x7F80u;
        const float inv = finite ? __frcp_rn(s) : 0.0f;
        const float lim = 7.0f * s, half = 0.5f * s;
        uint32_t code[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t c2 = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x = fminf(fmaxf(__uint_as_float(e ? xw[k] & 0xFFFF0000u : xw[k] << 16), -lim), lim);
                // 1.5 * 2^23 + 8 + (x / s rounded): the code sits in the sum's low bits. The product
                // with the rounded reciprocal is off by less than a quotient's distance from
                // a tie (x has 8 bits, s four), except at a tie: there x - n s = +-s/2 exactly, and the even
                // neighbour is the nearest multiple of two, from a sum whose unit is 2.
                float m = __fmaf_rn(x, inv, 12582920.0f);
                const float n = m - 12582920.0f;
                if (fabsf(__fmaf_rn(-n, s, x)) == half) m = (__fmaf_rn(x, inv, 25165824.0f) - 25165824.0f) + 12582920.0f;
                c2 |= (__float_as_uint(m) & 15u) << (16 * e);
            }
            code[k] = (finite ? c2 : 0x00080008u) << (4 * q);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            code[k] |= __shfl_xor_sync(0xffffffffu, code[k], 1);
            code[k] |= __shfl_xor_sync(0xffffffffu, code[k], 2);
        }
        // code[a] is the segment's 32-bit word of r = 2a, 2a + 1: lane q stores word q
        const uint32_t mine = q == 0 ? code[0] : q == 1 ? code[1] : q == 2 ? code[2] : code[3];
        if (!BI_IN_BOUNDS(row < p.c.num_blocks * p.c.Hkv * p.c.bs, p.status)) continue;
        const int at = i4_place(i, static_cast<int>(row % p.c.bs)) * 16 + 4 * q;
        *reinterpret_cast<uint32_t *>((is_v ? p.c.vc : p.c.kc) + row * kI4Row + at) = mine;
        if (q == 0)
            (is_v ? p.c.vs : p.c.ks)[row * kI4Scales + i] = static_cast<uint16_t>(finite ? __float_as_uint(s) >> 16 : 0x7FFFu);
    }
}

__global__ void __launch_bounds__(kThreads)
kv_int4_read_kernel(const RowsParams p) {
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    const int lane = threadIdx.x & 31, is_v = lane >> 4, i = (lane >> 2) & 3, q = lane & 3;
    const int64_t pairs = p.T * p.c.Hkv;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t w = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5); w < pairs; w += warps) {
        const int64_t t = w / p.c.Hkv;
        const int g = static_cast<int>(w % p.c.Hkv);
        const int64_t row = slot_row(p, t, g);
        uint4 seg = make_uint4(0u, 0u, 0u, 0u);
        uint32_t sc = 0;
        if (row >= 0 && BI_IN_BOUNDS(row < p.c.num_blocks * p.c.Hkv * p.c.bs, p.status)) {
            seg = *reinterpret_cast<const uint4 *>((is_v ? p.c.vc : p.c.kc) + row * kI4Row +
                                                   i4_place(i, static_cast<int>(row % p.c.bs)) * 16);
            sc = (is_v ? p.c.vs : p.c.ks)[row * kI4Scales + i];
        }
        const uint32_t s2 = sc | (sc << 16), c2 = mul_bf16x2(s2, kBf16x2_m136);
        const uint32_t cw[4] = {seg.x, seg.y, seg.z, seg.w};
        uint32_t out[4];
#pragma unroll
        for (int a = 0; a < 4; ++a)
            out[a] = row < 0 ? 0u : fma_bf16x2(((cw[a] >> (4 * q)) & 0x000F000Fu) | 0x43004300u, s2, c2);
        uint16_t *dst = (is_v ? p.V + t * p.ldv : p.K + t * p.ldk) + g * kRowDims + 32 * i + 8 * q;
        *reinterpret_cast<uint4 *>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
    }
}

template <typename Kernel>
bi_status launch_rows(Kernel kernel, const RowsParams &p, cudaStream_t s) {
    int dev = 0;
    const DeviceInfo *info = nullptr;
    const bi_status st = current_device(&dev, &info);
    if (st != BI_OK) return st;
    const int64_t ctas = (p.T * p.c.Hkv + kThreads / 32 - 1) / (kThreads / 32), cap = static_cast<int64_t>(info->sm_count) * 8;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas < cap ? ctas : cap)), dim3(kThreads), 0, s, p);
}

}  // namespace

bi_status launch_kv_int4_append(const KvInt4 &c, const int64_t *slots, const void *K, int64_t ldk, const void *V,
                                int64_t ldv, int64_t T, cudaStream_t s) {
    RowsParams p{c, slots, static_cast<uint16_t *>(const_cast<void *>(K)), static_cast<uint16_t *>(const_cast<void *>(V)),
                 ldk, ldv, T, device_status_word()};
    return launch_rows(kv_int4_append_kernel, p, s);
}

bi_status launch_kv_int4_read(const KvInt4 &c, const int64_t *slots, void *K, int64_t ldk, void *V, int64_t ldv,
                              int64_t T, cudaStream_t s) {
    RowsParams p{c, slots, static_cast<uint16_t *>(K), static_cast<uint16_t *>(V), ldk, ldv, T, device_status_word()};
    return launch_rows(kv_int4_read_kernel, p, s);
}

}  // namespace bi
