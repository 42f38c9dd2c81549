// gemm_int4.cu -- batch-invariant linear layer with 4-bit weights and group scales.
//
//   Y[m][n] = bf16( sum over groups of s[n][g] * ( sum_{k in g} X[m][k] (u[n][k] - z[n][g]) ) )
//
// For few rows the weights' bytes bound it: half a byte each, read once. The
// codes go from global memory to registers and straight into tensor-core
// operands: the bits 0x4300 | u are the bf16 number 128 + u, and subtracting
// 128 + z leaves the integer u - z exactly, so the products see the weights
// without a rounding; each group's sum is scaled in fp32.
//   A = 16 weight rows x 16 k, B = 16 k x 8 rows of X (m16n8k16): few rows of X
//   waste columns of a narrow operand instead of rows of a wide one.
// The k of one product step need not be neighbours as long as A and B agree: a
// lane takes its k as whole 32-bit words of the weight row (eight codes, two
// steps), and the nibbles q and q + 4 of a word are one operand pair.
//
// The sum's order is fixed by (K, group): K is cut into blocks of 128 and the
// blocks into S segments, one a warp; a warp adds its groups in ascending
// order, and the segments' sums are added in order. The number of rows decides
// only how many 8-row column tiles a warp carries.
#include "attn_common.cuh"
#include "bi_internal.h"
#include "bi_ptx.cuh"
#include "kv_int4.cuh"

namespace bi {
namespace {

constexpr int kBlockK = 128;                   // k of one step of a warp's loop
constexpr int kRows = 16;                      // weight rows of a CTA
constexpr int kMaxSegments = 8;

struct GemmI4Params {
    const uint16_t *X;       // [M][ldx]
    const uint8_t *W;        // [N][K / 2]
    const uint16_t *S;       // [N][K / group] bf16
    const uint8_t *Z;        // [N][K / group] or null
    uint16_t *Y;             // [M][ldy]
    int64_t ldx, ldy, M, N, K, group;
    unsigned *status;
};

// GS: k per scale inside a block (32, 64, or 128 for groups of a multiple of 128)
template <int GS, int NT>
__global__ void __launch_bounds__(32 * kMaxSegments)
gemm_int4_kernel(const GemmI4Params p) {
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    constexpr int kSub = kBlockK / GS, kWords = GS / 32;   // groups of a block, a lane's words of a group
    __shared__ float red[kMaxSegments][kRows][8 * NT + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, segments = blockDim.x >> 5;
    const int gq = lane >> 2, cq = lane & 3;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kRows, m0 = static_cast<int64_t>(blockIdx.y) * (8 * NT);
    const int64_t blocks = (p.K + kBlockK - 1) / kBlockK, groups = p.K / p.group;
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][e] = 0.0f;
    for (int64_t kb = warp * blocks / segments; kb < (warp + 1) * blocks / segments; ++kb) {
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
            const int64_t k0 = kb * kBlockK + sub * GS + 8 * kWords * cq;   // the lane's k of this group
            const bool in_k = kb * kBlockK + sub * GS < p.K;
            uint32_t w[2][kWords], z2[2];
            float sc[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t n = n0 + gq + 8 * h;
                sc[h] = 0.0f;
                z2[h] = 0xC308C308u;                       // -(128 + 8)
#pragma unroll
                for (int j = 0; j < kWords; ++j) w[h][j] = 0u;
                if (in_k && n < p.N) {
                    const uint8_t *src = p.W + n * (p.K / 2) + k0 / 2;
#pragma unroll
                    for (int j = 0; j < kWords; ++j) w[h][j] = reinterpret_cast<const uint32_t *>(src)[j];
                    const int64_t gi = n * groups + (kb * kBlockK + sub * GS) / p.group;
                    sc[h] = __uint_as_float(static_cast<uint32_t>(p.S[gi]) << 16);
                    if (p.Z) z2[h] = 0xC300C300u | ((p.Z[gi] & 15u) * 0x00010001u);
                }
            }
            float part[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) part[t][e] = 0.0f;
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                uint32_t a[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    a[h][0] = fma_bf16x2(i4_pair<0>(w[h][j]), 0x3F803F80u, z2[h]);
                    a[h][1] = fma_bf16x2(i4_pair<1>(w[h][j]), 0x3F803F80u, z2[h]);
                    a[h][2] = fma_bf16x2(i4_pair<2>(w[h][j]), 0x3F803F80u, z2[h]);
                    a[h][3] = fma_bf16x2(i4_pair<3>(w[h][j]), 0x3F803F80u, z2[h]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int64_t m = m0 + 8 * t + gq;
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (in_k && m < p.M) x = *reinterpret_cast<const uint4 *>(p.X + m * p.ldx + k0 + 8 * j);
                    mma_16816(part[t], a[0][0], a[1][0], a[0][1], a[1][1], zip16<0>(x.x, x.z), zip16<1>(x.x, x.z));
                    mma_16816(part[t], a[0][2], a[1][2], a[0][3], a[1][3], zip16<0>(x.y, x.w), zip16<1>(x.y, x.w));
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[t][e] = __fmaf_rn(sc[e >> 1], part[t][e], acc[t][e]);
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[warp][gq + 8 * (e >> 1)][8 * t + 2 * cq + (e & 1)] = acc[t][e];
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * 8 * NT; i += blockDim.x) {
        const int r = i % kRows, t = i / kRows;
        float y = red[0][r][t];
        for (int s = 1; s < segments; ++s) y += red[s][r][t];
        if (m0 + t < p.M && n0 + r < p.N && BI_IN_BOUNDS((m0 + t) * p.ldy + n0 + r < p.M * p.ldy, p.status))
            p.Y[(m0 + t) * p.ldy + n0 + r] = static_cast<uint16_t>(pack_bf16x2(__float_as_uint(y), 0u) & 0xFFFFu);
    }
}

template <int GS, int NT>
bi_status launch_shape(const GemmI4Params &p, cudaStream_t s) {
    const int64_t blocks = (p.K + kBlockK - 1) / kBlockK;
    const int segments = static_cast<int>(blocks < 4 ? 1 : blocks / 4 > kMaxSegments ? kMaxSegments : blocks / 4);
    const int64_t gx = (p.N + kRows - 1) / kRows, gy = (p.M + 8 * NT - 1) / (8 * NT);
    if (gx > 0x7FFFFFFF || gy > 65535) return BI_ERR_UNSUPPORTED;
    return launch_pdl(gemm_int4_kernel<GS, NT>, dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)),
                      dim3(32 * segments), 0, s, p);
}
template <int GS>
bi_status launch_group(const GemmI4Params &p, cudaStream_t s) {
    if (p.M <= 8) return launch_shape<GS, 1>(p, s);
    if (p.M <= 16) return launch_shape<GS, 2>(p, s);
    if (p.M <= 32) return launch_shape<GS, 4>(p, s);
    return launch_shape<GS, 8>(p, s);
}

}  // namespace

bi_status launch_gemm_int4(const void *X, int64_t ldx, const uint8_t *W, const void *scales, const uint8_t *zeros, void *Y,
                           int64_t ldy, int64_t M, int64_t N, int64_t K, int64_t group, cudaStream_t s) {
    const GemmI4Params p{static_cast<const uint16_t *>(X), W, static_cast<const uint16_t *>(scales), zeros,
                         static_cast<uint16_t *>(Y), ldx, ldy, M, N, K, group, device_status_word()};
    if (group == 32) return launch_group<32>(p, s);
    if (group == 64) return launch_group<64>(p, s);
    return launch_group<128>(p, s);
}

}  // namespace bi
