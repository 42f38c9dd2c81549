// gemm_int4.cu -- batch-invariant linear layer with 4-bit weights and group scales.
//
//   Y[m][n] = bf16( sum over groups of s[n][g] * ( sum_{k in g} X[m][k] (u[n][k] - z[n][g]) ) )
//
// For few rows the weights' bytes bound it: half a byte each, read once. The
// codes go from shared memory straight into tensor-core operands: the bits
// 0x4300 | u are the bf16 number 128 + u, and subtracting 128 + z leaves the
// integer u - z exactly, so the products see the weights without a rounding;
// each group's sum is scaled in fp32.
//   A = 16 weight rows x 16 k, B = 16 k x 8 rows of X (m16n8k16): few rows of X
//   waste columns of a narrow operand instead of rows of a wide one.
// The k of one product step need not be neighbours as long as A and B agree: a
// lane takes its k as whole 32-bit words of the weight row (eight codes, two
// steps), and the nibbles q and q + 4 of a word are one operand pair.
//
// The sum's order is fixed by (K, group): K is cut into blocks of 128 and the
// blocks into S segments; a segment's groups are added in ascending order, and
// the segments' sums in order. The number of rows decides only who computes
// what:
//   - few rows (gemm_int4_rows_kernel, M <= 16): a warp a segment, the CTA's
//     warps share 16 or 32 weight rows; every warp has its own ring of TMA
//     copies and nobody waits for anybody before the final sum;
//   - more (gemm_int4_tile_kernel): a CTA a tile of 128 weight rows x 64 rows of
//     X, both staged by TMA for all warps; it walks the segments, or, where the
//     tiles would not fill the GPU, the CTAs of a cluster take one each.
#include "attn_common.cuh"
#include "bi_internal.h"
#include "bi_ptx.cuh"
#include "kv_int4.cuh"

namespace bi {
namespace {

constexpr int kBlockK = 128;                   // k of a staged block
constexpr int kMaxSegments = 8;

struct GemmI4Params {
    const uint16_t *S;       // [N][groups] bf16
    const uint8_t *Z;        // [N][groups] or null
    uint16_t *Y;             // [M][ldy]
    int64_t ldy, M, N, K, group, groups, blocks;
    int32_t segments;
    unsigned *status;
};

// (scale as fp32, -(128 + z) as a bf16 pair) of weight row n's group at k.
__device__ __forceinline__ uint2 load_scale(const GemmI4Params &p, int64_t n, int64_t k) {
    uint2 v = make_uint2(0u, 0xC308C308u);
    if (n < p.N && k < p.K) {
        const int64_t gi = n * p.groups + k / p.group;
        v.x = static_cast<uint32_t>(p.S[gi]) << 16;
        if (p.Z) v.y = 0xC300C300u | ((p.Z[gi] & 15u) * 0x00010001u);
    }
    return v;
}

// Where lane (g, c) finds its operands of a block, GS k a scale: word j of group
// `sub` holds k = GS sub + (GS / 4) c + 8 j and the seven after it. Weight rows
// are 64 bytes a block (64-byte swizzle), rows of X two boxes of 64 k (128-byte swizzle).
template <int GS>
__device__ __forceinline__ void load_words(uint32_t w_row, int row, int sub, int cq, uint32_t (&w)[GS / 32]) {
    const int byte = GS / 2 * sub + GS / 8 * cq;
    const uint32_t at = w_row + ((((byte >> 4) ^ (row >> 1)) & 3) << 4) + (byte & 15);
    if constexpr (GS == 128)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
    else if constexpr (GS == 64)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at));
}
// The B operands of word j: (b0, b1) of its two steps. `rows` rows of X a box.
template <int GS>
__device__ __forceinline__ void load_x(uint32_t x_tile, int rows, int row, int sub, int cq, int j, uint32_t (&b)[4]) {
    const int k = GS * sub + GS / 4 * cq + 8 * j;
    uint32_t x0, x1, x2, x3;
    ld_shared_v4(x_tile + ((k >> 6) * rows + row) * 128 + ((((k >> 3) ^ row) & 7) << 4), x0, x1, x2, x3);
    b[0] = zip16<0>(x0, x2), b[1] = zip16<1>(x0, x2), b[2] = zip16<0>(x1, x3), b[3] = zip16<1>(x1, x3);
}
__device__ __forceinline__ void expand_weights(uint32_t w, uint32_t z2, uint32_t (&a)[4]) {
    a[0] = fma_bf16x2(i4_pair<0>(w), 0x3F803F80u, z2);
    a[1] = fma_bf16x2(i4_pair<1>(w), 0x3F803F80u, z2);
    a[2] = fma_bf16x2(i4_pair<2>(w), 0x3F803F80u, z2);
    a[3] = fma_bf16x2(i4_pair<3>(w), 0x3F803F80u, z2);
}

// acc += the block's groups, each scaled, for 16 MR weight rows x 8 NT rows of X.
// `sc`: [16 MR][groups of the block] scales.
template <int GS, int MR, int NT>
__device__ __forceinline__ void block_product(uint32_t w_tile, uint32_t x_tile, int x_rows, int x_row0, const uint2 *sc,
                                              int gq, int cq, float (&acc)[MR][NT][4]) {
    constexpr int kSub = kBlockK / GS;
#pragma unroll
    for (int sub = 0; sub < kSub; ++sub) {
        uint32_t w[MR][2][GS / 32];
        uint2 s[MR][2];
        float part[MR][NT][4];
#pragma unroll
        for (int m = 0; m < MR; ++m) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = 16 * m + 8 * h + gq;
                load_words<GS>(w_tile + row * (kBlockK / 2), row, sub, cq, w[m][h]);
                s[m][h] = sc[row * kSub + sub];
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) part[m][t][e] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < GS / 32; ++j) {
            uint32_t a[MR][2][4];
#pragma unroll
            for (int m = 0; m < MR; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) expand_weights(w[m][h][j], s[m][h].y, a[m][h]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                uint32_t b[4];
                load_x<GS>(x_tile, x_rows, x_row0 + 8 * t + gq, sub, cq, j, b);
#pragma unroll
                for (int m = 0; m < MR; ++m)
                    mma_16816(part[m][t], a[m][0][0], a[m][1][0], a[m][0][1], a[m][1][1], b[0], b[1]);
#pragma unroll
                for (int m = 0; m < MR; ++m)
                    mma_16816(part[m][t], a[m][0][2], a[m][1][2], a[m][0][3], a[m][1][3], b[2], b[3]);
            }
        }
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[m][t][e] = __fmaf_rn(__uint_as_float(s[m][e >> 1].x), part[m][t][e], acc[m][t][e]);
    }
}

__device__ __forceinline__ void store_y(const GemmI4Params &p, int64_t m, int64_t n, float y) {
    if (m < p.M && n < p.N && BI_IN_BOUNDS(m * p.ldy + n < (p.M - 1) * p.ldy + p.N, p.status))
        p.Y[m * p.ldy + n] = static_cast<uint16_t>(pack_bf16x2(__float_as_uint(y), 0u) & 0xFFFFu);
}

// ---------------------------------------------------------------- few rows ---

constexpr int kRing = 3;                       // blocks of a warp in shared memory
template <int MR, int NT>
constexpr int rows_stage() { return MR * 16 * (kBlockK / 2) + NT * 8 * kBlockK * 2; }   // W, X
template <int GS, int MR, int NT>
constexpr int rows_warp() { return kRing * rows_stage<MR, NT>() + 2 * 16 * MR * (kBlockK / GS) * 8; }

template <int GS, int MR, int NT>
__global__ void __launch_bounds__(32 * kMaxSegments)
gemm_int4_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const GemmI4Params p) {
    constexpr int kSub = kBlockK / GS, kStage = rows_stage<MR, NT>(), kWBytes = MR * 16 * (kBlockK / 2);
    constexpr int kScales = 16 * MR * kSub, kPer = (kScales + 31) / 32;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t full[kMaxSegments][kRing];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, cq = lane & 3;
    uint8_t *ring = smem + warp * kRing * kStage;
    uint2 *scales = reinterpret_cast<uint2 *>(smem + p.segments * kRing * kStage) + warp * 2 * kScales;
    if (lane == 0) {
        for (int k = 0; k < kRing; ++k) mbar_init(&full[warp][k], 1);
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    __syncwarp();
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * MR);
    const int b0 = static_cast<int>(warp * p.blocks / p.segments), b1 = static_cast<int>((warp + 1) * p.blocks / p.segments);
    auto issue = [&](int blk) {                            // one lane
        const int slot = (blk - b0) % kRing;
        uint8_t *dst = ring + slot * kStage;
        uint64_t *bar = &full[warp][slot];
        mbar_arrive_expect_tx(bar, kStage);
        tma_load_2d(dst, &tmW, bar, blk * (kBlockK / 2), static_cast<int32_t>(n0));
        tma_load_2d(dst + kWBytes, &tmX, bar, blk * kBlockK, 0);
        tma_load_2d(dst + kWBytes + NT * 8 * 128, &tmX, bar, blk * kBlockK + 64, 0);
    };
    uint2 sv[kPer];
    auto fetch_scales = [&](int blk) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int v = lane + 32 * i;
            sv[i] = v < kScales ? load_scale(p, n0 + v / kSub, static_cast<int64_t>(blk) * kBlockK + v % kSub * GS) : make_uint2(0u, 0u);
        }
    };
    if (lane == 0)
        for (int blk = b0; blk < b1 && blk < b0 + kRing; ++blk) issue(blk);
    float acc[MR][NT][4];
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][t][e] = 0.0f;
    fetch_scales(b0);
    bool ok = true;
    for (int blk = b0; blk < b1; ++blk) {
        const int i = blk - b0, slot = i % kRing;
        uint2 *sc = scales + (i & 1) * kScales;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (lane + 32 * k < kScales) sc[lane + 32 * k] = sv[k];
        if (blk + 1 < b1) fetch_scales(blk + 1);
        ok = mbar_wait(&full[warp][slot], (i / kRing) & 1, nullptr);
        __syncwarp();
        if (!__all_sync(0xffffffffu, ok)) {                // ran out: report; the copies in flight get another limit
            if (lane == 0) {
                atomicOr(p.status, kDevTimeout);
                for (int k = 0; k < kRing && blk + k < b1; ++k) mbar_wait(&full[warp][(i + k) % kRing], ((i + k) / kRing) & 1, nullptr);
            }
            break;
        }
        const uint32_t w_tile = smem_u32(ring + slot * kStage);
        block_product<GS, MR, NT>(w_tile, w_tile + kWBytes, 8 * NT, 0, sc, gq, cq, acc);
        __syncwarp();                                      // every lane has read the slot
        if (lane == 0 && blk + kRing < b1) issue(blk + kRing);
    }
    // the segments' sums, added in order (the rings are done with: each warp's sums lie in its own)
    constexpr int kCols = 8 * NT + 1;
    float *red = reinterpret_cast<float *>(ring);
    static_assert(16 * MR * kCols * 4 <= kRing * kStage, "the sums fit the ring");
    __syncwarp();
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) red[(16 * m + gq + 8 * (e >> 1)) * kCols + 8 * t + 2 * cq + (e & 1)] = acc[m][t][e];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * MR * 8 * NT; i += blockDim.x) {
        const int r = i % (16 * MR), t = i / (16 * MR);
        if (t >= p.M) break;
        const float *v = reinterpret_cast<const float *>(smem) + r * kCols + t;
        float y = v[0];
        for (int s = 1; s < p.segments; ++s) y += v[s * (kRing * kStage / 4)];
        store_y(p, t, n0 + r, y);
    }
}

// -------------------------------------------------------------------- tiles ---

constexpr int kTileN = 128, kTileM = 64;       // weight rows, rows of X of a CTA
constexpr int kTileThreads = 256;              // warps: four of 32 weight rows x two of 32 rows of X
constexpr int kTileStages = 3;
constexpr int kTileW = kTileN * (kBlockK / 2), kTileStage = kTileW + kTileM * kBlockK * 2;   // 24 KB
template <int GS>
constexpr int tile_smem() { return 1024 + kTileStages * kTileStage + 2 * kTileN * (kBlockK / GS) * 8; }
static_assert(kTileN * kTileM * 4 <= kTileStages * kTileStage, "a segment's sums fit the stages");

// One segment a CTA (a cluster's ranks in segment order), or all segments in turn (SPLIT false).
template <int GS, bool SPLIT>
__global__ void __launch_bounds__(kTileThreads, SPLIT ? 2 : 1)
gemm_int4_tile_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const GemmI4Params p) {
    constexpr int kSub = kBlockK / GS, kScales = kTileN * kSub, kPer = (kScales + kTileThreads - 1) / kTileThreads;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint2 *scales = reinterpret_cast<uint2 *>(smem + kTileStages * kTileStage);
    __shared__ uint64_t full[kTileStages];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gq = lane >> 2, cq = lane & 3, wn = warp & 3, wm = warp >> 2;
    if (tid == 0) {
        for (int k = 0; k < kTileStages; ++k) mbar_init(&full[k], 1);
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    __syncthreads();
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    // tiles: X's fastest, so that the CTAs at work together share weight rows
    const int rank = SPLIT ? static_cast<int>(blockIdx.x % p.segments) : 0;
    const int64_t tile = SPLIT ? blockIdx.x / p.segments : blockIdx.x;
    const int64_t tiles_m = (p.M + kTileM - 1) / kTileM;
    const int64_t m0 = tile % tiles_m * kTileM, n0 = tile / tiles_m * kTileN;
    const int first = SPLIT ? static_cast<int>(rank * p.blocks / p.segments) : 0;
    const int last = SPLIT ? static_cast<int>((rank + 1) * p.blocks / p.segments) : static_cast<int>(p.blocks);
    auto issue = [&](int blk) {                            // thread 0
        const int slot = (blk - first) % kTileStages;
        uint8_t *dst = smem + slot * kTileStage;
        mbar_arrive_expect_tx(&full[slot], kTileStage);
        tma_load_2d(dst, &tmW, &full[slot], blk * (kBlockK / 2), static_cast<int32_t>(n0));
        tma_load_2d(dst + kTileW, &tmX, &full[slot], blk * kBlockK, static_cast<int32_t>(m0));
        tma_load_2d(dst + kTileW + kTileM * 128, &tmX, &full[slot], blk * kBlockK + 64, static_cast<int32_t>(m0));
    };
    uint2 sv[kPer];
    auto fetch_scales = [&](int blk) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int v = tid + kTileThreads * i;
            sv[i] = v < kScales ? load_scale(p, n0 + v / kSub, static_cast<int64_t>(blk) * kBlockK + v % kSub * GS) : make_uint2(0u, 0u);
        }
    };
    if (tid == 0)
        for (int blk = first; blk < last && blk < first + kTileStages - 1; ++blk) issue(blk);
    float acc[2][4][4], tot[2][4][4];
    auto clear = [&](float (&v)[2][4][4]) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[m][t][e] = 0.0f;
    };
    clear(acc);
    fetch_scales(first);
    int seg = 0;                                           // SPLIT false: the segment at work, and its end
    int seg_end = static_cast<int>(p.blocks / p.segments);
    bool ok = true;
    for (int blk = first; blk < last; ++blk) {
        const int i = blk - first, slot = i % kTileStages;
        uint2 *sc = scales + (i & 1) * kScales;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (tid + kTileThreads * k < kScales) sc[tid + kTileThreads * k] = sv[k];
        if (blk + 1 < last) fetch_scales(blk + 1);
        ok = mbar_wait(&full[slot], (i / kTileStages) & 1, nullptr);
        if (__syncthreads_or(!ok)) {                       // (and: the scales are written, block i - 1 is done with)
            if (tid == 0) {                                // ran out: report; the copies in flight get another limit
                atomicOr(p.status, kDevTimeout);
                for (int k = 0; k < kTileStages - 1 && blk + k < last; ++k)
                    mbar_wait(&full[(i + k) % kTileStages], ((i + k) / kTileStages) & 1, nullptr);
            }
            break;
        }
        if (tid == 0 && blk + kTileStages - 1 < last) issue(blk + kTileStages - 1);
        const uint32_t w_tile = smem_u32(smem + slot * kTileStage);
        block_product<GS, 2, 4>(w_tile + wn * 32 * (kBlockK / 2), w_tile + kTileW, kTileM, 32 * wm, sc + wn * 32 * kSub, gq, cq, acc);
        if (!SPLIT && blk + 1 == seg_end) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) tot[m][t][e] = seg == 0 ? acc[m][t][e] : tot[m][t][e] + acc[m][t][e];
            clear(acc);
            ++seg;
            seg_end = static_cast<int>((seg + 1) * p.blocks / p.segments);
        }
    }
    // the tile's sums through shared memory, [row of X][weight row] with the rows four apart in banks
    constexpr int kLd = kTileN + 4;
    static_assert(kTileM * kLd * 4 <= kTileStages * kTileStage, "the tile's sums fit the stages");
    float *red = reinterpret_cast<float *>(smem);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[(32 * wm + 8 * t + 2 * cq + (e & 1)) * kLd + 32 * wn + 16 * m + gq + 8 * (e >> 1)] =
                    SPLIT ? acc[m][t][e] : tot[m][t][e];
    if (SPLIT)
        cluster_sync();
    else
        __syncthreads();
    const int ranks = SPLIT ? p.segments : 1;
    // each CTA of the cluster adds and stores its share of the tile's rows of X
    for (int i = tid; i < kTileM * (kTileN / 8); i += kTileThreads) {
        const int t = i / (kTileN / 8), n = i % (kTileN / 8) * 8;
        if ((SPLIT && t % ranks != rank) || m0 + t >= p.M || n0 + n >= p.N) continue;
        float y[8];
        const uint32_t at = smem_u32(red + t * kLd + n);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            float4 x = *reinterpret_cast<const float4 *>(red + t * kLd + n + 4 * v);
            if (SPLIT) {
                for (int s = 0; s < ranks; ++s) {
                    float4 r;
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "r"(mapa_shared(at + 16 * v, s)));
                    x = s == 0 ? r : make_float4(x.x + r.x, x.y + r.y, x.z + r.z, x.w + r.w);
                }
            }
            y[4 * v] = x.x, y[4 * v + 1] = x.y, y[4 * v + 2] = x.z, y[4 * v + 3] = x.w;
        }
        if (BI_IN_BOUNDS((m0 + t) * p.ldy + n0 + n + 8 <= (p.M - 1) * p.ldy + p.N, p.status))   // N % 8 == 0
            st_global_v4(p.Y + (m0 + t) * p.ldy + n0 + n, pack_bf16x2(__float_as_uint(y[0]), __float_as_uint(y[1])),
                         pack_bf16x2(__float_as_uint(y[2]), __float_as_uint(y[3])),
                         pack_bf16x2(__float_as_uint(y[4]), __float_as_uint(y[5])),
                         pack_bf16x2(__float_as_uint(y[6]), __float_as_uint(y[7])));
    }
    if (SPLIT) cluster_sync();                             // no CTA leaves while its sums are read
}

// ----------------------------------------------------------------- launches ---

template <int GS, int MR, int NT>
bi_status launch_rows(const CUtensorMap &tmW, const CUtensorMap &tmX, const GemmI4Params &p, cudaStream_t s) {
    static unsigned long long configured = 0;
    constexpr int most = 1024 + kMaxSegments * rows_warp<GS, MR, NT>();
    static_assert(most <= 232448 - 1024, "one CTA's shared memory");
    if (ensure_smem_attr(reinterpret_cast<const void *>(gemm_int4_rows_kernel<GS, MR, NT>), most, &configured) != BI_OK)
        return BI_ERR_CUDA;
    const int64_t grid = (p.N + 16 * MR - 1) / (16 * MR);
    return launch_pdl(gemm_int4_rows_kernel<GS, MR, NT>, dim3(static_cast<unsigned>(grid)), dim3(32 * p.segments),
                      1024 + p.segments * rows_warp<GS, MR, NT>(), s, tmW, tmX, p);
}

template <int GS, bool SPLIT>
bi_status launch_tiles(const CUtensorMap &tmW, const CUtensorMap &tmX, const GemmI4Params &p, int64_t tiles, cudaStream_t s) {
    static unsigned long long configured = 0;
    if (ensure_smem_attr(reinterpret_cast<const void *>(gemm_int4_tile_kernel<GS, SPLIT>), tile_smem<GS>(), &configured) != BI_OK)
        return BI_ERR_CUDA;
    const int64_t grid = tiles * (SPLIT ? p.segments : 1);
    if (grid > 0x7FFFFFFF) return BI_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = tile_smem<GS>();
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(SPLIT ? p.segments : 1);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = SPLIT ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, gemm_int4_tile_kernel<GS, SPLIT>, tmW, tmX, p) == cudaSuccess) return BI_OK;
    cudaGetLastError();
    return BI_ERR_CUDA;
}

template <int GS>
bi_status launch_group(const void *X, int64_t ldx, const uint8_t *W, GemmI4Params &p, int sms, cudaStream_t s) {
    const bool rows = p.M <= 16;
    const int nt = p.M <= 8 ? 1 : 2;
    // 32 weight rows a CTA halve the reads of X; 16 where that would leave SMs without a CTA
    const int mr = p.M > 4 && p.N >= 32 * 2 * static_cast<int64_t>(sms) ? 2 : 1;
    CUtensorMap tmW{}, tmX{};
    if (make_tmap_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, W, p.K / 2, p.N, p.K / 2, kBlockK / 2, rows ? 16 * mr : kTileN,
                     CU_TENSOR_MAP_SWIZZLE_64B) != BI_OK ||
        make_tmap_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, X, p.K, p.M, ldx * 2, 64, rows ? 8 * nt : kTileM,
                     CU_TENSOR_MAP_SWIZZLE_128B) != BI_OK)
        return BI_ERR_CUDA;
    if (rows) {
        if (mr == 1) return nt == 1 ? launch_rows<GS, 1, 1>(tmW, tmX, p, s) : launch_rows<GS, 1, 2>(tmW, tmX, p, s);
        return nt == 1 ? launch_rows<GS, 2, 1>(tmW, tmX, p, s) : launch_rows<GS, 2, 2>(tmW, tmX, p, s);
    }
    // one CTA a segment while the tiles alone would not keep two CTAs an SM at work
    const int64_t tiles = (p.N + kTileN - 1) / kTileN * ((p.M + kTileM - 1) / kTileM);
    if (p.segments > 1 && tiles < 4 * static_cast<int64_t>(sms)) return launch_tiles<GS, true>(tmW, tmX, p, tiles, s);
    return launch_tiles<GS, false>(tmW, tmX, p, tiles, s);
}

}  // namespace

bi_status launch_gemm_int4(const void *X, int64_t ldx, const uint8_t *W, const void *scales, const uint8_t *zeros, void *Y,
                           int64_t ldy, int64_t M, int64_t N, int64_t K, int64_t group, cudaStream_t s) {
    int dev = 0;
    const DeviceInfo *info = nullptr;
    const bi_status st = current_device(&dev, &info);
    if (st != BI_OK) return st;
    GemmI4Params p{static_cast<const uint16_t *>(scales), zeros, static_cast<uint16_t *>(Y), ldy, M, N, K, group, K / group,
                   (K + kBlockK - 1) / kBlockK, 0, device_status_word()};
    p.segments = static_cast<int32_t>(p.blocks < 4 ? 1 : p.blocks / 4 > kMaxSegments ? kMaxSegments : p.blocks / 4);
    if (group == 32) return launch_group<32>(X, ldx, W, p, info->sm_count, s);
    if (group == 64) return launch_group<64>(X, ldx, W, p, info->sm_count, s);
    return launch_group<128>(X, ldx, W, p, info->sm_count, s);
}

}  // namespace bi
