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
// The sum's order is fixed by (K, group): K is cut into units of 256 and the
// units into S segments; a segment's groups (of longer ones, each 128 k) are added
// in ascending order, and the segments' sums in order. The number of rows of X
// decides only who computes what:
//   - few rows (gemm_int4_rows_kernel, M <= 16): a warp (two for M > 8) a
//     segment, with its own ring of TMA copies, so that nobody waits for another
//     segment before the final sum;
//   - more (gemm_int4_tile_kernel): a CTA a tile of 128 weight rows x 32 or 64
//     rows of X, both staged by TMA for all warps; it walks the segments, or the CTAs
//     of a cluster take one each.
//
// What bounds it: a word of eight codes costs 11 instructions to expand (three
// shifts, four logic operations, four multiply-adds), and the integer pipe, the
// packed bf16 pipe and mma.sync overlap only partly on this GPU: an expansion
// alone takes 16.4-17.6 cycles per warp and scheduler, with one product 21.6-24.7
// (17 and 8 apart; measured with independent chains). At the weights' HBM rate a
// scheduler has 22 cycles for a word; tiles spend 44 % of their cycles in mma.sync,
// 38 % and 19 % in the other two. Measured (GB300, weights from HBM), M = 1:
// 6144 x 4096, g = 128 7.7 us (1.7 TB/s; without the products 4.5), 24576 x 4096
// 18.3 us (2.9 TB/s; 10.4); M = 16, 24576 x 4096, g = 64 with zeros 29.8 us; M = 200,
// 4096 x 12288 111 us (g = 128) and 118 us (g = 32); M = 2048, 6144 x 4096 421 us
// (245 TFLOP/s). bi_gemm_bf16 over bf16 weights, which gives other bits, takes 16.6,
// 48.9, 49.9 (M = 16), 32 (M = 200) and 66 us: from 33 rows on it is the faster one
// (6144 x 4096: from 17). A form with the expanded weights in tensor memory and tcgen05
// products took 13.9, 39.9, 48, 88, 146 and 334 us in that order: faster for many
// rows, but every M has to give the same bits, which the two products do not, and
// few rows are what the call is for. Tiles of 128 rows of X (half the expansions a
// product, eight warps an SM) took 387 us at M = 2048, but 154 and 180 at M = 200;
// X's operand pairs made once, in place, a stage ahead, 5-7 % more than here.
#include "attn_common.cuh"
#include "bi_internal.h"
#include "bi_ptx.cuh"
#include "kv_int4.cuh"

namespace bi {
namespace {

constexpr int kBlockK = 128;                   // a group's longest product chain
constexpr int kUnitK = 256;                    // k of which segments are made
constexpr int kMaxSegments = 8;

struct GemmI4Params {
    const uint32_t *S;       // [N][groups] bf16, as words
    const uint32_t *Z;       // [N][groups] bytes, as words, or null
    uint16_t *Y;             // [M][ldy]
    int64_t ldy, M, N, s_last, z_last;       // last words of S and Z
    int32_t K;
    int32_t groups, group, blocks, units, segments;   // blocks: of kBlockK; units: of kUnitK
    int32_t x_rows;          // rows kernel: staged rows of X (1, 2, 4, 8 or 16)
    unsigned *status;
};

// The scales and zeros of KB staged k, GS k a scale: for each weight row the
// 32-bit words that hold them (their place in the first word depends on the row).
template <int GS, int KB>
struct ScaleTile {
    static constexpr int kSub = KB / GS;                          // groups (or a longer group's 128 k each)
    static constexpr int kSWords = (kSub + 1) / 2 + (kSub > 1);   // words of kSub 16-bit scales at any halfword
    static constexpr int kZWords = (kSub + 3) / 4 + (kSub > 1);   // words of kSub bytes at any byte
    static constexpr int bytes(int rows) { return rows * (kSWords + kZWords) * 4; }
};

__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Starts the copies of a block's scales and zeros for ROWS weight rows (of a tile of TILE) by THREADS threads, each of
// which arrives on the barrier once its copies have landed. row: the first of the rows in the tile; e0: its element of
// the first group in the arrays. Words past the arrays (rows past N, groups past K) repeat the last one.
template <int GS, int KB, int ROWS, int TILE, int THREADS, bool ZEROS>
__device__ __forceinline__ void stage_scales(const GemmI4Params &p, uint32_t dst, uint64_t *bar, int row, int64_t e0, int thread) {
    using T = ScaleTile<GS, KB>;
#pragma unroll
    for (int i = 0; i < (ROWS * T::kSWords + THREADS - 1) / THREADS; ++i) {
        const int v = thread + i * THREADS, r = v / T::kSWords, w = v % T::kSWords;
        if (v < ROWS * T::kSWords) cp_async_4(dst + (row * T::kSWords + v) * 4, p.S + min(((e0 + r * p.groups) >> 1) + w, p.s_last));
    }
    if (ZEROS) {
#pragma unroll
        for (int i = 0; i < (ROWS * T::kZWords + THREADS - 1) / THREADS; ++i) {
            const int v = thread + i * THREADS, r = v / T::kZWords, w = v % T::kZWords;
            if (v < ROWS * T::kZWords)
                cp_async_4(dst + (TILE * T::kSWords + row * T::kZWords + v) * 4, p.Z + min(((e0 + r * p.groups) >> 2) + w, p.z_last));
        }
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// (scale as fp32, -(128 + z) as a bf16 pair) of a staged row and its `at`-th staged group. `e` is the element of
// (row, the first staged group) modulo 4: tiles begin at multiples of 16 rows, so (row % 8) * groups + group will do.
template <int GS, int KB, int ROWS, bool ZEROS>
__device__ __forceinline__ void read_scale(const uint8_t *tile, int row, int e, int at, bool in, float &s, uint32_t &z2) {
    using T = ScaleTile<GS, KB>;
    const uint32_t bits = *reinterpret_cast<const uint16_t *>(tile + row * T::kSWords * 4 + (e & 1) * 2 + at * 2);
    s = in ? __uint_as_float(bits << 16) : 0.0f;
    z2 = kBf16x2_m136;
    if (ZEROS) z2 = __byte_perm(tile[(ROWS * T::kSWords + row * T::kZWords) * 4 + (e & 3) + at] & 15u, 0xC3u, 0x4040);
}

// The first product of a chain: D = A B.
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Where lane (g, c) finds its operands among KB staged k, GS k a scale: word j of
// group `sub` holds k = GS sub + (GS / 4) c + 8 j and the seven after it. Weight
// rows are KB / 2 bytes with the TMA's swizzle of that width, rows of X boxes of 64 k
// with the 128-byte swizzle, which goes by the address: a 16-byte piece is exchanged
// by the address's 128-byte line modulo 8. Boxes lie x_stride apart, which is 2 or 6
// lines modulo 8 (1 where X has one row): the pieces that eight lanes load at once, of
// two rows and (GS = 128) two boxes, are then in all the banks. With GS = 32 they are
// four neighbours of two rows, which have to be four lines apart: x_row.
template <int GS, int KB>
__device__ __forceinline__ void load_words(uint32_t w_row, int row, int sub, int cq, uint32_t (&w)[GS / 32]) {
    const int byte = GS / 2 * sub + GS / 8 * cq;
    const uint32_t at = w_row + (((byte >> 4) ^ (KB == 256 ? row & 7 : (row >> 1) & 3)) << 4) + (byte & 15);
    if constexpr (GS == 128)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
    else if constexpr (GS == 64)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at));
}
// The row of X (of eight) that column n of a product takes.
template <int GS>
__device__ __forceinline__ int x_row(int n) { return GS == 32 ? ((n & 1) << 2) | (n >> 1) : n; }
// Bytes between the boxes of X: of `rows` rows, and two more lines where four rows or more make their number 4 or 0
// modulo 8.
__host__ __device__ constexpr int x_box(int rows) { return rows * 128 + (rows >= 4 ? 256 : 0); }
// Address of word 0's piece of X (x_tile begins at a multiple of 1024).
template <int GS>
__device__ __forceinline__ uint32_t x_piece(uint32_t x_tile, int x_stride, int row, int sub, int cq) {
    const int k = GS * sub + GS / 4 * cq, line = (k >> 6) * (x_stride >> 7) + row;
    return x_tile + line * 128 + ((((k >> 3) ^ line) & 7) << 4);
}
// The B operands of word j: (b0, b1) of its two steps.
__device__ __forceinline__ void load_x(uint32_t piece, int j, uint32_t (&b)[4]) {
    uint32_t x0, x1, x2, x3;
    ld_shared_v4(piece ^ (j << 4), x0, x1, x2, x3);
    b[0] = zip16<0>(x0, x2), b[1] = zip16<1>(x0, x2), b[2] = zip16<0>(x1, x3), b[3] = zip16<1>(x1, x3);
}
__device__ __forceinline__ void expand_weights(uint32_t w, uint32_t z2, uint32_t (&a)[4]) {
    a[0] = fma_bf16x2(i4_pair<0>(w), 0x3F803F80u, z2);
    a[1] = fma_bf16x2(i4_pair<1>(w), 0x3F803F80u, z2);
    a[2] = fma_bf16x2(i4_pair<2>(w), 0x3F803F80u, z2);
    a[3] = fma_bf16x2(i4_pair<3>(w), 0x3F803F80u, z2);
}

// Block -> its first group, and on to the next: a block has several groups, or a group several blocks.
template <int GS>
struct GroupCursor {
    int group, left;         // left: blocks of the group still to come, this one included
    __device__ __forceinline__ GroupCursor(const GemmI4Params &p, int blk) {
        const int per = GS < kBlockK ? 1 : p.group / kBlockK;
        group = GS < kBlockK ? blk * (kBlockK / GS) : blk / per;
        left = per - (GS < kBlockK ? 0 : blk % per);
    }
    __device__ __forceinline__ void next(const GemmI4Params &p) {
        if (GS < kBlockK)
            group += kBlockK / GS;
        else if (--left == 0)
            ++group, left = p.group / kBlockK;
    }
};

// acc += KB staged k, each group scaled, for weight rows row0 .. row0 + 16 MR - 1 of
// the staged ROWS and 8 NT rows of X from x_row0 (x_mask: rows that are not there
// repeat others; their columns are not stored). `g`: the first group; k_left: k from
// the first one to K's end.
template <int GS, int KB, int MR, int NT, int ROWS, bool ZEROS>
__device__ __forceinline__ void product(uint32_t w_tile, uint32_t x_tile, const uint8_t *sc, int row0, int x_stride, int x_row0, int x_mask,
                                        int groups, const GroupCursor<GS> &g, int k_left, int gq, int cq,
                                        float (&acc)[MR][NT][4]) {
    constexpr int kSub = KB / GS;
    const int e = gq * groups + g.group;
#pragma unroll
    for (int sub = 0; sub < kSub; ++sub) {
        uint32_t w[MR][2][GS / 32], xp[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) xp[t] = x_piece<GS>(x_tile, x_stride, x_row0 + 8 * t + (x_row<GS>(gq) & x_mask), sub, cq);
        float s[MR][2];
        uint32_t z2[MR][2];
        float part[MR][NT][4];
#pragma unroll
        for (int m = 0; m < MR; ++m) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = row0 + 16 * m + 8 * h + gq;
                load_words<GS, KB>(w_tile + row * (KB / 2), row, sub, cq, w[m][h]);
                // a group of more than 128 k: the second 128 are the next group's only where the first one's is done
                const int at = GS < kBlockK || sub == 0 ? sub : g.left == 1;
                read_scale<GS, KB, ROWS, ZEROS>(sc, row, e, at, kSub == 1 || sub * GS < k_left, s[m][h], z2[m][h]);
            }
        }
#pragma unroll
        for (int j = 0; j < GS / 32; ++j) {
            uint32_t a[MR][2][4];
#pragma unroll
            for (int m = 0; m < MR; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) expand_weights(w[m][h][j], z2[m][h], a[m][h]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                uint32_t b[4];
                load_x(xp[t], j, b);
#pragma unroll
                for (int m = 0; m < MR; ++m) {
                    if (j == 0)
                        mma_first(part[m][t], a[m][0][0], a[m][1][0], a[m][0][1], a[m][1][1], b[0], b[1]);
                    else
                        mma_16816(part[m][t], a[m][0][0], a[m][1][0], a[m][0][1], a[m][1][1], b[0], b[1]);
                }
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
                for (int e = 0; e < 4; ++e) acc[m][t][e] = __fmaf_rn(s[m][e >> 1], part[m][t][e], acc[m][t][e]);
    }
}

__device__ __forceinline__ void store_y(const GemmI4Params &p, int64_t m, int64_t n, float y) {
    if (m < p.M && n < p.N && BI_IN_BOUNDS(m * p.ldy + n < (p.M - 1) * p.ldy + p.N, p.status))
        p.Y[m * p.ldy + n] = static_cast<uint16_t>(pack_bf16x2(__float_as_uint(y), 0u) & 0xFFFFu);
}

// ---------------------------------------------------------------- few rows ---

// CTAs walk the tiles of 32 weight rows a warp; a segment's ring of kRing stages runs on from one tile to the next.
// Two row tiles a warp, and KB = 256 k a stage where X has at most eight rows, spread the waits, the copies' issue and
// the operands of X over more weights; with up to 16 rows of X, two warps (of 64 weight rows) share a segment's stages,
// so that 16 warps fit an SM either way.
constexpr int kRing = 2;
template <int NT>
constexpr int rows_n() { return 32 * NT; }     // weight rows of a CTA: NT warps a segment
template <int NT>
constexpr int rows_kb() { return NT == 1 ? 256 : 128; }
template <int NT>
constexpr int rows_w() { return rows_n<NT>() * (rows_kb<NT>() / 2); }
template <int NT>
constexpr int rows_sums() { return rows_n<NT>() * (8 * NT + 1); }   // floats of a segment's sums
template <int GS, int NT>
constexpr int rows_stage(int x_rows) {
    return rows_w<NT>() + (rows_kb<NT>() / 64 * x_box(x_rows) + ScaleTile<GS, rows_kb<NT>()>::bytes(rows_n<NT>()) + 1023) / 1024 * 1024;
}
template <int NT>
constexpr int rows_buffers() { return NT == 1 ? 2 : 1; }       // of the sums
template <int GS, int NT>
constexpr int rows_segment(int x_rows) { return kRing * rows_stage<GS, NT>(x_rows) + rows_buffers<NT>() * rows_sums<NT>() * 4; }

template <int GS, int NT, bool ZEROS>
__global__ void __launch_bounds__(32 * kMaxSegments * NT, NT == 1 ? 2 : 1)
gemm_int4_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const GemmI4Params p) {
    constexpr int KB = rows_kb<NT>(), kBlocks = KB / kBlockK, kW = rows_w<NT>(), kCols = 8 * NT + 1, kSums = rows_sums<NT>();
    constexpr int kN = rows_n<NT>(), kBuffers = rows_buffers<NT>();
    const int x_stride = x_box(p.x_rows), x_bytes = KB / 64 * x_stride, stage_bytes = rows_stage<GS, NT>(p.x_rows);
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t full[kMaxSegments][kRing], empty[kMaxSegments][kRing];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, cq = lane & 3, seg = warp / NT, wn = warp % NT;
    uint8_t *ring = smem + seg * kRing * stage_bytes;                                      // a stage: W, X, scales
    float *sums = reinterpret_cast<float *>(smem + p.segments * kRing * stage_bytes);   // [kBuffers][segments][kSums]
    if (wn == 0 && lane == 0) {
        for (int k = 0; k < kRing; ++k) {
            mbar_init(&full[seg][k], 32 * NT + 1);         // the lanes' scale copies, and the TMA's bytes
            mbar_init(&empty[seg][k], NT);
        }
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (NT == 1)
        __syncwarp();
    else
        __syncthreads();
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    const int tiles = static_cast<int>((p.N + kN - 1) / kN);
    // the segment's stages of KB k
    const int b0 = static_cast<int>(static_cast<int64_t>(seg) * p.units / p.segments) * (kUnitK / KB);
    const int u1 = static_cast<int>(static_cast<int64_t>(seg + 1) * p.units / p.segments);
    const int b1 = KB == kUnitK ? u1 : min(p.blocks, 2 * u1);
    const GroupCursor<GS> g0(p, b0 * kBlocks);
    // the next stage to be copied (W and X by the segment's first warp, scales by each warp its rows'), its group, and
    // its slot
    int ft = blockIdx.x, fb = b0, fs = 0;
    GroupCursor<GS> fg = g0;
    int64_t row_e = (static_cast<int64_t>(ft) * kN + 32 * wn) * p.groups;   // element (the warp's first row, group 0)
    const int64_t step_e = static_cast<int64_t>(gridDim.x) * kN * p.groups;
    auto fill = [&]() {
        if (ft >= tiles) return;
        uint8_t *dst = ring + fs * stage_bytes;
        uint64_t *bar = &full[seg][fs];
        if (wn == 0 && lane == 0) {
            mbar_arrive_expect_tx(bar, kW + p.x_rows * KB * 2);
            tma_load_2d(dst, &tmW, bar, fb * (KB / 2), ft * kN);
#pragma unroll
            for (int k = 0; k < KB / 64; ++k)
                tma_load_2d(dst + kW + k * x_stride, &tmX, bar, fb * KB + 64 * k, 0);
        }
        stage_scales<GS, KB, 32, kN, 32, ZEROS>(p, smem_u32(dst + kW + x_bytes), bar, 32 * wn, row_e + fg.group, lane);
        if (++fs == kRing) fs = 0;
        for (int k = 0; k < kBlocks; ++k) fg.next(p);
        if (++fb == b1) fb = b0, fg = g0, ft += gridDim.x, row_e += step_e;
    };
    for (int k = 0; k < kRing; ++k) fill();
    int slot = 0, buf = 0;
    uint32_t parity = 0;
    bool ok = true;
    int tile = blockIdx.x, blk = b0;                       // the stage at work
    for (; tile < tiles; tile += gridDim.x, buf = (buf + 1) % kBuffers) {
        const int64_t n0 = static_cast<int64_t>(tile) * kN;
        float acc[2][NT][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][t][e] = 0.0f;
        GroupCursor<GS> g = g0;
        for (blk = b0; blk < b1 && ok; ++blk) {
            ok = __all_sync(0xffffffffu, mbar_wait(&full[seg][slot], parity, nullptr));
            __syncwarp();
            if (!ok) break;
            const uint8_t *st = ring + slot * stage_bytes;
            product<GS, KB, 2, NT, kN, ZEROS>(smem_u32(st), smem_u32(st) + kW, st + kW + x_bytes, 32 * wn, x_stride, 0,
                                                     NT == 1 ? p.x_rows - 1 : 7, p.groups, g, p.K - blk * KB, gq, cq, acc);
            for (int k = 0; k < kBlocks; ++k) g.next(p);
            __syncwarp();                                  // every lane has read the slot
            if (NT > 1) {
                if (lane == 0) mbar_arrive(&empty[seg][slot]);
                if (wn == 0) ok = __all_sync(0xffffffffu, mbar_wait(&empty[seg][slot], parity, nullptr));
            }
            if (ok) fill();
            if (++slot == kRing) slot = 0, parity ^= 1;
        }
        // the segments' sums, added in order
        float *mine = sums + (buf * p.segments + seg) * kSums + 32 * wn * kCols;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) mine[(16 * m + gq + 8 * (e >> 1)) * kCols + 8 * t + x_row<GS>(2 * cq + (e & 1))] = acc[m][t][e];
        if (__syncthreads_or(!ok)) {                       // (two buffers: the one before last has been read)
            // a wait of the CTA ran out: report; every segment's copies in flight, the stages from the one at work up to
            // the next to be copied, get another limit
            if (!ok && lane == 0) atomicOr(p.status, kDevTimeout);
            asm volatile("cp.async.wait_all;" ::: "memory");
            const int flying = (ft - tile) / static_cast<int>(gridDim.x) * (b1 - b0) + fb - blk;
            for (int k = 0; wn == 0 && k < flying; ++k) {
                mbar_wait(&full[seg][slot], parity, nullptr);
                if (++slot == kRing) slot = 0, parity ^= 1;
            }
            return;
        }
        for (int i = threadIdx.x; i < kN * 8 * NT; i += blockDim.x) {
            const int r = i % kN, t = i / kN;
            if (t >= p.M) break;
            const float *v = sums + buf * p.segments * kSums + r * kCols + t;
            float y = v[0];
            for (int s = 1; s < p.segments; ++s) y += v[s * kSums];
            store_y(p, t, n0 + r, y);
        }
        if (kBuffers == 1) __syncthreads();
    }
}

// -------------------------------------------------------------------- tiles ---

constexpr int kTileN = 128;                    // weight rows of a CTA
constexpr int kTileThreads = 256;              // warps: four of 32 weight rows x two of TM / 2 rows of X
constexpr int kTileW = kTileN * (kBlockK / 2); // 8 KB a stage
template <int TM>
constexpr int tile_stage() { return kTileW + (2 * x_box(TM) + 1023) / 1024 * 1024; }
template <int TM>
constexpr int tile_stages() { return TM == 64 ? 3 : 5; }
template <int GS, int TM>
constexpr int tile_smem() { return 1024 + tile_stages<TM>() * (tile_stage<TM>() + ScaleTile<GS, kBlockK>::bytes(kTileN)); }

// One segment a CTA (a cluster's ranks in segment order), or all segments in turn (SPLIT false).
template <int GS, int TM, bool SPLIT, bool ZEROS>
__global__ void __launch_bounds__(kTileThreads, TM == 64 && !SPLIT ? 1 : 2)
gemm_int4_tile_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const GemmI4Params p) {
    constexpr int kScaleBytes = ScaleTile<GS, kBlockK>::bytes(kTileN), kTileStage = tile_stage<TM>(), kTileStages = tile_stages<TM>();
    constexpr int kTileM = TM, WM = 2, MR = 2, NT = TM / 16;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *scales = smem + kTileStages * kTileStage;
    __shared__ uint64_t full[kTileStages];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gq = lane >> 2, cq = lane & 3, wn = warp % (8 / WM), wm = warp / (8 / WM);
    if (tid == 0) {
        for (int k = 0; k < kTileStages; ++k) mbar_init(&full[k], kTileThreads + 1);   // scale copies, the TMA's bytes
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
    const int first = SPLIT ? 2 * static_cast<int>(static_cast<int64_t>(rank) * p.units / p.segments) : 0;
    const int last = SPLIT ? min(p.blocks, 2 * static_cast<int>(static_cast<int64_t>(rank + 1) * p.units / p.segments)) : p.blocks;
    GroupCursor<GS> g(p, first), fg = g;                   // of the block at work, of the next to be copied
    auto fill = [&](int blk) {
        const int slot = (blk - first) % kTileStages;
        uint8_t *dst = smem + slot * kTileStage;
        if (tid == 0) {
            mbar_arrive_expect_tx(&full[slot], kTileW + kTileM * kBlockK * 2);
            tma_load_2d(dst, &tmW, &full[slot], blk * (kBlockK / 2), static_cast<int32_t>(n0));
            tma_load_2d(dst + kTileW, &tmX, &full[slot], blk * kBlockK, static_cast<int32_t>(m0));
            tma_load_2d(dst + kTileW + x_box(kTileM), &tmX, &full[slot], blk * kBlockK + 64, static_cast<int32_t>(m0));
        }
        stage_scales<GS, kBlockK, kTileN, kTileN, kTileThreads, ZEROS>(p, smem_u32(scales + slot * kScaleBytes), &full[slot], 0, n0 * p.groups + fg.group, tid);
        fg.next(p);
    };
    for (int blk = first; blk < last && blk < first + kTileStages - 1; ++blk) fill(blk);
    float acc[MR][NT][4], tot[MR][NT][4];
    auto clear = [&](float (&v)[MR][NT][4]) {
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[m][t][e] = 0.0f;
    };
    clear(acc);
    int seg = 0;                                           // SPLIT false: the segment at work, and its end
    int seg_end = min(p.blocks, 2 * (p.units / p.segments));
    bool ok = true;
    for (int blk = first; blk < last; ++blk) {
        const int i = blk - first, slot = i % kTileStages;
        ok = mbar_wait(&full[slot], (i / kTileStages) & 1, nullptr);
        if (__syncthreads_or(!ok)) {                       // (and: block i - 1 is done with)
            if (tid == 0) {                                // ran out: report; the copies in flight get another limit
                atomicOr(p.status, kDevTimeout);
                for (int k = 0; k < kTileStages - 1 && blk + k < last; ++k)
                    mbar_wait(&full[(i + k) % kTileStages], ((i + k) / kTileStages) & 1, nullptr);
            }
            break;
        }
        if (blk + kTileStages - 1 < last) fill(blk + kTileStages - 1);
        const uint32_t st = smem_u32(smem + slot * kTileStage);
        product<GS, kBlockK, MR, NT, kTileN, ZEROS>(st, st + kTileW, scales + slot * kScaleBytes, 16 * MR * wn, x_box(kTileM), 8 * NT * wm, 7,
                                                          p.groups, g, p.K - blk * kBlockK, gq, cq, acc);
        g.next(p);
        if (!SPLIT && blk + 1 == seg_end) {
#pragma unroll
            for (int m = 0; m < MR; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) tot[m][t][e] = seg == 0 ? acc[m][t][e] : tot[m][t][e] + acc[m][t][e];
            clear(acc);
            ++seg;
            seg_end = min(p.blocks, 2 * static_cast<int>(static_cast<int64_t>(seg + 1) * p.units / p.segments));
        }
    }
    // the tile's sums through shared memory, [row of X][weight row] with the rows four apart in banks
    constexpr int kLd = kTileN + 4;
    static_assert(kTileM * kLd * 4 <= kTileStages * kTileStage, "the tile's sums fit the stages");
    float *red = reinterpret_cast<float *>(smem);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[(8 * NT * wm + 8 * t + x_row<GS>(2 * cq + (e & 1))) * kLd + 16 * MR * wn + 16 * m + gq + 8 * (e >> 1)] =
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

template <int GS, int NT, bool ZEROS>
bi_status launch_rows(const CUtensorMap &tmW, const CUtensorMap &tmX, const GemmI4Params &p, int sms, cudaStream_t s) {
    static unsigned long long configured = 0;
    constexpr int most = 1024 + kMaxSegments * rows_segment<GS, NT>(8 * NT);
    static_assert(most <= 232448 - 1024, "one CTA's shared memory");
    if (ensure_smem_attr(reinterpret_cast<const void *>(gemm_int4_rows_kernel<GS, NT, ZEROS>), most, &configured) != BI_OK)
        return BI_ERR_CUDA;
    // as many CTAs as the shared memory of the SMs takes at once
    const int64_t tiles = (p.N + rows_n<NT>() - 1) / rows_n<NT>();
    const int smem = 1024 + p.segments * rows_segment<GS, NT>(p.x_rows), fit = 232448 / (smem + 2048);
    const int64_t most_ctas = static_cast<int64_t>(sms) * (fit > 4 ? 4 : fit);
    return launch_pdl(gemm_int4_rows_kernel<GS, NT, ZEROS>, dim3(static_cast<unsigned>(tiles < most_ctas ? tiles : most_ctas)),
                      dim3(32 * NT * p.segments), smem, s, tmW, tmX, p);
}

template <int GS, int TM, bool SPLIT, bool ZEROS>
bi_status launch_tile_kernel(const CUtensorMap &tmW, const CUtensorMap &tmX, const GemmI4Params &p, int64_t tiles,
                       cudaStream_t s) {
    static unsigned long long configured = 0;
    if (ensure_smem_attr(reinterpret_cast<const void *>(gemm_int4_tile_kernel<GS, TM, SPLIT, ZEROS>), tile_smem<GS, TM>(), &configured) != BI_OK)
        return BI_ERR_CUDA;
    const int64_t grid = tiles * (SPLIT ? p.segments : 1);
    if (grid > 0x7FFFFFFF) return BI_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = tile_smem<GS, TM>();
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
    if (cudaLaunchKernelEx(&cfg, gemm_int4_tile_kernel<GS, TM, SPLIT, ZEROS>, tmW, tmX, p) == cudaSuccess) return BI_OK;
    cudaGetLastError();
    return BI_ERR_CUDA;
}

// Rows of X a tile (32 or 64), and whether the CTAs of a cluster take a segment each, by the time it should take (tenths
// of a microsecond). The SMs work in rounds: one CTA an SM with tiles of 64 rows and all segments, else two. Per block of
// 128 k a round takes 1.2 us with tiles of 64 rows, 1.3 with two CTAs of 32 (0.9 with one); of one segment 1.4 with tiles
// of 32 and 2.1 with 64, and 4 or 5.5 us for filling the stages and joining the sums. Measured, tiles of 32 / 64 rows /
// segments with 32 / 64 (g = 128): 17 x 6144 x 4096 28.5 / 39.3 / 18.5 / 23.1 us; 64 rows 28.6 / 39.4 / 31.4 / 28.4; 96
// rows 28.7 / 39.5 / 44.0 / 43.4; 200 rows 68.5 / 77.5 / 91.4 / 77.8; 200 x 24576 x 4096 193 / 231 / 347 / 286;
// 130 x 4096 x 12288 126 / 110 / 94 / 89, 200 rows 126 / 110 / 125 / 112.
struct TilePlan {
    int rows;
    bool split;
};
TilePlan tile_plan(const GemmI4Params &p, int sms) {
    const int64_t tiles_n = (p.N + kTileN - 1) / kTileN, t32 = tiles_n * ((p.M + 31) / 32), t64 = tiles_n * ((p.M + 63) / 64);
    const int64_t two = 2 * static_cast<int64_t>(sms), left = t32 % two, seg = (p.blocks + p.segments - 1) / p.segments;
    const int64_t all32 = (t32 / two * 13 + (left > sms ? 14 : left > 0 ? 9 : 0)) * p.blocks;
    const int64_t all64 = (t64 + sms - 1) / sms * 12 * p.blocks;
    TilePlan best{all32 <= all64 ? 32 : 64, false};
    if (p.segments > 1) {
        const int64_t seg32 = (t32 * p.segments + two - 1) / two * (40 + 14 * seg), seg64 = (t64 * p.segments + two - 1) / two * (55 + 21 * seg);
        const int64_t least = seg32 < seg64 ? seg32 : seg64;
        if (least < (all32 <= all64 ? all32 : all64)) best = TilePlan{seg32 < seg64 ? 32 : 64, true};
    }
    return best;
}

template <int GS, int TM, bool ZEROS>
bi_status launch_tiles(const CUtensorMap &tmW, const CUtensorMap &tmX, const GemmI4Params &p, bool split, cudaStream_t s) {
    const int64_t tiles = (p.N + kTileN - 1) / kTileN * ((p.M + TM - 1) / TM);
    return split ? launch_tile_kernel<GS, TM, true, ZEROS>(tmW, tmX, p, tiles, s) : launch_tile_kernel<GS, TM, false, ZEROS>(tmW, tmX, p, tiles, s);
}

template <int GS, bool ZEROS>
bi_status launch_group(const void *X, int64_t ldx, const uint8_t *W, GemmI4Params &p, int sms, cudaStream_t s) {
    // Rows kernel / tile kernel, g = 128: 9 x 6144 x 4096 9.9 / 16.9 us, 16 rows 10.0 / 17.5, 16 x 24576 x 4096 24.5 / 45.8.
    const bool rows = p.M <= 16;
    const TilePlan plan = tile_plan(p, sms);
    const int tm = plan.rows, kb = p.M <= 8 ? rows_kb<1>() : rows_kb<2>();
    p.x_rows = p.M <= 2 ? static_cast<int>(p.M) : p.M <= 4 ? 4 : p.M <= 8 ? 8 : 16;
    CUtensorMap tmW{}, tmX{};
    if (make_tmap_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, W, p.K / 2, p.N, p.K / 2, (rows ? kb : kBlockK) / 2, rows ? (p.M <= 8 ? rows_n<1>() : rows_n<2>()) : kTileN,
                     rows && kb == 256 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) != BI_OK ||
        make_tmap_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, X, p.K, p.M, ldx * 2, 64, rows ? p.x_rows : tm,
                     CU_TENSOR_MAP_SWIZZLE_128B) != BI_OK)
        return BI_ERR_CUDA;
    if (rows) return p.M <= 8 ? launch_rows<GS, 1, ZEROS>(tmW, tmX, p, sms, s) : launch_rows<GS, 2, ZEROS>(tmW, tmX, p, sms, s);
    if (tm == 32) return launch_tiles<GS, 32, ZEROS>(tmW, tmX, p, plan.split, s);
    return launch_tiles<GS, 64, ZEROS>(tmW, tmX, p, plan.split, s);
}

}  // namespace

bi_status launch_gemm_int4(const void *X, int64_t ldx, const uint8_t *W, const void *scales, const uint8_t *zeros, void *Y,
                           int64_t ldy, int64_t M, int64_t N, int64_t K, int64_t group, cudaStream_t s) {
    int dev = 0;
    const DeviceInfo *info = nullptr;
    const bi_status st = current_device(&dev, &info);
    if (st != BI_OK) return st;
    GemmI4Params p{};
    p.S = static_cast<const uint32_t *>(scales);
    p.Z = reinterpret_cast<const uint32_t *>(zeros);
    p.Y = static_cast<uint16_t *>(Y);
    p.ldy = ldy;
    p.M = M, p.N = N, p.K = static_cast<int32_t>(K);
    p.groups = static_cast<int32_t>(K / group);
    p.s_last = N * p.groups / 2 - 1, p.z_last = N * p.groups / 4 - 1;   // (N % 8 == 0)
    p.group = static_cast<int32_t>(group);
    p.blocks = static_cast<int32_t>((K + kBlockK - 1) / kBlockK);
    p.units = static_cast<int32_t>((K + kUnitK - 1) / kUnitK);
    p.segments = p.units < 4 ? 1 : p.units / 2 > kMaxSegments ? kMaxSegments : p.units / 2;
    p.status = device_status_word();
    const int sms = info->sm_count;
    if (group == 32) return zeros ? launch_group<32, true>(X, ldx, W, p, sms, s) : launch_group<32, false>(X, ldx, W, p, sms, s);
    if (group == 64) return zeros ? launch_group<64, true>(X, ldx, W, p, sms, s) : launch_group<64, false>(X, ldx, W, p, sms, s);
    return zeros ? launch_group<128, true>(X, ldx, W, p, sms, s) : launch_group<128, false>(X, ldx, W, p, sms, s);
}

}  // namespace bi
