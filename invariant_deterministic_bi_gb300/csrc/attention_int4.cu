// attention_int4.cu -- attention over the paged 4-bit K/V cache for few query
// rows a sequence: decode, and extend by a few tokens. (Extend by many tokens
// expands the codes into the tiles of attention.cu's extend kernel.)
//
// The results are bi_attention_decode's / _extend's over a bf16 cache that
// holds the same values, bit for bit: the values are bf16 numbers exactly
// (kv_int4.cuh), and the 128-token chunks, the tensor-core chains (ascending
// dimension steps for q.k, ascending token steps with p's high part before its
// low part for p.v), the order of each sum and the chunk merge are the same.
// What differs is the split of the work.
//
// Step 1, attn_split_int4_kernel: one warp computes one item, a chunk of one KV
// head for eight query rows (8 / G new tokens of the G query heads that share
// the KV head; decode has one token), without a barrier. A chunk is 18 KB here,
// not 64, and its codes are expanded in registers. The products are taken
// transposed, tokens (or dimensions) as the 16 rows of m16n8k16 and the query
// rows as its 8 columns: half the tensor work of 16 query rows of which at most
// eight exist.
//   q.k: A = 16 tokens x 16 dimensions of K, B = q^T.
//   p.v: A = 16 dimensions x 16 tokens of V, B = p: the scores' fragment
//        transposed by movmatrix.
// Step 2, attn_merge_int4_kernel, one CTA per (query token, query head): the
//   chunk results are merged in chunk order and o / l is rounded to bf16.
//
// What bounds it: not HBM (3.6 times fewer bytes than bf16 leave 45 us at
// 64 x 4096 tokens, 8 KV heads) but its instructions, 3184 an item: expanding 128
// words of eight codes takes 1408 of them, their scales 256, mma.sync 192, softmax,
// transposes, stores and the walk the rest, on pipes that overlap only partly (a
// word and a product: 21.6-24.7 cycles per warp and scheduler, 17 and 8 apart). Measured (GB300): 64 x 4096, 32 heads over 8
// 91 us, 3.3 TB/s (bf16 cache: 187 us); 1 x 4096 10.1 us (9.9); 2 x 131072, 64 over
// 8 heads 102 us; 16 sequences x 5 new tokens over 100..4000 58 us. Per warp two 9 KB
// buffers and 12 warps; 16 warps with three 4.5 KB buffers each took 102 us (the
// pipes, not the latencies, are what a warp waits for); reading the codes from
// global memory into registers, 133 us.
#include "attn_common.cuh"
#include "bi_internal.h"
#include "bi_ptx.cuh"
#include "kv_int4.cuh"

namespace bi {
namespace {

constexpr int kMaxWarps = 12;                  // warps of a CTA, each with a chunk in hand and one on the way
constexpr int kCodeBytes = kChunk * kI4Row, kScaleBytes = kChunk * kI4Scales * 2;
constexpr int kHalfBytes = kCodeBytes + kScaleBytes;   // a chunk's K (or V): 9 KB
constexpr int kWarpBytes = 2 * kHalfBytes;
constexpr uint32_t kNoRow = 0xFFFFFFFFu;
constexpr int kRecord = kD + 2;                // floats of a chunk result: m, l, o
constexpr int kMergeThreads = 128;             // and a warp that loads
constexpr int kMergeTile = 32, kMergeRing = 8; // chunk results of a tile, tiles on the way at most
constexpr int kMergeStage = (kMergeTile * kRecord * 4 + 16 + 15) / 16 * 16;
// Extend takes this split or the tiled kernel by their estimated times (the sizes decide, not the data; the SMs are
// these because the workspace's size is asked for without a device): a CTA of the tiled kernel spends about 13 K cycles
// on a chunk for up to 128 query rows, one CTA an SM and no split of the chunks; an SM here about 1.7 K for each eight
// rows. Measured, 32 heads over 8, 4000 cached tokens each, tiled / split: 16 sequences x 5 tokens 263 / 75 us, x 16
// 227 / 194; 1 x 5 257 / 13, 1 x 16 215 / 22, 1 x 64 203 / 52, 4 x 8 (64 heads) 218 / 53; 64 x 16 over 2000 455 / 405;
// 64 x 1 over 4096 1057 / 103. The estimate knows neither the number of sequences nor their tokens, only the sum and
// max_q, and both kernels work for max_q tokens of each sequence, so uneven batches are not what it is made for:
// 63 x 1 and one x 64 over 4096 1059 / 553, one x 200 1073 / 1065, one x 512 1288 (tiled); 255 x 1 and one x 64 over
// 1000 951 (tiled); 256 x 1 over 1000 with max_q 256 1005 / 2649, where it takes the split, with max_q 1 940 / 106.
// The chunk results take at most kFewBytes.
constexpr int64_t kSms = 152, kTiledCost = 130, kSplitCost = 17;
constexpr int64_t kFewBytes = 512ll << 20;

struct SplitParams {
    KvInt4 c;
    const uint16_t *Q;       // [rows][Hq][D]
    const int32_t *cu_q;     // [B+1], extend only
    const int32_t *table;    // [B][max_blocks]
    const int32_t *lens;     // [B]
    float *ws;               // [rows][Hq][chunks][kRecord]
    uint16_t *O;             // [rows][Hq][D]
    int64_t batch;
    int32_t total_q, max_q, tiles;   // extend: query rows, a sequence's most, its tiles of 8 / G tokens
    int32_t max_blocks, Hq, chunks, max_len;
    bool scan;               // look for the longest sequence first
    float scale;
    unsigned *status;
};

// The query tokens of a sequence: q0 its first row of Q, len0 what its first token sees. False: none.
template <bool EXT>
__device__ __forceinline__ bool sequence(const SplitParams &p, int64_t b, int64_t &q0, int &qlen, int &len0, bool report) {
    const int L = p.lens[b];
    bool ok = L <= p.max_len && L <= static_cast<int64_t>(p.max_blocks) * p.c.bs;
    if (EXT) {
        q0 = p.cu_q[b];
        const int64_t n = p.cu_q[b + 1] - q0;
        ok = ok && q0 >= 0 && n >= 0 && q0 + n <= p.total_q && n <= p.max_q && L >= n;
        qlen = ok ? static_cast<int>(n) : 0;
        len0 = L - qlen + 1;
    } else {
        q0 = b;
        ok = ok && L >= 1;
        qlen = ok ? 1 : 0;
        len0 = L;
    }
    if (!ok && report) atomicOr(p.status, kDevBadOffsets);
    return qlen > 0;
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Where a warp is in the items: (sequence, chunk, tile, KV head), the last fastest, so that
// the heads of one cache block, and the tiles that read the same chunk, are at work together.
struct Cursor {
    int64_t b;
    int c, tile, g;
};

// What a warp has to know of an item.
struct Item {
    int64_t row0;            // first query row (token) in Q and the workspace
    int g, c;
    int n;                   // tokens of the chunk that some row sees; 0: nothing to do
    int ntok, see0;          // query tokens; of the chunk's tokens, how many the first one sees
    bool whole;              // every row sees all 128, in blocks of the cache
    uint32_t valid[4];       // tokens with a row in the cache (set where not whole)
    // block copies: lane i's run of the chunk in one block; row copies: rows of tokens lane + 32 k
    uint32_t row[4];         // (block copies: row[0], token row[1], tokens row[2])
};

template <int G, bool EXT, bool BLOCKS>
__device__ __forceinline__ Item load_item(const SplitParams &p, const Cursor &u, int lane) {
    constexpr int kTQ = EXT ? 8 / G : 1;
    Item x;
    x.g = u.g;
    x.c = u.c;
    x.n = 0;
    int qlen, len0;
    if (!sequence<EXT>(p, u.b, x.row0, qlen, len0, lane == 0 && u.c == 0 && u.g == 0 && u.tile == 0)) return x;
    const int i0 = u.tile * kTQ, j0 = u.c * kChunk;
    x.ntok = min(kTQ, qlen - i0);
    if (x.ntok <= 0) return x;
    x.row0 += i0;
    x.see0 = len0 + i0 - j0;
    x.n = max(0, min(kChunk, x.see0 + x.ntok - 1));
    if (x.n == 0) return x;
    const int32_t *table = p.table + u.b * p.max_blocks;
    bool bad = false;
    if (BLOCKS) {
        const int first = j0 / p.c.bs, blk_i = first + lane;
        const int64_t start = static_cast<int64_t>(blk_i) * p.c.bs - j0;   // the block's first token in the chunk
        const int t0 = static_cast<int>(min(max(start, static_cast<int64_t>(0)), static_cast<int64_t>(x.n)));
        const int t1 = static_cast<int>(min(start + p.c.bs, static_cast<int64_t>(x.n)));
        x.row[0] = 0, x.row[1] = 0, x.row[2] = 0;
        if (t0 < t1) {
            const int64_t blk = table[blk_i];
            bad = blk < 0 || blk >= p.c.num_blocks;
            if (!bad) {
                x.row[0] = static_cast<uint32_t>((blk * p.c.Hkv + x.g) * p.c.bs + (t0 - start));
                x.row[1] = t0;
                x.row[2] = t1 - t0;
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x.row[k] = kNoRow;
            const int t = lane + 32 * k;
            if (t < x.n) {
                const int64_t blk = table[(j0 + t) / p.c.bs];
                if (blk >= 0 && blk < p.c.num_blocks)
                    x.row[k] = static_cast<uint32_t>((blk * p.c.Hkv + x.g) * p.c.bs + (j0 + t) % p.c.bs);
                else
                    bad = true;
            }
        }
    }
    if (bad) atomicOr(p.status, kDevBadOffsets);
    const uint32_t bads = __ballot_sync(0xffffffffu, bad);
    x.whole = x.see0 >= kChunk && bads == 0;
    if (!x.whole) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int t = lane + 32 * k;
            const bool in = BLOCKS ? t < x.n && ((bads >> ((j0 + t) / p.c.bs - j0 / p.c.bs)) & 1) == 0 : x.row[k] != kNoRow;
            x.valid[k] = __ballot_sync(0xffffffffu, in);
        }
    }
    return x;
}

// Byte offset of segment i of token t's codes in a staged tile.
__device__ __forceinline__ int tile_seg(int t, int i) { return t * kI4Row + 16 * i4_place(i, t); }

// Starts the copies of a chunk's K (or V) codes and scales. Where blocks are multiples of eight tokens, one bulk
// copy a block takes the codes as they lie (a token's place in the chunk and in the block agree modulo eight), one its
// scales, counted on the barrier. Else 16-byte copies, one group; rows without a token become zeros.
template <bool BLOCKS>
__device__ __forceinline__ void stage(const uint8_t *codes, const uint16_t *scales, const Item &x, int bs, uint8_t *dst,
                                      uint64_t *bar, int lane) {
    if (BLOCKS) {
        // an odd number of tokens takes the block's next scale row along (copies are multiples of 16 bytes)
        const uint32_t cb = x.row[2] * kI4Row, sb = ((x.row[2] + 1) & ~1u) * kI4Scales * 2;
        const uint32_t bytes = __reduce_add_sync(0xffffffffu, cb + sb);
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        __syncwarp();
        if (cb) {
            bulk_load(dst + x.row[1] * kI4Row, codes + static_cast<int64_t>(x.row[0]) * kI4Row, cb, bar);
            bulk_load(dst + kCodeBytes + x.row[1] * kI4Scales * 2, scales + static_cast<int64_t>(x.row[0]) * kI4Scales, sb, bar);
        }
    } else {
        const uint32_t d = smem_u32(dst);
#pragma unroll
        for (int s = 0; s < kChunk / 8; ++s) {             // eight rows a step, four lanes a row
            const int t = 8 * s + (lane >> 2), i = lane & 3;
            const uint32_t row = __shfl_sync(0xffffffffu, x.row[s >> 2], t & 31);
            const bool in = row != kNoRow;
            cp_async_16(d + tile_seg(t, i),
                        in ? codes + static_cast<int64_t>(row) * kI4Row + 16 * i4_place(i, static_cast<int>(row % bs)) : codes,
                        in ? 16u : 0u);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bool in = x.row[k] != kNoRow;
            cp_async_8(d + kCodeBytes + (lane + 32 * k) * 8, in ? scales + static_cast<int64_t>(x.row[k]) * kI4Scales : scales,
                       in ? 8u : 0u);
        }
        cp_async_commit();
    }
}

// Waits for a staged half; false: the wait ran out (block copies).
template <bool BLOCKS>
__device__ __forceinline__ bool staged(uint64_t *bar, uint32_t parity) {
    bool ok = true;
    if (BLOCKS)
        ok = mbar_wait(bar, parity, nullptr);
    else
        cp_async_wait<1>();
    __syncwarp();                                          // every lane sees every lane's copies
    return __all_sync(0xffffffffu, ok);
}

// The q rows as B fragments: column j is query token j / G, head g G + j % G.
template <int G, bool EXT>
__device__ __forceinline__ void load_q(const SplitParams &p, const Item &x, int gq, int cq, uint32_t (&qb)[kD / 16][2]) {
    const bool in = gq / G < (EXT ? x.ntok : 1);
    const uint16_t *q = p.Q + ((x.row0 + (in ? gq / G : 0)) * p.Hq + x.g * G + gq % G) * kD + 2 * cq;
#pragma unroll
    for (int ks = 0; ks < kD / 16; ++ks) {
        qb[ks][0] = in ? *reinterpret_cast<const uint32_t *>(q + 16 * ks) : 0u;
        qb[ks][1] = in ? *reinterpret_cast<const uint32_t *>(q + 16 * ks + 8) : 0u;
    }
}

// Each warp walks the items blockIdx.x + gridDim.x * (warp + warps * i) (which
// warp computes an item changes no arithmetic). Its K and V buffers are filled
// by asynchronous copies: the next item's K while this item's softmax and p.v
// run, its V while the next item's scores do. No warp waits for another.
template <int G, bool EXT, bool BLOCKS>
__global__ void __launch_bounds__(32 * kMaxWarps, 1)
attn_split_int4_kernel(const SplitParams p) {
    constexpr int kTQ = EXT ? 8 / G : 1;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t bars[2 * kMaxWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, cq = lane & 3;               // fragment row group, column pair
    uint64_t *barK = bars + 2 * warp, *barV = barK + 1;
    if (lane == 0) {
        mbar_init(barK, 1);
        mbar_init(barV, 1);
        fence_mbar_init();
    }
    __syncwarp();
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    uint8_t *Ks = smem + warp * kWarpBytes, *Vs = Ks + kHalfBytes;
    const int64_t ws_head = static_cast<int64_t>(p.chunks) * kRecord;   // next query head's records
    // the walk over (sequence, chunk, tile, head), as far as the longest sequence's last chunk where that is looked
    // for; `step` items on, digit by digit
    int chunks = p.chunks;
    if (p.scan) {
        int longest = 1;
        for (int64_t b = lane; b < p.batch; b += 32) {
            const int L = p.lens[b];
            if (L <= p.max_len) longest = max(longest, L);
        }
        chunks = (__reduce_max_sync(0xffffffffu, longest) + kChunk - 1) / kChunk;
    }
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    auto split = [&](int64_t i) {
        Cursor u;
        u.g = static_cast<int>(i % p.c.Hkv);
        i /= p.c.Hkv;
        u.tile = EXT ? static_cast<int>(i % p.tiles) : 0;
        if (EXT) i /= p.tiles;
        u.c = static_cast<int>(i % chunks);
        u.b = i / chunks;
        return u;
    };
    Cursor u = split(blockIdx.x + static_cast<int64_t>(gridDim.x) * warp);
    const Cursor step = split(stride);
    auto next = [&]() {                                    // the next item with work
        Item x;
        x.n = 0;
        while (x.n == 0 && u.b < p.batch) {
            x = load_item<G, EXT, BLOCKS>(p, u, lane);
            int carry = (u.g += step.g) >= p.c.Hkv;
            if (carry) u.g -= p.c.Hkv;
            if (EXT) {
                carry = (u.tile += step.tile + carry) >= p.tiles;
                if (carry) u.tile -= p.tiles;
            }
            carry = (u.c += step.c + carry) >= chunks;
            if (carry) u.c -= chunks;
            u.b += step.b + carry;
        }
        return x;
    };
    Item cur = next();
    if (cur.n == 0) return;
    stage<BLOCKS>(p.c.kc, p.c.ks, cur, p.c.bs, Ks, barK, lane);
    stage<BLOCKS>(p.c.vc, p.c.vs, cur, p.c.bs, Vs, barV, lane);
    uint32_t qb[kD / 16][2];
    load_q<G, EXT>(p, cur, gq, cq, qb);
    uint32_t parity = 0;
    // addresses of this lane's operand rows: ldmatrix takes token lane % 8, segment lane / 8
    const uint32_t k_addr = smem_u32(Ks) + tile_seg(lane & 7, lane >> 3);
    const uint32_t v_addr = smem_u32(Vs) + tile_seg(lane & 7, lane >> 3);
    while (true) {
        const Item nxt = next();
        if (!staged<BLOCKS>(barK, parity)) {
            if (lane == 0) atomicOr(p.status, kDevTimeout);
            staged<BLOCKS>(barK, parity);                  // the copies in flight get another limit
            staged<BLOCKS>(barV, parity);
            return;
        }
        // scores: s[mt][e], token 16 mt + gq + 8 (e / 2), query row 2 cq + e % 2
        float s[kChunk / 16][4];
#pragma unroll
        for (int mt = 0; mt < kChunk / 16; ++mt) {
            uint32_t kw[2][4];
            uint2 sc[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ldmatrix_x4(kw[h][0], kw[h][1], kw[h][2], kw[h][3], k_addr + (16 * mt + 8 * h) * kI4Row);
                sc[h] = *reinterpret_cast<const uint2 *>(Ks + kCodeBytes + 8 * (16 * mt + 8 * h + gq));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][e] = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {                  // 32 dimensions: one scale, two 16-dimension steps
                uint32_t a[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t sw = i < 2 ? sc[h].x : sc[h].y;
                    const uint32_t s2 = i & 1 ? dup16<1>(sw) : dup16<0>(sw);
                    i4_expand(kw[h][i], s2, mul_bf16x2(s2, kBf16x2_m136), a[h]);
                }
                mma_16816(s[mt], a[0][0], a[1][0], a[0][1], a[1][1], qb[2 * i][0], qb[2 * i][1]);
                mma_16816(s[mt], a[0][2], a[1][2], a[0][3], a[1][3], qb[2 * i + 1][0], qb[2 * i + 1][1]);
            }
        }
        __syncwarp();                                      // every lane has read K
        if (nxt.n) {
            stage<BLOCKS>(p.c.kc, p.c.ks, nxt, p.c.bs, Ks, barK, lane);
            load_q<G, EXT>(p, nxt, gq, cq, qb);
        } else if (!BLOCKS) {
            cp_async_commit();
        }
#pragma unroll
        for (int mt = 0; mt < kChunk / 16; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][e] = __fmul_rn(s[mt][e], p.scale);
        float m[2] = {-INFINITY, -INFINITY};
        if (!cur.whole) {
#pragma unroll
            for (int mt = 0; mt < kChunk / 16; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 16 * mt + gq + 8 * (e >> 1);
                    const bool in = ((cur.valid[mt >> 1] >> (t & 31)) & 1) && (!EXT || t < cur.see0 + (2 * cq + (e & 1)) / G);
                    if (!in) s[mt][e] = -INFINITY;
                }
            int first = 0x7FFFFFFF;                        // the chunk's first token with a row in the cache
#pragma unroll
            for (int k = 3; k >= 0; --k)
                if (cur.valid[k]) first = 32 * k + __ffs(cur.valid[k]) - 1;
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (first >= cur.see0 + (EXT ? (2 * cq + e) / G : 0)) m[e] = kNoScore;
        }
        // per row: the maximum, the exponentials, and their sum in the bf16 kernels' order: tokens
        // L, L + 32, L + 64, L + 96 in turn (mt = L / 16 % 2 + 0, 2, 4, 6), then a butterfly over
        // L xor 16 (mt), 8 (the fragment's half), 4, 2, 1 (lanes)
        float l[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
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
        // this lane's two rows' records (column j: token j / G, head g G + j % G)
        float *ws[2];
        bool out[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int j = 2 * cq + e;
            out[e] = j / G < (EXT ? cur.ntok : 1) && BI_IN_BOUNDS(cur.row0 + j / G < (EXT ? p.total_q : p.batch) && cur.c < p.chunks, p.status);
            ws[e] = p.ws + ((cur.row0 + j / G) * p.Hq + cur.g * G + j % G) * ws_head + static_cast<int64_t>(cur.c) * kRecord;
            if (gq == 0 && out[e]) *reinterpret_cast<float2 *>(ws[e]) = make_float2(m[e], l[e]);
        }
        // p as B fragments (high and low bf16 parts): the score fragment is [token][row], B wants
        // lane (row gq, tokens 2 cq, 2 cq + 1)
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
        if (!staged<BLOCKS>(barV, parity)) {
            if (lane == 0) atomicOr(p.status, kDevTimeout);
            staged<BLOCKS>(barV, parity);
            if (nxt.n) staged<BLOCKS>(barK, parity ^ 1);
            return;
        }
        // a token that some row does not see must not bring it a NaN (0 * v): the groups of tokens see0 .. see0 + 7 that
        // are not finite (bit 4 (t - see0) + i) become zeros here, and NaN in the rows that see them below
        uint32_t nans = 0;
        if (kTQ > 1 && cur.ntok > 1 && !cur.whole) {
            const int t = cur.see0 + (lane >> 2);
            uint16_t *s1 = reinterpret_cast<uint16_t *>(Vs + kCodeBytes) + t * kI4Scales + (lane & 3);
            const uint32_t valid = t < 64 ? (t < 32 ? cur.valid[0] : cur.valid[1]) : (t < 96 ? cur.valid[2] : cur.valid[3]);
            const bool nan = t >= 0 && t < cur.n && ((valid >> (t & 31)) & 1) && !i4_finite(*s1);
            nans = __ballot_sync(0xffffffffu, nan);
            if (nan) *s1 = 0;
            if (nans) __syncwarp();
        }
        if (!cur.whole && BLOCKS) {                        // nor one without a row
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (!((cur.valid[k] >> lane) & 1))
                    *reinterpret_cast<uint2 *>(Vs + kCodeBytes + 8 * (lane + 32 * k)) = make_uint2(0u, 0u);
            fence_proxy_async_smem();                      // before later bulk copies into these rows
            __syncwarp();
        }
        // values: o[j][e], dimension 16 j + gq + 8 (e / 2), query row 2 cq + e % 2
        float o[kD / 16][4];
#pragma unroll
        for (int j = 0; j < kD / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < kChunk / 16; ++ks) {
            uint32_t vw[2][4], sc[2][4];                   // token pairs 2 cq, + 1 and + 8, + 9 of the step
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                ldmatrix_x4_trans(vw[k][0], vw[k][1], vw[k][2], vw[k][3], v_addr + (16 * ks + 8 * k) * kI4Row);
                const uint4 x = *reinterpret_cast<const uint4 *>(Vs + kCodeBytes + 8 * (16 * ks + 8 * k + 2 * cq));
                sc[k][0] = zip16<0>(x.x, x.z), sc[k][1] = zip16<1>(x.x, x.z);
                sc[k][2] = zip16<0>(x.y, x.w), sc[k][3] = zip16<1>(x.y, x.w);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {                  // 32 dimensions: tiles 2 i and 2 i + 1
                uint32_t a[2][4];                          // [token pair][nibble]
#pragma unroll
                for (int k = 0; k < 2; ++k) i4_expand(vw[k][i], sc[k][i], mul_bf16x2(sc[k][i], kBf16x2_m136), a[k]);
                mma_16816(o[2 * i], a[0][0], a[0][1], a[1][0], a[1][1], ph[ks][0], ph[ks][1]);
                mma_16816(o[2 * i + 1], a[0][2], a[0][3], a[1][2], a[1][3], ph[ks][0], ph[ks][1]);
                mma_16816(o[2 * i], a[0][0], a[0][1], a[1][0], a[1][1], pl[ks][0], pl[ks][1]);
                mma_16816(o[2 * i + 1], a[0][2], a[0][3], a[1][2], a[1][3], pl[ks][0], pl[ks][1]);
            }
        }
        if (kTQ > 1 && nans) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int j = 0; j < kD / 16; ++j)
                    if (nans & (0x11111111u << (j / 2)) & ((1u << (4 * ((2 * cq + e) / G))) - 1u)) o[j][e] = o[j][2 + e] = __int_as_float(0x7FFFFFFF);
        }
        __syncwarp();                                      // every lane has read V
        if (nxt.n)
            stage<BLOCKS>(p.c.vc, p.c.vs, nxt, p.c.bs, Vs, barV, lane);
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (out[e]) {
                float *w = ws[e] + 2 + gq;
#pragma unroll
                for (int j = 0; j < kD / 16; ++j) {
                    w[16 * j] = o[j][e];
                    w[16 * j + 8] = o[j][2 + e];
                }
            }
        if (nxt.n == 0) return;                            // nothing is in flight
        cur = nxt;
        parity ^= 1;
    }
}

// Merges the chunk results of one (query token, query head) in chunk order, thread d its dimension d (warps 0 .. 3).
// The records of a head lie one after the other: warp 4 keeps up to `ring` tiles of 32 on the way to shared memory.
// The running maximum before a chunk is a prefix maximum (exact in any order), so it also prepares the next tile's
// factors in parallel, while the others merge: one product and one fused multiply-add a chunk in order. With a long
// sequence's loads so far ahead, its merge is bound by those operations and not by a tile's load latency.
template <bool EXT>
__global__ void __launch_bounds__(kMergeThreads + 32)
attn_merge_int4_kernel(const SplitParams p, int ring) {
    constexpr int kTile = kMergeTile;
    extern __shared__ __align__(16) uint8_t tiles[];       // [ring][kMergeStage]
    __shared__ float fa[2][kTile], fb[2][kTile], fl[2][kTile];   // alpha, beta, l of a tile's chunks
    __shared__ uint64_t full[kMergeRing];
    __shared__ int failed[2];                              // tile t's wait ran out: [t % 2], read while t + 1's may be set
    const int d = threadIdx.x, lane = d & 31;
    const bool loader = d >= kMergeThreads;
    if (d == kMergeThreads) {
        for (int k = 0; k < ring; ++k) mbar_init(&full[k], 1);
        fence_mbar_init();
        failed[0] = failed[1] = 0;
    }
    __syncthreads();
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    const int h = blockIdx.x % p.Hq;
    const int64_t y = blockIdx.x / p.Hq, b = EXT ? y / p.max_q : y;
    const int i = EXT ? static_cast<int>(y % p.max_q) : 0;
    int64_t row;
    int qlen, len0;
    if (!sequence<EXT>(p, b, row, qlen, len0, false) || i >= qlen) return;
    row += i;
    const int nc = (len0 + i + kChunk - 1) / kChunk, nt = (nc + kTile - 1) / kTile;
    if (!BI_IN_BOUNDS(nc <= p.chunks && row < (EXT ? p.total_q : p.batch), p.status)) return;
    const float *w = p.ws + (row * p.Hq + h) * static_cast<int64_t>(p.chunks) * kRecord;
    const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(w) & 15u) / 4);   // copies begin at 16 bytes
    // floats of tile t's stage; where they end inside 16 bytes, the last two are not part of the copy (it would read
    // past the workspace) but loaded by hand
    auto floats = [&](int t) { return min(kTile, nc - t * kTile) * kRecord + skew; };
    auto fill = [&](int t) {                               // one lane
        const uint32_t bytes = static_cast<uint32_t>(floats(t) & ~3) * 4;
        mbar_arrive_expect_tx(&full[t % ring], bytes);
        bulk_load(tiles + t % ring * kMergeStage, w - skew + static_cast<int64_t>(t) * kTile * kRecord, bytes, &full[t % ring]);
    };
    auto tile_at = [&](int t) { return reinterpret_cast<const float *>(tiles + t % ring * kMergeStage) + skew; };
    float m_run = -INFINITY;                               // the loader's running maximum
    auto factors = [&](int t) {                            // warp 4: tile t's factors, once it has landed
        if (!mbar_wait(&full[t % ring], (t / ring) & 1, nullptr)) failed[t & 1] = 1;
        __syncwarp();
        const int n = floats(t);
        if ((n & 2) && lane < 2)
            reinterpret_cast<float *>(tiles + t % ring * kMergeStage)[n - 2 + lane] =
                w[static_cast<int64_t>(t) * kTile * kRecord + n - 2 + lane - skew];
        const float *rec = tile_at(t) + lane * kRecord;
        const bool in = t * kTile + lane < nc;
        const float mc = in ? rec[0] : -INFINITY, lc = in ? rec[1] : 0.0f;
        float incl = mc;                                   // max(m_c0 .. m_c) over the tile
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl = fmaxf(incl, v);
        }
        float before = __shfl_up_sync(0xffffffffu, incl, 1);
        before = lane == 0 ? m_run : fmaxf(m_run, before);
        float mn, a, bt;
        merge_factors(before, mc, mn, a, bt);
        fa[t & 1][lane] = a, fb[t & 1][lane] = bt, fl[t & 1][lane] = lc;
        m_run = fmaxf(m_run, __shfl_sync(0xffffffffu, incl, 31));
    };
    if (loader) {
        if (lane == 0)
            for (int t = 0; t < nt && t < ring; ++t) fill(t);
        __syncwarp();
        factors(0);
    }
    float o = 0.0f, l = 0.0f;
    for (int t = 0; t < nt; ++t) {
        __syncthreads();                                   // tile t's factors are there, tile t - 1 is merged
        if (failed[t & 1]) {                               // a wait ran out: report; the copies in flight get another limit
            if (d == kMergeThreads) {
                atomicOr(p.status, kDevTimeout);
                for (int k = t; k < nt && k < t + ring - (t > 0); ++k) mbar_wait(&full[k % ring], (k / ring) & 1, nullptr);
            }
            return;
        }
        if (loader) {
            if (lane == 0 && t > 0 && t - 1 + ring < nt) fill(t - 1 + ring);
            __syncwarp();
            if (t + 1 < nt) factors(t + 1);
        } else {
            const float *rec = tile_at(t) + 2 + d;
            const int n = min(kTile, nc - t * kTile);
            if (n == kTile) {
#pragma unroll
                for (int c = 0; c < kTile; ++c) {
                    o = merge_value(o, rec[c * kRecord], fa[t & 1][c], fb[t & 1][c]);
                    l = merge_value(l, fl[t & 1][c], fa[t & 1][c], fb[t & 1][c]);
                }
            } else {
                for (int c = 0; c < n; ++c) {
                    o = merge_value(o, rec[c * kRecord], fa[t & 1][c], fb[t & 1][c]);
                    l = merge_value(l, fl[t & 1][c], fa[t & 1][c], fb[t & 1][c]);
                }
            }
        }
    }
    if (!loader)
        p.O[(row * p.Hq + h) * kD + d] = static_cast<uint16_t>(pack_bf16x2(__float_as_uint(__fdiv_rn(o, l)), 0u) & 0xFFFFu);
}

template <int G, bool EXT, bool BLOCKS>
bi_status launch_split(int64_t items, int sms, const SplitParams &p, cudaStream_t s) {
    static unsigned long long configured = 0;
    constexpr int most = kMaxWarps * kWarpBytes;
    if (ensure_smem_attr(reinterpret_cast<const void *>(attn_split_int4_kernel<G, EXT, BLOCKS>), most, &configured) != BI_OK)
        return BI_ERR_CUDA;
    // one CTA per SM, with as many warps as there are items for it
    const int64_t per_sm = (items + sms - 1) / sms;
    const int warps = static_cast<int>(per_sm < kMaxWarps ? per_sm : kMaxWarps);
    return launch_pdl(attn_split_int4_kernel<G, EXT, BLOCKS>, dim3(static_cast<unsigned>(items < sms ? items : sms)),
                      dim3(32 * warps), warps * kWarpBytes, s, p);
}

template <bool EXT>
bi_status launch_few(SplitParams &p, cudaStream_t s) {
    int dev = 0;
    const DeviceInfo *info = nullptr;
    bi_status st = current_device(&dev, &info);
    if (st != BI_OK) return st;
    const int G = p.Hq / p.c.Hkv;
    p.tiles = EXT ? (p.max_q + 8 / G - 1) / (8 / G) : 1;
    p.chunks = static_cast<int32_t>((static_cast<int64_t>(p.max_len) + kChunk - 1) / kChunk);
    p.status = device_status_word();
    const int64_t items = p.batch * p.tiles * p.c.Hkv * static_cast<int64_t>(p.chunks);
    // Where the maximum length would make a walk of many steps (each some 450 cycles if there is nothing to do), a warp
    // first reads all lengths: 64 sequences of 1000 tokens, 32 heads over 8, maximum 131072: 96 us without this
    // and the merge's room below, 49 with this, 31 with both (29 at a maximum of 1000).
    p.scan = items >= 16 * static_cast<int64_t>(kMaxWarps) * info->sm_count && p.chunks * static_cast<int64_t>(p.tiles) * p.c.Hkv >= 64;
    const int64_t merges = p.batch * (EXT ? p.max_q : 1) * p.Hq;
    if (merges > 0x7FFFFFFF) return BI_ERR_UNSUPPORTED;
    // Block sizes that are multiples of eight can be copied as they lie (64 x 4096 tokens, blocks of 16: 91 us; by
    // rows, the same with 64 more copies a lane, 131 against 100 when it was measured).
    const bool blocks = p.c.bs % 8 == 0;
#define BI_SPLIT(g) st = blocks ? launch_split<g, EXT, true>(items, info->sm_count, p, s) \
                                : launch_split<g, EXT, false>(items, info->sm_count, p, s)
    switch (G) {
        case 1: BI_SPLIT(1); break;
        case 2: BI_SPLIT(2); break;
        case 4: BI_SPLIT(4); break;
        case 8: BI_SPLIT(8); break;
        default: return BI_ERR_UNSUPPORTED;
    }
#undef BI_SPLIT
    if (st != BI_OK) return st;
    static unsigned long long configured = 0;
    if (ensure_smem_attr(reinterpret_cast<const void *>(attn_merge_int4_kernel<EXT>), kMergeRing * kMergeStage, &configured) != BI_OK)
        return BI_ERR_CUDA;
    // Tiles on the way: as many as leave room for the other CTAs of the SM, up to six of them (256 sequences of 300
    // tokens, maximum 131072: 57 us for both kernels; with eight tiles, one CTA an SM, 135).
    const int64_t per_sm = (merges + info->sm_count - 1) / info->sm_count;
    const int tiles = (p.chunks + kMergeTile - 1) / kMergeTile;
    const int room = info->max_smem_optin / (kMergeStage + 1024) / static_cast<int>(per_sm < 6 ? per_sm : 6);
    int ring = tiles < kMergeRing ? tiles : kMergeRing;
    if (ring > room) ring = room;
    // and two at least where there are two: a tile's factors are made while the one before it is merged
    static_assert(kMergeRing >= 2, "two tiles of the merge");
    if (ring < 2 && tiles > 1) ring = 2;
    return launch_pdl(attn_merge_int4_kernel<EXT>, dim3(static_cast<unsigned>(merges)), dim3(kMergeThreads + 32), ring * kMergeStage, s,
                      p, ring);
}

}  // namespace

int64_t attention_extend_int4_workspace_bytes(int64_t total_q, int32_t Hq, int32_t Hkv, int32_t max_len, int32_t max_q) {
    const int64_t bytes = attention_decode_workspace_bytes(total_q, Hq, max_len);
    if (bytes < 0) return -1;
    if (bytes > kFewBytes) return 0;
    // (total_q is small here) sequences at least, the tiled kernel's CTAs with work at least
    const int64_t rows = total_q * (Hq / Hkv), seqs = (total_q + max_q - 1) / max_q;   // (max_q > total_q: one)
    const int64_t tiles = (rows + 127) / 128 > seqs ? (rows + 127) / 128 : seqs;
    const int64_t tiled = (tiles * Hkv + kSms - 1) / kSms * kTiledCost, split = (rows + 7) / 8 * Hkv * kSplitCost / kSms;
    return split < tiled ? bytes : 0;
}

bi_status launch_attention_decode_int4(const void *Q, const KvInt4 &c, const int32_t *table, int32_t max_blocks,
                                       const int32_t *lens, int64_t B, int32_t Hq, int32_t max_len, float scale,
                                       void *workspace, void *O, cudaStream_t s) {
    SplitParams p{};
    p.c = c;
    p.Q = static_cast<const uint16_t *>(Q);
    p.table = table;
    p.lens = lens;
    p.ws = static_cast<float *>(workspace);
    p.O = static_cast<uint16_t *>(O);
    p.batch = B;
    p.max_blocks = max_blocks;
    p.Hq = Hq;
    p.max_len = max_len;
    p.scale = scale;
    return launch_few<false>(p, s);
}

bi_status launch_attention_extend_int4_few(const void *Q, const int32_t *cu_q, int32_t total_q, const KvInt4 &c,
                                           const int32_t *table, int32_t max_blocks, const int32_t *lens, int64_t B,
                                           int32_t Hq, int32_t max_len, int32_t max_q, float scale, void *workspace,
                                           void *O, cudaStream_t s) {
    SplitParams p{};
    p.c = c;
    p.Q = static_cast<const uint16_t *>(Q);
    p.cu_q = cu_q;
    p.total_q = total_q;
    p.max_q = max_q;
    p.table = table;
    p.lens = lens;
    p.ws = static_cast<float *>(workspace);
    p.O = static_cast<uint16_t *>(O);
    p.batch = B;
    p.max_blocks = max_blocks;
    p.Hq = Hq;
    p.max_len = max_len;
    p.scale = scale;
    return launch_few<true>(p, s);
}

}  // namespace bi
