// attention_extend.cu -- extend (prefill) attention over the paged bf16 cache
// with a sliding window and first tokens that stay visible.
//
// A token's result is that of windowed decode of its cut sequence, bit for bit:
// the chunks of 128 tokens by position in which it sees something, the same
// chains of mma.sync m16n8k16 (q.k over ascending dimensions, p.V over ascending
// tokens with p as bf16 hi + lo), the same maximum, exponentials and order of the
// sum, the same merge in chunk order.
//
// One CTA per (sequence, KV head, 128 query rows = 128 / G tokens x G heads), one
// an SM. A loading warp brings the chunks' K and V into two buffers each (TMA boxes,
// one per cache block; 16-byte copies where boxes cannot tile the block size),
// counted on "full" barriers and given back, K and V apart, on "empty" ones. Eight
// warps of 16 rows compute, each at its own pace: no barrier of all warps stands
// between two chunks, so one warp's softmax and merge run under the other's products on
// the same scheduler (1 x 4096 tokens over 8192, window 2000: 744 us when this was measured; with
// the two taking turns on the tensor pipe 817, and with barriers between the chunks, as
// in the kernel without a window, 859). A warp goes from p.V of a chunk straight to q.k of the next.
// Scores, p and a chunk's sums are in registers; the running outputs, 64 a thread, are
// in tensor memory and fetched to merge a chunk. Twelve warps of 160 registers were
// slower (871; 757 with p.V in two halves); so were warps that left out chunks none of
// their own rows sees (799: the loop's code falls apart into pieces that are scheduled apart).
//
// What is out of sight: rows that no token of the tile sees are zeroed in V by the
// loading warp; of the others, a row that is out of some token's sight and not
// finite would reach it as 0 * NaN. The loading warp looks through V of the chunks
// that are masked for some token (two or three a tile), and where it finds such a
// value, p.V runs once for every token of a warp's rows, with zeros for the tokens
// out of that one's sight.
//
// Bound by mma.sync (1.5 times the operations, for p in two parts: some 62 % of its pipe
// while an SM is busy) and the eight warps' ldmatrix of K and V, then by a tile's start
// (6600 cycles of 80000 for five chunks) and the last round of tiles. 4096 tokens over 8192: window 2000
// 698 us (194 TFLOP/s); without a window that matters 1669 (247), attention.cu's kernel 1909.
#include "attn_common.cuh"
#include "bi_internal.h"

namespace bi {
namespace {

constexpr int kRows = 128;                     // query rows (token, head) per CTA: one m16 tile per warp
constexpr int kConsumers = 256;
// Of the loading warpgroup one warp loads; it is a whole one so that registers can be moved to the consumers, 384
// threads of 168 at launch.
constexpr int kThreads = kConsumers + 128;
constexpr int kLaunchRegs = 168, kLoadRegs = 40, kConsumerRegs = 232;
static_assert(kConsumers * kConsumerRegs + (kThreads - kConsumers) * kLoadRegs <= kThreads * kLaunchRegs, "registers to share");
constexpr int kStages = 2;                     // buffers of K and of V
constexpr int kFlagSets = 4;                   // row flags: those of chunk c are read until its softmax, and K of chunk c + 2 comes before
constexpr int kTmemCols = 128;                 // running outputs: 64 columns for each of the two warps of a quadrant
constexpr int kBarriers = 4 * kStages + 1;
constexpr int kSmem = 1024 + 2 * kStages * kTileBytes + kRows * kRowBytes + kFlagSets * kChunk + kBarriers * 8 + 16 * 4;
static_assert(kSmem <= 232448, "one CTA's shared memory");

struct ExtParams {
    const uint16_t *Q;       // [total_q][Hq][D]
    const int32_t *cu_q;     // [B+1]
    const uint16_t *K;       // [blocks][bs][Hkv][D]
    const uint16_t *V;
    const int32_t *table;    // [B][max_blocks]
    const int32_t *lens;     // [B], cached length including the new tokens
    uint16_t *O;             // [total_q][Hq][D]
    int64_t num_blocks, batch;
    int32_t total_q, max_blocks, Hq, Hkv, bs, max_len, max_q;
    int32_t few;             // sequences of at most this many new tokens are computed elsewhere
    int32_t window, sinks, box_rows;
    float scale;
    unsigned *status;
};

template <int G>
__global__ void __launch_bounds__(kThreads, 1)
attn_extend_window_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const ExtParams p) {
    constexpr int kTQ = kRows / G;                     // query tokens per CTA
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *Kt = smem, *Vt = smem + kStages * kTileBytes;                              // [kStages] tiles, as TMA swizzles them
    uint16_t *qb = reinterpret_cast<uint16_t *>(smem + 2 * kStages * kTileBytes);       // [kRows][kD]
    uint8_t *flags = reinterpret_cast<uint8_t *>(qb + kRows * kD);                      // [kFlagSets][kChunk]: row is in the cache
    uint64_t *fullK = reinterpret_cast<uint64_t *>(flags + kFlagSets * kChunk);
    uint64_t *fullV = fullK + kStages, *emptyK = fullV + kStages, *emptyV = emptyK + kStages, *land = emptyV + kStages;
    volatile int *bad_of = reinterpret_cast<volatile int *>(land + 1);                  // [kFlagSets]: a row in sight is not in the cache
    volatile int *odd_of = bad_of + kFlagSets;                                          // [kStages]: p.V by tokens
    volatile int *abort_flag = odd_of + kStages;
    __shared__ uint32_t tmem_base;
    __shared__ int sequence;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == kThreads / 32 - 1) {                   // beside the others' search for the tile
        tmem_alloc(&tmem_base, kTmemCols);
        tmem_relinquish();
    }
    // blockIdx.x = (tile from the last, KV head): late tokens, which see more, start first. Sequence b's tiles are
    // numbered from cu_q[b] / kTQ + b on, so that there are no more of them than tokens / kTQ + sequences, whatever
    // the longest: the last b that begins at or before this one, 32 at a time.
    const int g = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.Hkv));
    const int64_t v = (gridDim.x - 1 - blockIdx.x) / static_cast<unsigned>(p.Hkv);
    auto wrong = [&](int64_t x0, int64_t x1, int n) {
        return x0 < 0 || x1 < x0 || x1 > p.total_q || x1 - x0 > p.max_q || n < x1 - x0 || n > p.max_len ||
               n > static_cast<int64_t>(p.max_blocks) * p.bs;
    };
    // One warp searches and hands the sequence on (with the search in every warp the consumers spilled more: 4096 tokens over
    // 8192, window 2000, 707 us against 702).
    if (warp == kConsumers / 32) {
        int64_t at = 0;
        for (int64_t span = p.batch; span > 1;) {
            const int64_t step = (span + 31) / 32, x = at + lane * step;
            const bool starts = lane * step < span && (lane == 0 || p.cu_q[x] / kTQ + x <= v);
            const int last = 31 - __clz(static_cast<int>(__ballot_sync(0xffffffffu, starts)));
            at += last * step;
            span = min(step, span - last * step);
        }
        // An offset out of range leads the search astray: then it is the sequence in range, of all of them, that has this tile.
        const int64_t x0 = p.cu_q[at], x1 = p.cu_q[at + 1];
        if (wrong(x0, x1, p.lens[at]) || x0 / kTQ + at > v || (at + 1 < p.batch && x1 / kTQ + at + 1 <= v)) {
#pragma unroll 1
            for (int64_t x = lane; x - lane < p.batch; x += 32) {
                bool has = false;
                if (x < p.batch) {
                    const int64_t y0 = p.cu_q[x], y1 = p.cu_q[x + 1], tile = v - (y0 / kTQ + x);
                    has = !wrong(y0, y1, p.lens[x]) && tile >= 0 && tile * kTQ < y1 - y0;
                }
                const unsigned found = __ballot_sync(0xffffffffu, has);
                if (found) {
                    at = x - lane + __ffs(static_cast<int>(found)) - 1;
                    break;
                }
            }
        }
        if (lane == 0) sequence = static_cast<int>(at);
    }
    __syncthreads();
    const int b = sequence, q0 = p.cu_q[b], q1 = p.cu_q[b + 1], L = p.lens[b];
    const int64_t tile = v - (q0 / kTQ + b), qlen = static_cast<int64_t>(q1) - q0;
    if (blockIdx.x == 0)                               // one CTA looks at every sequence
        for (int64_t x = tid; x < p.batch; x += kThreads)
            if (wrong(p.cu_q[x], p.cu_q[x + 1], p.lens[x])) atomicOr(p.status, kDevBadOffsets);
    if (wrong(q0, q1, L) || qlen <= p.few || tile < 0 || tile * kTQ >= qlen) {
        tc_fence_before();
        __syncthreads();                               // (the allocation has been written)
        tc_fence_after();
        if (warp == kThreads / 32 - 1) tmem_dealloc(tmem_base, kTmemCols);
        return;
    }
    const int i0 = static_cast<int>(tile) * kTQ;       // first query token of this CTA
    const int ntok = min(kTQ, q1 - q0 - i0);
    const int base = L - (q1 - q0);                    // position of query token 0
    const int first_n = base + i0 + 1, last_n = base + i0 + ntok;   // what the first and the last token would see without a window
    const Seen w(first_n - p.window, p.sinks);         // what the tile's tokens see together
    const int nchunks = w.chunks(last_n);

    if (tid == 0) {
        const int copies = p.box_rows > 0 ? 1 : 64;    // arrivals that fill a buffer: one with the bytes, or two a lane
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&fullK[s], copies);
            mbar_init(&fullV[s], copies);
            mbar_init(&emptyK[s], kConsumers / 32);
            mbar_init(&emptyV[s], kConsumers / 32);
        }
        mbar_init(land, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    // q rows: row r = token r / G, head g*G + r % G (zero rows past the tokens);
    // 16-byte piece x of row r at piece x ^ (r % 8)
    if (warp < kConsumers / 32) {
        for (int i = tid; i < kRows * kD / 8; i += kConsumers) {
            const int r = i / (kD / 8), x = i % (kD / 8);
            const bool v = r / G < ntok;
            cp_async_16(smem_u32(qb + r * kD + ((x ^ (r & 7)) * 8)),
                        v ? p.Q + (static_cast<int64_t>(q0 + i0 + r / G) * p.Hq + g * G + r % G) * kD + x * 8 : p.Q, v ? 16u : 0u);
        }
        cp_async_commit();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    if (warp >= kConsumers / 32) {
        setmaxnreg_dec<kLoadRegs>();
        if (warp > kConsumers / 32) {
            __syncthreads();                           // the consumers' last
            return;
        }
        // ---- loading warp
        if (lane == 0 && p.box_rows > 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        int lands = 0, lastK = -1, lastV = -1;
        auto freed = [&](uint64_t *bar, int c) {       // the buffer's last chunk is done with
            if (c < kStages || mbar_wait(bar, ((c / kStages) - 1) & 1, abort_flag)) return true;
            if (lane == 0) {
                atomicOr(p.status, kDevTimeout);
                *abort_flag = 1;
            }
            return false;
        };
        for (int c = 0; c < nchunks; ++c) {
            const int s = c % kStages, j0 = w.start(c), n = min(kChunk, last_n - j0);
            const int h0 = max(w.first - j0, 0), h1 = min(w.lo - j0, n);        // [h0, h1): out of the tile's sight
            // masked for some token: the first one's length, or the last one's window
            const bool masked = j0 + kChunk > first_n || (j0 < last_n - p.window && j0 + kChunk > p.sinks);
            // the chunk's rows: block, offset, flag
            int32_t row_blk[kChunk / 32];              // per-row copies: each row's block, -1: none
            uint32_t in = 0, wrong = 0;                // bit i: row lane + 32 i is in the cache; or in sight, but not there
            int32_t blk = -1;                          // boxes: lane i holds box i's block
            const bool box = p.box_rows > 0 && lane * p.box_rows < n && (lane * p.box_rows < h0 || (lane + 1) * p.box_rows > h1);
            if (box) blk = p.table[static_cast<int64_t>(b) * p.max_blocks + (j0 + lane * p.box_rows) / p.bs];
#pragma unroll
            for (int i = 0; i < kChunk / 32; ++i) {
                const int t = lane + 32 * i;
                const bool seen = t < n && !(t >= h0 && t < h1);
                int32_t x = -1;
                if (p.box_rows > 0)
                    x = __shfl_sync(0xffffffffu, blk, t / p.box_rows);
                else if (seen)
                    x = p.table[static_cast<int64_t>(b) * p.max_blocks + (j0 + t) / p.bs];
                const bool ok = seen && x >= 0 && x < p.num_blocks;
                row_blk[i] = ok ? x : -1;
                in |= static_cast<uint32_t>(ok) << i;
                wrong |= static_cast<uint32_t>(seen && !ok);
            }
            if (wrong) atomicOr(p.status, kDevBadOffsets);
            wrong = __any_sync(0xffffffffu, wrong != 0);
            if (!freed(&emptyK[s], c)) break;
            uint8_t *f = flags + (c % kFlagSets) * kChunk;
#pragma unroll
            for (int i = 0; i < kChunk / 32; ++i) f[lane + 32 * i] = (in >> i) & 1u;
            if (lane == 0) bad_of[c % kFlagSets] = wrong;
            __syncwarp();
            uint8_t *Ks = Kt + s * kTileBytes, *Vs = Vt + s * kTileBytes;
            const int tok = (j0 + lane * p.box_rows) % p.bs;
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, box)) * p.box_rows * kRowBytes;
            auto boxes = [&](uint8_t *dst, const CUtensorMap *tm, uint64_t *bar) {
                if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
                __syncwarp();
                if (box) {                             // a block outside the cache arrives as zeros
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        tma_load_4d(dst + half * kHalfTile + lane * p.box_rows * 128, tm, bar, half * 64, g, tok, blk);
                }
            };
            auto rows = [&](uint8_t *dst, const uint16_t *src) {   // two rows an instruction; rows that are not there become zeros
#pragma unroll
                for (int i = 0; i < kChunk / 32; ++i)
#pragma unroll 1
                    for (int k = 0; k < 16; ++k) {
                        const int t = 32 * i + 2 * k + (lane >> 4), x = lane & 15;
                        const int64_t o = __shfl_sync(0xffffffffu, row_blk[i], t & 31);
                        cp_async_16(smem_u32(dst) + kv_piece(t, x),
                                    o >= 0 ? src + ((o * p.bs + (j0 + t) % p.bs) * p.Hkv + g) * kD + x * 8 : src, o >= 0 ? 16u : 0u);
                    }
            };
            auto arrive_rows = [&](uint64_t *bar) {    // now, and once this lane's copies have landed
                mbar_arrive(bar);
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
            };
            if (p.box_rows > 0) {
                boxes(Ks, &tmK, &fullK[s]);
            } else {
                rows(Ks, p.K);
                arrive_rows(&fullK[s]);
            }
            lastK = c;
            if (!freed(&emptyV[s], c)) break;
            if (!masked) {
                if (lane == 0) odd_of[s] = 0;
                __syncwarp();
                if (p.box_rows > 0) {
                    boxes(Vs, &tmV, &fullV[s]);
                } else {
                    rows(Vs, p.V);
                    arrive_rows(&fullV[s]);
                }
            } else {
                // wait for V here: zero the rows that no token sees, look for values that are not finite in the others
                bool ok = true;
                if (p.box_rows > 0) {
                    boxes(Vs, &tmV, land);
                    ok = mbar_wait(land, lands++ & 1, abort_flag);
                } else {
                    rows(Vs, p.V);
                    cp_async_commit();
                    cp_async_wait<0>();
                    __syncwarp();
                }
                if (!__all_sync(0xffffffffu, ok)) {
                    if (lane == 0) {
                        atomicOr(p.status, kDevTimeout);
                        *abort_flag = 1;
                        mbar_wait(land, (lands - 1) & 1, nullptr);   // its copies, with a limit of their own
                    }
                    __syncwarp();
                    break;
                }
                // (rows that every token sees need neither)
                const int every = first_n - j0, from = last_n - p.window - j0;
                bool fine = true;
#pragma unroll 4
                for (int i = 0; i < kChunk / 2; ++i) {
                    const int t = 2 * i + (lane >> 4);
                    if (t < every && (t < p.sinks - j0 || t >= from)) continue;
                    const uint32_t a = smem_u32(Vs) + kv_piece(t, lane & 15);
                    if (t < n && !(t >= h0 && t < h1)) {
                        uint32_t x0, x1, x2, x3;
                        ld_shared_v4(a, x0, x1, x2, x3);
                        fine = fine && finite_pair(x0) && finite_pair(x1) && finite_pair(x2) && finite_pair(x3);
                    } else {
                        st_shared_v4(a, 0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async_smem();              // before later bulk copies into these rows
                fine = __all_sync(0xffffffffu, fine);
                if (lane == 0) odd_of[s] = !fine;
                __syncwarp();
                if (p.box_rows == 0) {
                    mbar_arrive(&fullV[s]);
                    mbar_arrive(&fullV[s]);
                } else if (lane == 0) {
                    mbar_arrive(&fullV[s]);
                }
            }
            lastV = c;
        }
        // the copies of the last chunks must land before the CTA exits
        for (int d = 0; d < kStages; ++d) {
            if (lastK - d >= 0) mbar_wait(&fullK[(lastK - d) % kStages], ((lastK - d) / kStages) & 1, nullptr);
            if (lastV - d >= 0) mbar_wait(&fullV[(lastV - d) % kStages], ((lastV - d) / kStages) & 1, nullptr);
        }
        __syncthreads();                               // the consumers' last
        return;
    }

    setmaxnreg_inc<kConsumerRegs>();
    // ---- consumers: warp rt has rows 16 rt .. 16 rt + 15
    const int gq = lane >> 2, cq = lane & 3;           // fragment row group, column pair
    const int rt = warp;                               // row tile
    const int ra = rt * 16 + gq, rb = ra + 8;          // this thread's two rows
    const int qrow = rt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
    const uint32_t qaddr = smem_u32(qb) + qrow * kRowBytes;
    const uint32_t o_run = tmem_base + (static_cast<uint32_t>(warp & 3) << 21) + (warp >> 2) * 64;   // this warp's lanes and columns
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.0f, 0.0f};
    {
        uint32_t z[16] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_st_32x32b_x16(o_run + 16 * i, z, 0);
    }
    // the causal length of each row: position + 1 (0 for rows past the tokens)
    const int len_a = ra / G < ntok ? base + i0 + ra / G + 1 : 0;
    const int len_b = rb / G < ntok ? base + i0 + rb / G + 1 : 0;
    bool dead = false;                                 // a wait ran out: go on to the end of the protocol, store nothing
    auto landed = [&](uint64_t *bar, int c) {
        if (!mbar_wait(bar, (c / kStages) & 1, abort_flag)) {
            if (lane == 0) {
                atomicOr(p.status, kDevTimeout);
                *abort_flag = 1;
            }
            dead = true;
        }
        __syncwarp();
    };

    constexpr int kTokens = 16 / G;                    // of this warp's rows
    const f2 scale2 = f2_of(p.scale, p.scale);
    auto pair = [](const float (&x)[4], int h) { return f2_of(x[2 * h], x[2 * h + 1]); };
    auto unpair = [](f2 v, float (&x)[4], int h) { x[2 * h] = __uint_as_float(lo_of(v)), x[2 * h + 1] = __uint_as_float(hi_of(v)); };
    // scores q . k of the tile's 16 rows and a chunk's 128 tokens, dimensions ascending in
    // 16-dimension steps. s[nt][e]: row ra (e < 2) or rb, token 8 nt + 2 cq + (e & 1).
    float s[kChunk / 8][4];
    auto scores = [&](int c) {
        landed(&fullK[c % kStages], c);
        const uint32_t Ks = smem_u32(Kt + (c % kStages) * kTileBytes);
#pragma unroll
        for (int nt = 0; nt < kChunk / 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
#pragma unroll
        for (int kp = 0; kp < kD / 32; ++kp) {                     // two 16-dimension steps per ldmatrix
            uint32_t qf[2][4];
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
                const int piece = 2 * (2 * kp + k2) + (lane >> 4);
                ldmatrix_x4(qf[k2][0], qf[k2][1], qf[k2][2], qf[k2][3], qaddr + ((piece ^ (qrow & 7)) << 4));
            }
#pragma unroll
            for (int nt = 0; nt < kChunk / 8; ++nt) {
                uint32_t b0, b1, b2, b3;
                ldmatrix_x4(b0, b1, b2, b3, Ks + kv_piece(nt * 8 + (lane & 7), 4 * kp + (lane >> 3)));
                mma_16816(s[nt], qf[0][0], qf[0][1], qf[0][2], qf[0][3], b0, b1);
                mma_16816(s[nt], qf[1][0], qf[1][1], qf[1][2], qf[1][3], b2, b3);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&emptyK[c % kStages]);
    };
    // values: sum_t p_t v_t for all 128 dimensions, p = hi + lo (two products a step), tokens
    // ascending in 16-token steps; p is already in the A-fragment layout. BY_TOKEN: zeros for the
    // tokens t >= tn and those in [ts, tf).
    float acc[kD / 8][4];
    auto values = [&](uint32_t Vs, auto by_token, int tn, int ts, int tf) {
#pragma unroll
        for (int nt = 0; nt < kD / 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] = 0.0f;
        const int mi = lane >> 3, mr = lane & 7;       // ldmatrix: matrix, row
#pragma unroll
        for (int ks = 0; ks < kChunk / 16; ++ks) {
            uint32_t ph0, pl0, ph1, pl1, ph2, pl2, ph3, pl3;
            split_bf16x2(s[2 * ks][0], s[2 * ks][1], ph0, pl0);
            split_bf16x2(s[2 * ks][2], s[2 * ks][3], ph1, pl1);
            split_bf16x2(s[2 * ks + 1][0], s[2 * ks + 1][1], ph2, pl2);
            split_bf16x2(s[2 * ks + 1][2], s[2 * ks + 1][3], ph3, pl3);
            const int tok = ks * 16 + (mi & 1) * 8 + mr;
            uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};         // of the fragments' token pairs
            if (decltype(by_token)::value) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int t = ks * 16 + 8 * h + 2 * cq;
                    keep[h] = (t < tn && !(t >= ts && t < tf) ? 0xFFFFu : 0u) |
                              (t + 1 < tn && !(t + 1 >= ts && t + 1 < tf) ? 0xFFFF0000u : 0u);
                }
            }
            // dimensions in two halves of 64 (four ldmatrix each); each accumulator takes hi, then lo
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t v[4][4];
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {       // two 8-dimension tiles per ldmatrix
                    ldmatrix_x4_trans(v[q4][0], v[q4][1], v[q4][2], v[q4][3], Vs + kv_piece(tok, 2 * (4 * half + q4) + (mi >> 1)));
                    if (decltype(by_token)::value) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[q4][k] &= keep[k & 1];
                    }
                }
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                    const int np = 4 * half + q4;
                    mma_16816(acc[2 * np], ph0, ph1, ph2, ph3, v[q4][0], v[q4][1]);
                    mma_16816(acc[2 * np + 1], ph0, ph1, ph2, ph3, v[q4][2], v[q4][3]);
                }
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                    const int np = 4 * half + q4;
                    mma_16816(acc[2 * np], pl0, pl1, pl2, pl3, v[q4][0], v[q4][1]);
                    mma_16816(acc[2 * np + 1], pl0, pl1, pl2, pl3, v[q4][2], v[q4][3]);
                }
            }
        }
    };
    // the chunk's sums into the rows' running state, for the rows that take part
    auto merge = [&](bool in_a, bool in_b, const float (&m)[2], const float (&l)[2]) {
        const bool in[2] = {in_a, in_b};
        float al[2], be[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float mn;
            merge_factors(m_run[h], m[h], mn, al[h], be[h]);
            if (in[h]) {
                m_run[h] = mn;
                l_run[h] = merge_value(l_run[h], l[h], al[h], be[h]);
            }
        }
        tmem_wait_st();                                // the merge before
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t run[32];
            tmem_ld_32x32b_x32(o_run + 32 * i, run);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; k += 2) {              // (merge_value, two dimensions at once)
                const int nt = 8 * i + k / 4, h = (k >> 1) & 1;
                if (in[h]) {
                    const f2 x = fma2(pair(acc[nt], h), f2_of(be[h], be[h]), mul2(f2_of(run[k], run[k + 1]), f2_of(al[h], al[h])));
                    run[k] = lo_of(x), run[k + 1] = hi_of(x);
                }
            }
            tmem_st_32x32b_x16(o_run + 32 * i, run, 0);
            tmem_st_32x32b_x16(o_run + 32 * i + 16, run, 16);
        }
    };

    cp_async_wait<0>();                                // q rows: this thread's
    asm volatile("bar.sync 3, 256;" ::: "memory");     // every consumer's
    if (rt * kTokens >= ntok) {                        // no rows: give the chunks back
        for (int c = 0; c < nchunks; ++c) {
            landed(&fullK[c % kStages], c);
            if (lane == 0) mbar_arrive(&emptyK[c % kStages]);
            landed(&fullV[c % kStages], c);
            if (lane == 0) mbar_arrive(&emptyV[c % kStages]);
        }
    } else {
        scores(0);
        for (int c = 0; c < nchunks; ++c) {
            const int j0 = w.start(c);
            const uint8_t *in_cache = flags + (c % kFlagSets) * kChunk;
            const bool bad = bad_of[c % kFlagSets] != 0;
            // tokens of this chunk each row sees: t < na (nb), and t < s0 or t >= fa (fb)
            const int na = max(0, min(kChunk, len_a - j0)), nb = max(0, min(kChunk, len_b - j0));
            const int s0 = p.sinks - j0, fa = len_a - p.window - j0, fb = len_b - p.window - j0;
            auto sees = [&](int h, int t) { return t < (h ? nb : na) && (t < s0 || t >= (h ? fb : fa)); };
            auto sees_any = [&](int h) { return (h ? nb : na) > 0 && (s0 > 0 || (h ? fb : fa) < (h ? nb : na)); };
            // a chunk every row of the tile sees whole, with every block valid, needs no masks
            const bool whole = !bad && __all_sync(0xffffffffu, na == kChunk && nb == kChunk && (s0 >= kChunk || (fa <= 0 && fb <= 0)));
            float m[2] = {-INFINITY, -INFINITY}, l[2];
            if (whole) {
#pragma unroll
                for (int nt = 0; nt < kChunk / 8; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        unpair(mul2(pair(s[nt], h), scale2), s[nt], h);
                        m[h] = fmaxf(m[h], fmaxf(s[nt][2 * h], s[nt][2 * h + 1]));
                    }
            } else {
                // what a row does not see scores -inf, so p = 0 there
#pragma unroll
                for (int nt = 0; nt < kChunk / 8; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = nt * 8 + 2 * cq + (e & 1);
                        s[nt][e] = sees(e >> 1, t) ? __fmul_rn(s[nt][e], p.scale) : -INFINITY;
                    }
                if (bad) {                                 // a row of the chunk is not in the cache
                    int any[2] = {0, 0};
#pragma unroll
                    for (int nt = 0; nt < kChunk / 8; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int t = nt * 8 + 2 * cq + (e & 1);
                            any[e >> 1] |= sees(e >> 1, t) && in_cache[t];
                            if (!in_cache[t]) s[nt][e] = -INFINITY;
                        }
                    // the chunk counts nothing for a token that sees no row of it in the cache
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        any[h] |= __shfl_xor_sync(0xffffffffu, any[h], 1);
                        any[h] |= __shfl_xor_sync(0xffffffffu, any[h], 2);
                        if (!any[h]) m[h] = kNoScore;
                    }
                }
#pragma unroll
                for (int nt = 0; nt < kChunk / 8; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) m[e >> 1] = fmaxf(m[e >> 1], s[nt][e]);
            }
            // per row: max (any order gives the same value), then e^(s - m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                m[h] = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], 1));
                m[h] = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], 2));
            }
            const f2 minus[2] = {f2_of(-m[0], -m[0]), f2_of(-m[1], -m[1])};
#pragma unroll
            for (int nt = 0; nt < kChunk / 8; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    unpair(add2(pair(s[nt], h), minus[h]), s[nt], h);
                    s[nt][2 * h] = expf(s[nt][2 * h]);
                    s[nt][2 * h + 1] = expf(s[nt][2 * h + 1]);
                }
            // per row: the sum in decode's order. Lane L of decode sums tokens
            // L, L + 32, L + 64, L + 96 in turn, then a butterfly over lanes xor
            // 16, 8, 4, 2, 1. Here L = 8 (nt % 4) + 2 cq + (e & 1): the column
            // steps (nt + 4k) and the butterfly steps 16 and 8 (nt ^ 2, nt ^ 1) and
            // 1 (e ^ 1) are in this thread; steps 4 and 2 are lanes xor 2 and 1.
            // Each butterfly step adds two equal-rank partials, and a + b = b + a,
            // so every lane's total is the same bits as decode's.
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f2 col[4];                                                    // both e & 1 at once
#pragma unroll
                for (int n4 = 0; n4 < 4; ++n4) {
                    col[n4] = pair(s[n4], h);
#pragma unroll
                    for (int k = 1; k < 4; ++k) col[n4] = add2(col[n4], pair(s[n4 + 4 * k], h));
                }
                const f2 v = add2(add2(col[0], col[2]), add2(col[1], col[3]));   // steps 16 and 8
                float x[2] = {__uint_as_float(lo_of(v)), __uint_as_float(hi_of(v))};
#pragma unroll
                for (int e0 = 0; e0 < 2; ++e0) {
                    x[e0] += __shfl_xor_sync(0xffffffffu, x[e0], 2);          // step 4
                    x[e0] += __shfl_xor_sync(0xffffffffu, x[e0], 1);          // step 2
                }
                l[h] = x[0] + x[1];                                           // step 1
            }

            landed(&fullV[c % kStages], c);
            const uint32_t Vs = smem_u32(Vt + (c % kStages) * kTileBytes);
            const bool odd = odd_of[c % kStages] != 0;
            if (odd) {
                for (int u = 0; u < kTokens; ++u) {
                    const int n = base + i0 + rt * kTokens + u + 1 - j0;
                    values(Vs, std::true_type{}, n, max(s0, 0), n - p.window);
                    if (u + 1 < kTokens) merge(sees_any(0) && gq / G == u, sees_any(1) && (gq + 8) / G == u, m, l);
                }
            } else {
                values(Vs, std::false_type{}, 0, 0, 0);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&emptyV[c % kStages]);
            if (c + 1 < nchunks) scores(c + 1);
            constexpr int kLast = kTokens - 1;             // by tokens: the last one's
            merge(sees_any(0) && !(odd && gq / G != kLast), sees_any(1) && !(odd && (gq + 8) / G != kLast), m, l);
        }
    }

    // o / l, rounded to bf16, for the rows that exist
    tmem_wait_st();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t run[32];
        tmem_ld_32x32b_x32(o_run + 32 * i, run);
        tmem_wait_ld();
        // a row's quad has two dimensions of each tile in every lane: turned round, a lane has all eight of tiles cq, 4 + cq
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = h ? rb : ra;
            const bool stored = !dead && r / G < ntok && BI_IN_BOUNDS(q0 + i0 + r / G < p.total_q, p.status);
            uint16_t *orow = p.O + (static_cast<int64_t>(q0 + i0 + r / G) * p.Hq + g * G + r % G) * kD + 64 * i;
#pragma unroll
            for (int four = 0; four < 2; ++four) {
                uint32_t x[4], y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int at = 16 * four + 4 * k + 2 * h;
                    x[k] = pack_bf16x2(__float_as_uint(__fdiv_rn(__uint_as_float(run[at]), l_run[h])),
                                       __float_as_uint(__fdiv_rn(__uint_as_float(run[at + 1]), l_run[h])));
                }
                // lane cq gives tile k to lane k: exchanges with lanes cq ^ 1, then cq ^ 2
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, cq & 1 ? x[k] : x[k + 1], 1);
                    y[k] = cq & 1 ? got : x[k];
                    y[k + 1] = cq & 1 ? x[k + 1] : got;
                }
                // y[k], y[k + 1]: tile k + (cq & 1) of lanes cq & ~1 and cq | 1
                uint32_t lo[2], hi[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, cq & 2 ? y[k] : y[2 + k], 2);
                    lo[k] = cq & 2 ? got : y[k];
                    hi[k] = cq & 2 ? y[2 + k] : got;
                }
                if (stored) *reinterpret_cast<uint4 *>(orow + 32 * four + 8 * cq) = make_uint4(lo[0], lo[1], hi[0], hi[1]);
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

template <int G>
bi_status launch_g(const dim3 &grid, const CUtensorMap &tmK, const CUtensorMap &tmV, const ExtParams &p, cudaStream_t s) {
    static unsigned long long configured = 0;
    // the consumers wait for registers that have to be there
    static const bool enough = [] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, reinterpret_cast<const void *>(attn_extend_window_kernel<G>)) == cudaSuccess &&
               a.numRegs == kLaunchRegs;
    }();
    if (!enough) return BI_ERR_CUDA;
    if (ensure_smem_attr(reinterpret_cast<const void *>(attn_extend_window_kernel<G>), kSmem, &configured) != BI_OK)
        return BI_ERR_CUDA;
    return launch_pdl(attn_extend_window_kernel<G>, grid, dim3(kThreads), kSmem, s, tmK, tmV, p);
}

}  // namespace

// The chunk results of the split take at most kFewBytes.
constexpr int64_t kFewBytes = 512ll << 20;

int64_t attention_extend_window_workspace_bytes(int64_t total_q, int32_t Hq, int32_t max_len, int32_t window, int32_t sinks) {
    const int64_t bytes = attention_decode_workspace_bytes(total_q, Hq, max_len, window, sinks);
    return bytes > kFewBytes ? 0 : bytes;
}

// Which sequences are split over the chunks: all, where that should take less time for the call; else those of at most
// kFewRows query rows, for which it takes less of an SM's time (a chunk of a tile of 16 rows 1.4 us, of 128 rows 5.3).
// In us, on the sums that the host knows and for 152 SMs, so that the choice is the same wherever a size is asked for: drafts
// 16 x 5 over 100 to 4000, window 1024, 70 tiled, 38 split.
static bool split_all(int64_t B, int64_t total_q, int G, int32_t Hkv, int64_t seen, int64_t max_q) {
    constexpr int kSms = 152;
    const double chunks = static_cast<double>(seen);
    const int64_t rows = total_q * G, seqs = B < total_q ? B : total_q;
    const int64_t tiles = (rows + kRows - 1) / kRows > seqs ? (rows + kRows - 1) / kRows : seqs;
    const double tiled = static_cast<double>((tiles * Hkv + kSms - 1) / kSms) * (10.0 + 5.3 * chunks);
    const double split = 10.0 + static_cast<double>(((rows + 15) / 16 + seqs) * Hkv) * chunks * 1.4 / kSms;
    // (the split lays its work out for the most new tokens of every sequence: not where most of that would be empty)
    return split < tiled && B * max_q <= 4 * total_q;
}

// Results are held for the tokens that can be split, at most kFewBytes: for every row of Q, or, where those are fewer, `few`
// places a sequence (63 single tokens and a prompt of 2048, window 1024, 32 heads: 170 MB where every row would take 351). Where
// they would not fit, `few` is what does (the same with a window of 4096: 14 places a sequence instead of 16; 584 us, with
// the single tokens in tiles 1009).
FewPlan plan_few(int64_t B, int64_t total_q, int32_t Hq, int32_t Hkv, int32_t max_len, int32_t max_q, int32_t window, int32_t sinks) {
    constexpr int kFewRows = 64;
    const FewPlan none{0, 0, 0};
    if (B < 1 || total_q < 1) return none;
    const int64_t place = attention_decode_workspace_bytes(1, Hq, max_len, window, sinks), room = place > 0 ? kFewBytes / place : 0;
    const int G = Hq / Hkv;
    if (max_q > total_q) max_q = static_cast<int32_t>(total_q);
    int64_t few = kFewRows / G, places = total_q;
    if (total_q <= room && split_all(B, total_q, G, Hkv, seen_chunks(max_len, window, sinks), max_q)) {
        few = max_q;
    } else {
        if (total_q > room && few > room / B) {
            if (max_q <= few && total_q > B * (room / B)) return none;     // short ones alone, most of which would not fit
            few = room / B;
        }
        // mostly sequences of more tokens (a sequence of few has a tile of its own then; without any, the split's two
        // launches would cost 7 us for nothing): the tiled kernel alone
        if (max_q > few && (B == 1 || total_q > 4 * B * few)) few = 0;
        if (places > B * few) places = B * few;
    }
    // (the merge's grid)
    if (few == 0 || B * (few < max_q ? few : max_q) > 0x7fffffff / Hq) return none;
    return FewPlan{static_cast<int32_t>(few), places, places * place};
}

bi_status launch_attention_extend_window(const WindowCall &a, void *workspace, cudaStream_t s) {
    FewPlan plan{0, 0, 0};
    if (workspace) plan = plan_few(a.B, a.total_q, a.Hq, a.Hkv, a.max_len, a.max_q, a.window, a.sinks);
    if (plan.few > 0) {
        const bi_status st = launch_attention_few_window(a, plan, workspace, s);
        if (st != BI_OK || a.max_q <= plan.few) return st;
    }
    ExtParams p{};
    p.Q = static_cast<const uint16_t *>(a.Q);
    p.cu_q = a.cu_q;
    p.K = static_cast<const uint16_t *>(a.K);
    p.V = static_cast<const uint16_t *>(a.V);
    p.table = a.table;
    p.lens = a.lens;
    p.O = static_cast<uint16_t *>(a.O);
    p.num_blocks = a.num_blocks;
    p.batch = a.B;
    p.total_q = a.total_q;
    p.max_blocks = a.max_blocks;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.bs = a.bs;
    p.max_len = a.max_len;
    p.max_q = a.max_q;
    p.few = plan.few;
    p.window = a.window;
    p.sinks = a.sinks;
    p.scale = a.scale;
    p.status = device_status_word();
    CUtensorMap tmK{}, tmV{};
    p.box_rows = kv_box_maps(a.K, a.V, a.num_blocks, a.bs, a.Hkv, &tmK, &tmV);
    const int G = a.Hq / a.Hkv;
    const int64_t ctas = (a.total_q / (kRows / G) + a.B) * a.Hkv;   // (tile, KV head)
    if (ctas > 0x7fffffff) return BI_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(ctas));
    switch (G) {
        case 1: return launch_g<1>(grid, tmK, tmV, p, s);
        case 2: return launch_g<2>(grid, tmK, tmV, p, s);
        case 4: return launch_g<4>(grid, tmK, tmV, p, s);
        case 8: return launch_g<8>(grid, tmK, tmV, p, s);
        default: return BI_ERR_UNSUPPORTED;
    }
}

}  // namespace bi
