// attention_few.cu -- windowed extend attention for sequences with few new
// tokens (drafts to verify, single tokens in a batch with prompts): split over
// the cache's chunks like decode, with the same bits.
//
// An item is (sequence, tile of 16 / G or 32 / G new tokens, KV head, chunk in which one
// of them sees something); its 16 or 32 query rows are the tokens' G heads, and each row masks
// what is out of its own token's sight. The kernel is decode's ring
// (attention.cu): one CTA per SM walks the items, three (two, for 32 rows) loading warps fill as
// many slots, K and V halves apart, two groups of four warps compute. A row's chunk
// results go to the workspace where decode of its cut sequence would put them,
// record by record; attn_few_merge_kernel merges them in chunk order.
//
// Differences from decode: one score buffer a group instead of two (the next item's barrier
// comes before it is written again); p is split into bf16 hi and lo once, by the softmax, and
// read with ldmatrix (split by each warp as it reads: 381 us where this takes 357); no L2 policy, since a sequence's
// other tiles read the same chunks; and where V holds a value that is not finite out of
// some token's sight, p.V token by token with zeros there.
//
// 16 sequences of 5 drafts over 100 to 4000 tokens, window 1024, 32 heads over 8: 38 us for
// both kernels (the tiled kernel, one CTA a sequence and KV head: 70); 64 single tokens over 4000, 58 (260), and 92 where the
// call says that a sequence may have more than 16: its items and merges are laid out for 16 places then.
#include "attn_common.cuh"
#include "bi_internal.h"

namespace bi {
namespace {

constexpr int kConsumers = 8;                  // warps, in two groups
constexpr int NG = 2;
constexpr int kQStride = kRowBytes + 16;       // q rows 16 bytes apart more than they are long: no bank conflicts
constexpr int kSStride = kChunk + 8;           // scores of one row (padded)

// Shared memory and threads of the kernel for items of 16 MT rows: what fits, three slots or two.
template <int MT>
struct Shape {
    static constexpr int kSlots = MT == 1 ? 3 : 2;
    static constexpr int kThreads = 32 * (kConsumers + kSlots);
    static constexpr int kSlot = 4 * kHalfTile + (16 * MT * kQStride + 1023) / 1024 * 1024;   // K, V, q rows (the swizzle's 1024)
    static constexpr int kSFloats = 16 * MT * kSStride;
    static constexpr int kSmem = 1024 + kSlots * kSlot + NG * kSFloats * 4 + 2 * kSlots * (kChunk + 32) + (2 * NG + 2) * kSlots * 8 + 16;
    static constexpr int kTurn = kSlots % NG == 0 ? kSlots : kSlots * NG;   // items until a slot meets the same group again
    static_assert(kSmem <= 232448, "one CTA's shared memory");
};

struct FewParams {
    const uint16_t *Q;       // [total_q][Hq][D]
    const int32_t *cu_q;     // [B+1]
    const uint16_t *K;       // [blocks][bs][Hkv][D]
    const uint16_t *V;
    const int32_t *table;    // [B][max_blocks]
    const int32_t *lens;     // [B]
    float *ws;               // [places][Hq][chunks][kD + 2]
    uint16_t *O;             // [total_q][Hq][D]
    int64_t num_blocks, batch;
    int32_t total_q, max_blocks, Hq, Hkv, bs, chunks, max_len, max_q;
    int32_t few, tiles;      // the most new tokens of a sequence that is computed here, and its tiles
    int32_t places, by_seq;  // tokens that the workspace has room for: `few` of every sequence, or (by_seq 0) every row of Q
    int32_t window, sinks, box_rows;
    float scale;
    unsigned *status;
};

// Sequence b's new tokens, if they are computed here: their number (0 otherwise), first row, length of the whole.
__device__ __forceinline__ int sequence(const FewParams &p, int64_t b, int64_t &q0, int &L, bool &bad) {
    q0 = p.cu_q[b];
    const int64_t q1 = p.cu_q[b + 1], q = q1 - q0;
    L = p.lens[b];
    bad = q0 < 0 || q < 0 || q1 > p.total_q || q > p.max_q || L < q || L > p.max_len || L > static_cast<int64_t>(p.max_blocks) * p.bs;
    return !bad && q <= p.few ? static_cast<int>(q) : 0;
}

template <int G, int MT>
__global__ void __launch_bounds__(Shape<MT>::kThreads, 1)
attn_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const FewParams p) {
    constexpr int ROWS = 16 * MT, TQ = ROWS / G;           // query rows and tokens a tile
    constexpr int kSlots = Shape<MT>::kSlots, kSlot = Shape<MT>::kSlot, kTurn = Shape<MT>::kTurn, kSFloats = Shape<MT>::kSFloats;
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float *S0 = reinterpret_cast<float *>(smem + kSlots * kSlot);                 // [group][ROWS][kSStride] scores
    uint8_t *valid = reinterpret_cast<uint8_t *>(S0 + NG * kSFloats);             // [2][kSlots][kChunk]: row has K/V
    int *what = reinterpret_cast<int *>(valid + 2 * kSlots * kChunk);             // [2][kSlots][8]: the item (Item)
    // barriers and flag sets as in attn_split_kernel; the items are found by the loading warps alone, which hand them on with K
    uint64_t *full = reinterpret_cast<uint64_t *>(what + 2 * kSlots * 8);         // [kSlots][NG]: K, q
    uint64_t *fullV = full + kSlots * NG;                                         // [kSlots][NG]
    uint64_t *empty = fullV + kSlots * NG;                                        // [kSlots]: K, q
    uint64_t *emptyV = empty + kSlots;                                            // [kSlots]
    volatile int *abort_flag = reinterpret_cast<volatile int *>(emptyV + kSlots);
    __shared__ int most;                                   // chunks walked a tile
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < kSlots * NG; ++s) {
            mbar_init(&full[s], p.box_rows > 0 ? 32 : 64);
            mbar_init(&fullV[s], p.box_rows > 0 ? 32 : 64);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&empty[s], kConsumers / NG);
            mbar_init(&emptyV[s], kConsumers / NG);
        }
        *abort_flag = 0;
        most = 0;
        fence_mbar_init();
    }
    __syncthreads();
    for (int64_t b = tid; b < p.batch; b += Shape<MT>::kThreads) {
        int64_t q0;
        int L;
        bool bad;
        const int q = sequence(p, b, q0, L, bad);
        if (bad && blockIdx.x == 0) atomicOr(p.status, kDevBadOffsets);
        if (q > 0) atomicMax(&most, Seen(L - q + 1 - p.window, p.sinks).chunks(L));
    }
    __syncthreads();
    const int walk = most;
    const int64_t items = p.batch * p.tiles * p.Hkv * static_cast<int64_t>(walk);
    // item -> KV head (fastest), tile, chunk, sequence, stepped through without divisions
    struct Place {
        int g, u, c;
        int64_t b;
    };
    auto place = [&](int64_t it) {
        Place x;
        x.g = static_cast<int>(it % p.Hkv);
        it /= p.Hkv;
        x.u = static_cast<int>(it % p.tiles);
        it /= p.tiles;
        x.c = static_cast<int>(it % walk);
        x.b = it / walk;
        return x;
    };
    if (items == 0) return;
    Place now = place(blockIdx.x);
    const Place by = place(gridDim.x);
    struct Item {
        int t0, g, ntok, first_n;  // first token's row of Q (handed on: its place in the workspace), KV head, tokens (0: no more
                                   // items), what the first one would see without a window
        int j0, n, h0, h1;         // the chunk's first token and its tokens; [h0, h1) are out of the tile's sight
    };
    static_assert(sizeof(Item) == 32, "handed on in two 16-byte pieces");
    auto item = [&](Item &x, int64_t &b, int &at) {
        const int u = now.u, c = now.c;
        b = now.b;
        x.g = now.g;
        now.g += by.g;
        int carry = now.g >= p.Hkv;
        now.g -= carry ? p.Hkv : 0;
        now.u += by.u + carry;
        carry = now.u >= p.tiles;
        now.u -= carry ? p.tiles : 0;
        now.c += by.c + carry;
        carry = now.c >= walk;
        now.c -= carry ? walk : 0;
        now.b += by.b + carry;
        int64_t q0;
        int L;
        bool bad;
        const int q = sequence(p, b, q0, L, bad);
        if (u * TQ >= q) return false;
        x.t0 = static_cast<int>(q0) + u * TQ;
        at = static_cast<int>(p.by_seq ? b * p.few : q0) + u * TQ;
        x.ntok = min(TQ, q - u * TQ);
        x.first_n = L - q + u * TQ + 1;
        const int last_n = x.first_n + x.ntok - 1;
        const Seen w(x.first_n - p.window, p.sinks);
        if (c >= w.chunks(last_n)) return false;
        x.j0 = w.start(c);
        x.n = min(kChunk, last_n - x.j0);
        x.h0 = max(w.first - x.j0, 0);
        x.h1 = min(w.lo - x.j0, x.n);
        return true;
    };

    if (warp >= kConsumers) {
        // ---- loading warps: warp lw fills slot lw with items lw, lw + 3, ...
        const int lw = warp - kConsumers;
        if (lane == 0 && p.box_rows > 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        auto hand = [&](int k, const Item &x, int at) {
            int *w = what + (((k / kSlots) & 1) * kSlots + k % kSlots) * 8;
            st_shared_v4(smem_u32(w), at, x.g, x.ntok, x.first_n);
            st_shared_v4(smem_u32(w + 4), x.j0, x.n, x.h0, x.h1);
        };
        int k = 0, last = -1, lastV = -1;                  // this warp's last item whose K, V were issued
        bool gave_up = false;
        for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
            Item x;
            int64_t b;
            int at;
            if (!item(x, b, at)) continue;
            if (k % kSlots != lw) {
                ++k;
                continue;
            }
            // the chunk's rows: the block table first, it does not touch the slot
            int32_t row_blk[kChunk / 32], blk = -1;        // per-row copies: each row's block; boxes: lane i holds box i's
            uint32_t in = 0, wrong = 0;                    // bit i: row lane + 32 i is in the cache; a row in sight is not
            const bool box = p.box_rows > 0 && lane * p.box_rows < x.n && (lane * p.box_rows < x.h0 || (lane + 1) * p.box_rows > x.h1);
            if (box) blk = p.table[b * p.max_blocks + (x.j0 + lane * p.box_rows) / p.bs];
#pragma unroll
            for (int i = 0; i < kChunk / 32; ++i) {
                const int t = lane + 32 * i;
                const bool seen = t < x.n && !(t >= x.h0 && t < x.h1);
                int32_t r = -1;
                if (p.box_rows > 0)
                    r = __shfl_sync(0xffffffffu, blk, t / p.box_rows);
                else if (seen)
                    r = p.table[b * p.max_blocks + (x.j0 + t) / p.bs];
                const bool ok = seen && r >= 0 && r < p.num_blocks;
                row_blk[i] = ok ? r : -1;
                in |= static_cast<uint32_t>(ok) << i;
                wrong |= static_cast<uint32_t>(seen && !ok);
            }
            if (wrong) atomicOr(p.status, kDevBadOffsets);
            const int slot = k % kSlots;
            uint64_t *fb = &full[slot * NG + k % NG], *fbv = &fullV[slot * NG + k % NG];
            auto freed = [&](uint64_t *bar) {              // the half's last item is done with it
                if (k < kSlots || mbar_wait(bar, ((k / kSlots) - 1) & 1, abort_flag)) return true;
                if (lane == 0) {
                    atomicOr(p.status, kDevTimeout);
                    *abort_flag = 1;
                }
                gave_up = true;
                return false;
            };
            if (!freed(&empty[slot])) break;
            uint8_t *Ks = smem + slot * kSlot, *Vs = Ks + 2 * kHalfTile, *qs = Vs + 2 * kHalfTile;
            uint8_t *flags = valid + (((k / kSlots) & 1) * kSlots + slot) * kChunk;
#pragma unroll
            for (int i = 0; i < kChunk / 32; ++i) flags[lane + 32 * i] = (in >> i) & 1u;
            if (lane == 0) hand(k, x, at);
            auto q_row = [&](int r) { return p.Q + ((static_cast<int64_t>(x.t0) + r / G) * p.Hq + x.g * G + r % G) * kD; };
            const int rows = x.ntok * G;
            if (p.box_rows > 0) {
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, box)) * p.box_rows * kRowBytes;
                const int tok = (x.j0 + lane * p.box_rows) % p.bs;
                auto boxes = [&](uint8_t *dst, const CUtensorMap *tm, uint64_t *bar) {
                    if (box) {                             // a block outside the cache arrives as zeros
#pragma unroll
                        for (int half = 0; half < 2; ++half)
                            tma_load_4d(dst + half * kHalfTile + lane * p.box_rows * 128, tm, bar, half * 64, x.g, tok, blk);
                    }
                };
                __syncwarp();
                // each lane's arrival releases its shared-memory writes; lane 0 also sets the bytes to expect
                if (lane == 0)
                    mbar_arrive_expect_tx(fb, bytes + rows * kRowBytes);
                else
                    mbar_arrive(fb);
                __syncwarp();
                if (lane < rows) bulk_load(qs + lane * kQStride, q_row(lane), kRowBytes, fb);
                boxes(Ks, &tmK, fb);
                last = k;
                if (!freed(&emptyV[slot])) break;
                if (lane == 0)
                    mbar_arrive_expect_tx(fbv, bytes);
                else
                    mbar_arrive(fbv);
                __syncwarp();
                boxes(Vs, &tmV, fbv);
            } else {
                // 16-byte copies, two rows an instruction; a lane arrives now, and once its copies have landed
                auto copy = [&](uint8_t *dst, const uint16_t *src, uint64_t *bar) {
#pragma unroll
                    for (int i = 0; i < kChunk / 32; ++i)
#pragma unroll 1
                        for (int y = 0; y < 16; ++y) {
                            const int t = 32 * i + 2 * y + (lane >> 4), piece = lane & 15;
                            const int64_t o = __shfl_sync(0xffffffffu, row_blk[i], t & 31);
                            cp_async_16(smem_u32(dst) + kv_piece(t, piece),
                                        o >= 0 ? src + ((o * p.bs + (x.j0 + t) % p.bs) * p.Hkv + x.g) * kD + piece * 8 : src,
                                        o >= 0 ? 16u : 0u);
                        }
                    mbar_arrive(bar);
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
                };
                for (int y = lane; y < rows * 16; y += 32)
                    cp_async_16(smem_u32(qs) + (y >> 4) * kQStride + (y & 15) * 16, q_row(y >> 4) + (y & 15) * 8, 16u);
                copy(Ks, p.K, fb);
                last = k;
                if (!freed(&emptyV[slot])) break;
                copy(Vs, p.V, fbv);
            }
            lastV = k;
            ++k;
        }
        // the copies of this warp's last item must land before the CTA exits (K's wait comes first: the item below
        // may be counted on the same barrier)
        if (last >= 0) mbar_wait(&full[(last % kSlots) * NG + last % NG], (last / kTurn) & 1, nullptr);
        // one more item says that there are none: the group that comes to this slot next stops (the wait is that of any item)
        if (!gave_up) {
            while (k % kSlots != lw) ++k;
            const int slot = k % kSlots;
            uint64_t *fb = &full[slot * NG + k % NG];
            if (k < kSlots || mbar_wait(&empty[slot], ((k / kSlots) - 1) & 1, abort_flag)) {
                if (lane == 0) hand(k, Item{}, 0);
                __syncwarp();
                mbar_arrive(fb);
                if (p.box_rows == 0) mbar_arrive(fb);
            } else if (lane == 0) {
                atomicOr(p.status, kDevTimeout);
                *abort_flag = 1;
            }
        }
        if (lastV >= 0) mbar_wait(&fullV[(lastV % kSlots) * NG + lastV % NG], (lastV / kTurn) & 1, nullptr);
        return;
    }

    // ---- consumer warps: group grp computes the items k with k % NG == grp
    constexpr int GW = kConsumers / NG;                    // warps per group
    constexpr int NT = kChunk / 8 / GW;                    // score n-tiles per warp
    constexpr int DW = kD / GW;                            // value dimensions per warp
    const int grp = warp / GW, gw = warp % GW;
    const int gq = lane >> 2, cq = lane & 3;               // fragment rows gq and gq + 8, column pair
    float *S = S0 + grp * kSFloats;
    for (int k = grp;; k += NG) {
        const int slot = k % kSlots;
        auto stop = [&](bool ok) {                         // a wait ran out: the group's warps stop together
            if (!group_sync_or<GW>(grp, !ok)) return false;
            if (gw == 0 && lane == 0) {
                atomicOr(p.status, kDevTimeout);
                *abort_flag = 1;
            }
            return true;
        };
        if (stop(mbar_wait(&full[slot * NG + grp], (k / kTurn) & 1, abort_flag))) break;
        const uint8_t *Ks = smem + slot * kSlot, *Vs = Ks + 2 * kHalfTile, *qb = Vs + 2 * kHalfTile;
        const uint8_t *vrow = valid + (((k / kSlots) & 1) * kSlots + slot) * kChunk;
        const int4 *w = reinterpret_cast<const int4 *>(what + (((k / kSlots) & 1) * kSlots + slot) * 8);
        const int4 x0 = w[0], x1 = w[1];
        const Item x{x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
        if (x.ntok == 0) break;                            // no more items: the whole group
        const int rows = x.ntok * G, s0 = p.sinks - x.j0;
        // what row r sees of the chunk: t < end, and t < s0 or t >= end - window
        auto end_of = [&](int r) { return x.first_n + r / G - x.j0; };
        auto sees = [&](int end, int t) { return t < end && (t < s0 || t >= end - p.window); };
        // where row r's results go: the record that decode of its cut sequence has for this chunk, null if it sees nothing of it
        auto record = [&](int r) -> float * {
            const int n = x.first_n + r / G, c = x.j0 / kChunk;
            const Seen w(n - p.window, p.sinks);
            if (r >= rows || x.j0 >= n || (c >= w.ns && c < w.c0)) return nullptr;
            const int64_t i = c < w.ns ? c : c - w.c0 + w.ns;
            if (!BI_IN_BOUNDS(x.t0 + r / G < p.places && i < p.chunks, p.status)) return nullptr;
            return p.ws + (((static_cast<int64_t>(x.t0) + r / G) * p.Hq + x.g * G + r % G) * p.chunks + i) * (kD + 2);
        };

        // masked for some token of the tile; or whole for all, with every row in the cache
        const int last_n = x.first_n + x.ntok - 1;
        const bool masked = x.j0 + kChunk > x.first_n || (x.j0 < last_n - p.window && x.j0 + kChunk > p.sinks);
        const bool whole = __all_sync(0xffffffffu, reinterpret_cast<const uint32_t *>(vrow)[lane] == 0x01010101u) && !masked;

        // scores of the rows: warp gw takes tokens 8 NT gw .. 8 NT gw + 8 NT - 1, K ascending in 16-dimension steps
        {
            float acc[MT][NT][4] = {};
            uint32_t qa[MT][kD / 16][4];                   // rows gq, gq + 8; dimensions + 0, + 8
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int ks = 0; ks < kD / 16; ++ks) {
                    uint32_t(&a)[4] = qa[mt][ks];
                    ldmatrix_x4(a[0], a[1], a[2], a[3], smem_u32(qb + (16 * mt + (lane & 15)) * kQStride + 32 * ks + 16 * (lane >> 4)));
                }
#pragma unroll
            for (int kp = 0; kp < kD / 32; ++kp) {         // two 16-dimension steps per ldmatrix
                uint32_t bf[NT][4];
#pragma unroll
                for (int nb = 0; nb < NT; ++nb) {
                    const int t = gw * 8 * NT + nb * 8 + (lane & 7);
                    ldmatrix_x4(bf[nb][0], bf[nb][1], bf[nb][2], bf[nb][3], smem_u32(Ks + kv_piece(t, 4 * kp + (lane >> 3))));
                }
#pragma unroll
                for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const uint32_t(&a)[4] = qa[mt][2 * kp + k2];
#pragma unroll
                        for (int nb = 0; nb < NT; ++nb) mma_16816(acc[mt][nb], a[0], a[1], a[2], a[3], bf[nb][2 * k2], bf[nb][2 * k2 + 1]);
                    }
            }
            float *Sw = S + gq * kSStride + gw * 8 * NT + 2 * cq;
            if (whole) {                                   // (rows that do not exist are written too, and not read)
#pragma unroll
                for (int h = 0; h < 2 * MT; ++h)
#pragma unroll
                    for (int nb = 0; nb < NT; ++nb) {
                        const float *v = acc[h >> 1][nb] + 2 * (h & 1);
                        *reinterpret_cast<float2 *>(Sw + 8 * h * kSStride + 8 * nb) = make_float2(__fmul_rn(v[0], p.scale), __fmul_rn(v[1], p.scale));
                    }
            } else {
#pragma unroll
                for (int h = 0; h < 2 * MT; ++h) {
                    const int end = end_of(gq + 8 * h);
#pragma unroll
                    for (int nb = 0; nb < NT; ++nb)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int t = gw * 8 * NT + nb * 8 + 2 * cq + e;
                            Sw[8 * h * kSStride + 8 * nb + e] =
                                sees(end, t) && vrow[t] ? __fmul_rn(acc[h >> 1][nb][2 * (h & 1) + e], p.scale) : -INFINITY;
                        }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);          // this warp is done with K and q
        group_sync<GW>(grp);

        // per row: max, exponentials, sum (row r on warp r % GW; a warp's rows side by side, for their latencies); (m, l) to
        // the workspace. Rows that do not exist compute something that nothing reads.
        auto softmax = [&](auto count) {
            constexpr int R = decltype(count)::value;
            float sc[R][kChunk / 32], m[R], l[R];
#pragma unroll
            for (int y = 0; y < R; ++y) {
                m[y] = -INFINITY;
#pragma unroll
                for (int i = 0; i < kChunk / 32; ++i) {
                    sc[y][i] = S[(gw + GW * y) * kSStride + lane + 32 * i];
                    m[y] = fmaxf(m[y], sc[y][i]);
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int y = 0; y < R; ++y) m[y] = fmaxf(m[y], __shfl_xor_sync(0xffffffffu, m[y], o));
#pragma unroll
            for (int y = 0; y < R; ++y) {
                const int r = gw + GW * y;
                __syncwarp();                              // the row has been read
                if (m[y] == -INFINITY) {                   // does it see any token of the chunk in the cache?
                    bool any = false;
#pragma unroll
                    for (int i = 0; i < kChunk / 32; ++i) any |= sees(end_of(r), lane + 32 * i) && vrow[lane + 32 * i];
                    if (!__any_sync(0xffffffffu, any)) m[y] = kNoScore;
                }
                l[y] = 0.0f;
#pragma unroll
                for (int i = 0; i < kChunk / 32; ++i) {    // (-inf, and p = 0, for what it does not see)
                    sc[y][i] = expf(sc[y][i] - m[y]);
                    l[y] += sc[y][i];
                }
                // p takes the row's place as bf16, 128 hi and then 128 lo (see probability)
#pragma unroll
                for (int i = 0; i < kChunk / 32; i += 2) {
                    uint32_t hi, lo;
                    split_bf16x2(sc[y][i], sc[y][i + 1], hi, lo);
                    uint16_t *at = reinterpret_cast<uint16_t *>(S + r * kSStride) + (lane ^ (2 * r & 8));
                    at[32 * i] = static_cast<uint16_t>(hi);
                    at[32 * i + 32] = static_cast<uint16_t>(hi >> 16);
                    at[32 * i + kChunk] = static_cast<uint16_t>(lo);
                    at[32 * i + kChunk + 32] = static_cast<uint16_t>(lo >> 16);
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int y = 0; y < R; ++y) l[y] += __shfl_xor_sync(0xffffffffu, l[y], o);
            float ml = m[0], ll = l[0];                    // lane y stores row y's
#pragma unroll
            for (int y = 1; y < R; ++y) {
                ml = lane == y ? m[y] : ml;
                ll = lane == y ? l[y] : ll;
            }
            if (lane < R) {
                float *rec = record(gw + GW * lane);
                if (rec) *reinterpret_cast<float2 *>(rec) = make_float2(ml, ll);
            }
        };
        if (rows <= GW)
            softmax(std::integral_constant<int, 1>{});
        else if (rows <= 16)
            softmax(std::integral_constant<int, 16 / GW>{});
        else if (rows <= 24)
            softmax(std::integral_constant<int, MT == 1 ? 16 / GW : 24 / GW>{});
        else
            softmax(std::integral_constant<int, ROWS / GW>{});
        const bool ok_v = mbar_wait(&fullV[slot * NG + grp], (k / kTurn) & 1, abort_flag);
        // rows behind the last token's and rows out of the tile's sight, whether they came with a box or not: p = 0 has to
        // meet finite values
        if (p.box_rows > 0 && (x.n < kChunk || x.h1 > x.h0)) {
            for (int i = gw * 32 + lane; i < kChunk * (kRowBytes / 16); i += 32 * GW) {
                const int t = i / (kRowBytes / 16);
                if (t >= x.n || (t >= x.h0 && t < x.h1)) st_shared_v4(smem_u32(Vs) + kv_piece(t, i % (kRowBytes / 16)), 0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();                      // before later bulk copies into these rows
        }
        if (stop(ok_v)) break;

        // values: warp gw takes dimensions DW gw .. DW gw + DW - 1, tokens ascending in 16-token steps, hi before lo
        // p of rows 16 mt .. and tokens 16 ks .. (+ kChunk: lo). A row's 16-byte pieces are swapped in pairs in every other
        // four rows, so that eight rows' pieces lie in different banks. (The buffer is written again after the next item's
        // barrier; rows that do not exist hold anything.)
        auto probability = [&](int mt, int at, uint32_t (&a)[4]) {
            const int r = 16 * mt + (lane & 15);
            ldmatrix_x4(a[0], a[1], a[2], a[3], smem_u32(reinterpret_cast<const uint16_t *>(S + r * kSStride) + ((at + 8 * (lane >> 4)) ^ (2 * r & 8))));
        };
        const int d0 = gw * DW, mi = lane >> 3, mr = lane & 7;   // ldmatrix: matrix, row
        auto fetch = [&](int ks, uint32_t (&v)[DW / 16][4]) {
#pragma unroll
            for (int hf = 0; hf < DW / 16; ++hf)           // 16 dimensions per ldmatrix
                ldmatrix_x4_trans(v[hf][0], v[hf][1], v[hf][2], v[hf][3],
                                  smem_u32(Vs + kv_piece(ks * 16 + (mi & 1) * 8 + mr, ((d0 + 16 * hf) >> 3) + (mi >> 1))));
        };
        auto products = [&](float (&acc)[MT][DW / 8][4], auto by_token, int end) {
#pragma unroll
            for (int ks = 0; ks < kChunk / 16; ++ks) {
                uint32_t v[DW / 16][4];
                fetch(ks, v);
                if (decltype(by_token)::value) {           // zeros for what the token does not see
                    uint32_t keep[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int t = ks * 16 + 8 * h + 2 * cq;
                        keep[h] = (sees(end, t) ? 0xFFFFu : 0u) | (sees(end, t + 1) ? 0xFFFF0000u : 0u);
                    }
#pragma unroll
                    for (int hf = 0; hf < DW / 16; ++hf)
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[hf][i] &= keep[i & 1];
                }
                uint32_t ph[MT][4], pl[MT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    probability(mt, 16 * ks, ph[mt]);
                    probability(mt, 16 * ks + kChunk, pl[mt]);
                }
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const uint32_t(&a)[4] = part == 0 ? ph[mt] : pl[mt];
#pragma unroll
                        for (int hf = 0; hf < DW / 16; ++hf) {
                            mma_16816(acc[mt][2 * hf], a[0], a[1], a[2], a[3], v[hf][0], v[hf][1]);
                            mma_16816(acc[mt][2 * hf + 1], a[0], a[1], a[2], a[3], v[hf][2], v[hf][3]);
                        }
                    }
            }
        };
        // in a chunk that is masked for some of several tokens: a value that is not finite among this warp's dimensions?
        bool odd = false;
        if (x.ntok > 1 && masked) {
            bool fine = true;
#pragma unroll
            for (int ks = 0; ks < kChunk / 16; ++ks) {
                uint32_t v[DW / 16][4];
                fetch(ks, v);
#pragma unroll
                for (int hf = 0; hf < DW / 16; ++hf)
#pragma unroll
                    for (int i = 0; i < 4; ++i) fine = fine && finite_pair(v[hf][i]);
            }
            odd = __any_sync(0xffffffffu, !fine);
        }
        float acc[MT][DW / 8][4] = {};
        if (!odd) {
            products(acc, std::false_type{}, 0);
        } else {
#pragma unroll 1
            for (int u = 0; u < x.ntok; ++u) {
                float one[MT][DW / 8][4] = {};
                products(one, std::true_type{}, end_of(u * G));
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int nb = 0; nb < DW / 8; ++nb)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if ((16 * mt + gq + 8 * (e >> 1)) / G == u) acc[mt][nb][e] = one[mt][nb][e];
            }
        }
#pragma unroll
        for (int h = 0; h < 2 * MT; ++h) {
            float *rec = record(gq + 8 * h);
            if (!rec) continue;
            rec += 2 + d0 + 2 * cq;
#pragma unroll
            for (int nb = 0; nb < DW / 8; ++nb)
                *reinterpret_cast<float2 *>(rec + nb * 8) = make_float2(acc[h >> 1][nb][2 * (h & 1)], acc[h >> 1][nb][2 * (h & 1) + 1]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&emptyV[slot]);         // this warp is done with V
    }
}

// One CTA per (sequence, `per` new tokens, query head). BY_SEQ: p.by_seq (looked at here, 37.1 us for both kernels of 16 x 5
// tokens; now 36.5).
template <bool BY_SEQ>
__global__ void __launch_bounds__(kD)
attn_few_merge_kernel(const FewParams p, const int per) {
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    __shared__ MergeTile tile;
    const unsigned groups = (min(p.few, p.max_q) + per - 1) / per;
    const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.Hq));
    const unsigned r = blockIdx.x / static_cast<unsigned>(p.Hq);
    const int64_t b = r / groups;
    const int i0 = static_cast<int>(r % groups) * per, d = threadIdx.x;
    int64_t q0;
    int L;
    bool bad;
    const int q = sequence(p, b, q0, L, bad);
    for (int i = i0; i < min(q, i0 + per); ++i) {
        const int n = L - q + i + 1, nc = Seen(n - p.window, p.sinks).chunks(n);
        if (!BI_IN_BOUNDS(nc <= p.chunks, p.status)) return;
        const float *w = p.ws + (((BY_SEQ ? b * p.few : q0) + i) * p.Hq + h) * p.chunks * (kD + 2);
        float ov[kMergeTile];
        const int nt = min(kMergeTile, nc);
#pragma unroll
        for (int c = 0; c < kMergeTile; ++c) ov[c] = c < nt ? w[static_cast<int64_t>(c) * (kD + 2) + 2 + d] : 0.0f;
        const float mc = d < nt ? w[static_cast<int64_t>(d) * (kD + 2)] : -INFINITY;
        const float lc = d < nt ? w[static_cast<int64_t>(d) * (kD + 2) + 1] : 0.0f;
        p.O[((q0 + i) * p.Hq + h) * kD + d] = merge_records(w, nc, ov, mc, lc, tile);
    }
}

template <int G, int MT>
bi_status launch_mt(const CUtensorMap &tmK, const CUtensorMap &tmV, const FewParams &p, int sms, cudaStream_t s) {
    static unsigned long long configured = 0;
    constexpr int smem = Shape<MT>::kSmem;
    if (ensure_smem_attr(reinterpret_cast<const void *>(attn_few_kernel<G, MT>), smem, &configured) != BI_OK) return BI_ERR_CUDA;
    return launch_pdl(attn_few_kernel<G, MT>, dim3(static_cast<unsigned>(sms)), dim3(Shape<MT>::kThreads), smem, s, tmK, tmV, p);
}
// Items of 32 rows read a chunk half as often, for the fewer slots, where the longest sequence's tiles of 16 pair up and
// either there are many of them or the loading warps' copies by row are what takes the time. Tiles of 16, of 32 rows, in us for
// both kernels: 64 x 5 tokens, window 4096, 32 heads over 8: 357, 320; 32 x 5, window 2048: 158, 135; 16 x 5, window 4096
// (55 items an SM): 106, 101; 16 x 8, window 1024 (15 an SM): 51.7, 55.8; 64 x 12 (three tiles): 635, 727; copied
// by row, 16 x 5, window 1024: 140, 105.
template <int G>
bi_status launch_g(const CUtensorMap &tmK, const CUtensorMap &tmV, FewParams p, int most, int sms, cudaStream_t s) {
    p.tiles = (most + 16 / G - 1) / (16 / G);
    const double items = static_cast<double>(p.batch) * p.tiles * p.Hkv * p.chunks;
    if (p.tiles % 2 == 0 && (p.box_rows == 0 || items > 40.0 * sms)) {
        p.tiles /= 2;
        return launch_mt<G, 2>(tmK, tmV, p, sms, s);
    }
    return launch_mt<G, 1>(tmK, tmV, p, sms, s);
}

}  // namespace

bi_status launch_attention_few_window(const WindowCall &a, const FewPlan &plan, void *workspace, cudaStream_t s) {
    int dev = 0;
    const DeviceInfo *info = nullptr;
    bi_status st = current_device(&dev, &info);
    if (st != BI_OK) return st;
    const int G = a.Hq / a.Hkv, most = plan.few < a.max_q ? plan.few : a.max_q;
    FewParams p{};
    p.Q = static_cast<const uint16_t *>(a.Q);
    p.cu_q = a.cu_q;
    p.K = static_cast<const uint16_t *>(a.K);
    p.V = static_cast<const uint16_t *>(a.V);
    p.table = a.table;
    p.lens = a.lens;
    p.ws = static_cast<float *>(workspace);
    p.O = static_cast<uint16_t *>(a.O);
    p.num_blocks = a.num_blocks;
    p.batch = a.B;
    p.total_q = a.total_q;
    p.max_blocks = a.max_blocks;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.bs = a.bs;
    p.chunks = static_cast<int32_t>(seen_chunks(a.max_len, a.window, a.sinks));
    p.max_len = a.max_len;
    p.max_q = a.max_q;
    p.few = plan.few;
    p.places = static_cast<int32_t>(plan.places);
    p.by_seq = plan.places < a.total_q;
    p.window = a.window;
    p.sinks = a.sinks;
    p.scale = a.scale;
    p.status = device_status_word();
    CUtensorMap tmK{}, tmV{};
    p.box_rows = kv_box_maps(a.K, a.V, a.num_blocks, a.bs, a.Hkv, &tmK, &tmV);
    switch (G) {
        case 1: st = launch_g<1>(tmK, tmV, p, most, info->sm_count, s); break;
        case 2: st = launch_g<2>(tmK, tmV, p, most, info->sm_count, s); break;
        case 4: st = launch_g<4>(tmK, tmV, p, most, info->sm_count, s); break;
        case 8: st = launch_g<8>(tmK, tmV, p, most, info->sm_count, s); break;
        default: return BI_ERR_UNSUPPORTED;
    }
    if (st != BI_OK) return st;
    // Where single tokens stand among longer sequences, most of the places for tokens are empty: then a CTA takes four
    // (64 sequences, 16 places each, 32 heads).
    const int per = a.B * most * a.Hq > 64ll * info->sm_count ? 4 : 1;
    return launch_pdl(p.by_seq ? attn_few_merge_kernel<true> : attn_few_merge_kernel<false>, dim3(static_cast<unsigned>(a.B * ((most + per - 1) / per) * a.Hq)), dim3(kD), 0, s, p, per);
}

}  // namespace bi
