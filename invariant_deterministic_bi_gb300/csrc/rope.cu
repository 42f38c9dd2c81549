// rope.cu -- what stands between the qkv projection and the attention: rotary
// positions, RMSNorm of query and key heads, and the append to the paged bf16
// cache, in one pass over the heads' rows.
//
// A row is one head of one token, D dimensions. Its norm (queries and keys,
// where weights are given) is x / sqrt(mean x^2 + eps) * w; its rotation turns
// the pair (a, b) of frequency f_i, i < R/2, at position p by the angle p f_i:
//   (m (a cos - b sin), m (b cos + a sin)),
// the pair being dimensions (i, i + R/2), or (2i, 2i+1) interleaved; dimensions
// from R on stay. fp32 throughout, one rounding to bf16 at the end.
//
// Angles: a frequency is held in turns per position as a 64-bit fraction, so
// p f_i modulo one turn is the low 64 bits of an integer product: exact but for
// the frequency itself, which is a double's (2^-56 turns a position for f = 1), at any
// position, with no table of positions and no argument reduction. sincospif takes the top 32
// bits as a signed number of half turns.
//
// Layout: LANES lanes hold a row, 16 dimensions each as two 16-byte vectors half the
// turned (or the unturned) part apart, so that a load or store of a warp covers
// whole lines. In both layouts of the pairs the two vectors hold eight whole pairs, so
// a pair never leaves its lane, and a lane needs the same frequencies for every
// row. The 32 / LANES rows of a warp are heads of one token: each computes a share
// of the token's sines and cosines, and shuffles pass them round.
//
// Bytes bound it where there are many tokens: 8155 tokens of 32 heads turned 19.2 us
// (7.0 TB/s), 40 heads normed and turned 27.5 (6.1), 8 + 8 heads into the cache 8.0, with
// 32 queries and norms 32.3 (6.2), of which some stays in L2. 64 tokens take 2.0 to 2.6 us: launch, one load, one store.
#include "attn_common.cuh"
#include "bi_internal.h"
#include "bi_ptx.cuh"

namespace bi {
namespace {

// Blocks are small, so that a finished one makes room soon: 8155 tokens, 40 normed heads, 128 threads 27.5 us, 256 threads 31.3.
constexpr int kThreads = 128;
constexpr int kDepth = 4;    // groups of heads a warp has on the way (2: 29.8 us, 3: 28.1, 6: 28.6; in registers, one ahead: 34.9)

constexpr f2 kMinus2 = 0x8000000080000000ull;          // (xor: both negated)

// A lane's two vectors of a row: the eight pairs (a_k, b_k) as packed a and b (interleaved, a vector holds four of them).
template <bool INTER>
__device__ __forceinline__ void unpack(const uint4 &v0, const uint4 &v1, f2 (&a)[4], f2 (&b)[4]) {
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (INTER) {
            a[k] = f2_of(w[2 * k] << 16, w[2 * k + 1] << 16);
            b[k] = f2_of(w[2 * k] & 0xFFFF0000u, w[2 * k + 1] & 0xFFFF0000u);
        } else {
            a[k] = f2_of(w[k] << 16, w[k] & 0xFFFF0000u);
            b[k] = f2_of(w[4 + k] << 16, w[4 + k] & 0xFFFF0000u);
        }
    }
}
template <bool INTER>
__device__ __forceinline__ void pack(const f2 (&a)[4], const f2 (&b)[4], uint4 &v0, uint4 &v1) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (INTER) {
            w[2 * k] = pack_bf16x2(lo_of(a[k]), lo_of(b[k]));
            w[2 * k + 1] = pack_bf16x2(hi_of(a[k]), hi_of(b[k]));
        } else {
            w[k] = pack_bf16x2(lo_of(a[k]), hi_of(a[k]));
            w[4 + k] = pack_bf16x2(lo_of(b[k]), hi_of(b[k]));
        }
    }
    v0 = make_uint4(w[0], w[1], w[2], w[3]);
    v1 = make_uint4(w[4], w[5], w[6], w[7]);
}

// Warp: token t and the groups of 32 / LANES heads s, s + splits, ... of its queries, keys and values.
template <int LANES, bool INTER, bool NORM>
__global__ void __launch_bounds__(kThreads, NORM ? 5 : 8)
heads_kernel(const HeadsParams p) {
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    constexpr int ROWS = 32 / LANES, SHARE = 8 / ROWS;     // heads a warp takes at once; frequencies a lane computes
    const int lane = threadIdx.x & 31, u = lane % LANES, r = lane / LANES;
    const int64_t w = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = p.splits == 1 ? w : w / p.splits;
    if (t >= p.T) return;
    const int first = static_cast<int>(w - t * p.splits);
    const bool holds = 16 * u < p.D, turns = 16 * u < p.R;
    // this lane's two vectors of a row
    const int v0 = turns ? 8 * u : p.R / 2 + 8 * u;
    const int v1 = v0 + (turns ? p.R / 2 : (p.D - p.R) / 2);
    const bool mine = holds && BI_IN_BOUNDS(v1 + 8 <= p.D, p.status);
    const int step = p.splits * ROWS;                      // heads between two of this warp's groups

    // Loads run DEPTH groups ahead, over the parts' ends; each lane copies its own vectors and reads them back, so the
    // warps never meet. lpart, lhead: the group that is loaded next.
    __shared__ uint4 ring[kThreads / 32][kDepth][2][32];
    uint4 (&mem)[kDepth][2][32] = ring[threadIdx.x >> 5];
    int lpart = 0, lhead = first * ROWS, lslot = 0;
    auto load_next = [&] {
        while (lpart < 3 && lhead >= p.part[lpart].heads) {
            lhead -= (p.part[lpart].heads + ROWS - 1) / ROWS * ROWS;   // (>= 0: a part's last group may be short)
            ++lpart;
        }
        if (lpart < 3) {
            const Heads &h = p.part[lpart];
            if (lhead + r < h.heads && mine) {
                const uint16_t *src = h.src + t * h.lds + static_cast<int64_t>(lhead + r) * p.D;
                cp_async_16(smem_u32(&mem[lslot][0][lane]), src + v0, 16u);
                cp_async_16(smem_u32(&mem[lslot][1][lane]), src + v1, 16u);
            }
            lhead += step;
        }
        cp_async_commit();
        lslot = lslot + 1 == kDepth ? 0 : lslot + 1;
    };
#pragma unroll
    for (int k = 0; k < kDepth; ++k) load_next();
    int64_t pos = 0, slot = 0;
    if (p.R > 0) pos = p.pos[t];
    if (p.slots) slot = p.slots[t];
    uint64_t f[SHARE];
#pragma unroll
    for (int k = 0; k < SHARE; ++k) {
        const int n = r * SHARE + k;                       // pair n of lane u
        f[k] = turns ? p.turns[!INTER ? 8 * u + n : n < 4 ? 4 * u + n : p.R / 4 + 4 * u + n - 4] : 0;
    }
    if (pos != static_cast<int32_t>(pos)) {                // the whole warp: one token
        if (lane == 0) atomicOr(p.status, kDevBadOffsets);
        cp_async_wait<0>();
        return;
    }
    const bool kept = slot >= 0 && slot < p.cache_rows;    // (without a cache: slot 0 of 1)
    if (!kept && slot != -1 && lane == 0) atomicOr(p.status, kDevBadOffsets);

    float cs[SHARE], sn[SHARE];
#pragma unroll
    for (int k = 0; k < SHARE; ++k) {
        const uint64_t phase = static_cast<uint64_t>(pos) * f[k];
        sincospif(__int2float_rn(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &sn[k], &cs[k]);
        cs[k] = __fmul_rn(cs[k], p.factor);
        sn[k] = __fmul_rn(sn[k], p.factor);
    }
    // sines and cosines of this lane's eight pairs, from the lanes that computed them
    auto share = [&](f2 (&c)[4], f2 (&s)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[i] = __shfl_sync(0xffffffffu, cs[(2 * k + i) % SHARE], (2 * k + i) / SHARE * LANES + u);
                v[2 + i] = __shfl_sync(0xffffffffu, sn[(2 * k + i) % SHARE], (2 * k + i) / SHARE * LANES + u);
            }
            c[k] = f2_of(v[0], v[1]);
            s[k] = f2_of(v[2], v[3]);
        }
    };
    // The groups of one part, in turn; `change` computes a group's two vectors from the loaded ones.
    int head = first * ROWS, cslot = 0;
    auto walk = [&](const Heads &h, bool cache, auto &&change) {
        uint16_t *dst = h.dst + (cache ? slot : t) * h.ldd + static_cast<int64_t>(head + r) * p.D;
        for (; head < h.heads; head += step) {
            cp_async_wait<kDepth - 1>();
            uint4 a = mem[cslot][0][lane], b = mem[cslot][1][lane];
            if (!mine) a = b = make_uint4(0u, 0u, 0u, 0u);     // (the norm sums over the row's lanes)
            change(a, b);
            if (head + r < h.heads && mine && (kept || !cache)) {
                *reinterpret_cast<uint4 *>(dst + v0) = a;
                *reinterpret_cast<uint4 *>(dst + v1) = b;
            }
            dst += static_cast<int64_t>(step) * p.D;
            load_next();                                   // into the slot just read
            cslot = cslot + 1 == kDepth ? 0 : cslot + 1;
        }
        head -= (h.heads + ROWS - 1) / ROWS * ROWS;
    };
    auto turned = [&](const Heads &h, bool cache) {
        if (h.heads == 0) return;
        f2 c[4], s[4];
        if (p.R > 0) share(c, s);
        if (NORM && h.w) {
            // rotation and weights in one: (a wa) c - (b wb) s = a (wa c) + b (-wb s), likewise for b
            f2 wa[4], wb[4], ac[4], as[4], bc[4], bs[4];
            uint4 x0 = make_uint4(0u, 0u, 0u, 0u), x1 = x0;
            if (mine) {
                x0 = *reinterpret_cast<const uint4 *>(h.w + v0);
                x1 = *reinterpret_cast<const uint4 *>(h.w + v1);
            }
            unpack<INTER>(x0, x1, wa, wb);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                ac[k] = turns ? mul2(wa[k], c[k]) : wa[k];
                bc[k] = turns ? mul2(wb[k], c[k]) : wb[k];
                if (turns) {
                    as[k] = mul2(wa[k], s[k]);
                    bs[k] = mul2(wb[k], s[k]) ^ kMinus2;
                }
            }
            walk(h, cache, [&](uint4 &x, uint4 &y) {
                f2 a[4], b[4], q = 0;
                unpack<INTER>(x, y, a, b);
#pragma unroll
                for (int k = 0; k < 4; ++k) q = fma2(b[k], b[k], fma2(a[k], a[k], q));
                float ss = __fadd_rn(__uint_as_float(lo_of(q)), __uint_as_float(hi_of(q)));
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
                const float rs = rsqrtf(__fmaf_rn(ss, p.inv_d, p.eps));
                const f2 rr = f2_of(rs, rs);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f2 xa = mul2(a[k], rr), xb = mul2(b[k], rr);
                    if (turns) {
                        a[k] = fma2(xa, ac[k], mul2(xb, bs[k]));
                        b[k] = fma2(xb, bc[k], mul2(xa, as[k]));
                    } else {
                        a[k] = mul2(xa, ac[k]);
                        b[k] = mul2(xb, bc[k]);
                    }
                }
                pack<INTER>(a, b, x, y);
            });
        } else if (p.R > 0) {
            walk(h, cache, [&](uint4 &x, uint4 &y) {
                if (!turns) return;                        // these dimensions stay, whatever they hold
                f2 a[4], b[4];
                unpack<INTER>(x, y, a, b);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f2 xa = a[k], xb = b[k];
                    a[k] = fma2(xa, c[k], mul2(xb, s[k]) ^ kMinus2);
                    b[k] = fma2(xb, c[k], mul2(xa, s[k]));
                }
                pack<INTER>(a, b, x, y);
            });
        } else {
            walk(h, cache, [](uint4 &, uint4 &) {});
        }
    };
    turned(p.part[0], false);
    turned(p.part[1], p.part[1].cache);
    if (p.part[2].heads > 0) walk(p.part[2], true, [](uint4 &, uint4 &) {});
}

template <int LANES>
bi_status launch_lanes(HeadsParams p, bool inter, int sms, cudaStream_t s) {
    constexpr int ROWS = 32 / LANES;
    int64_t g = 0;
    for (int i = 0; i < 3; ++i) g += (p.part[i].heads + ROWS - 1) / ROWS;
    // warps a token: as many as give every SM 16, and at most one a group (a token's sines and cosines are computed once
    // a warp: twice as many warps at 4096 tokens, 40 normed heads, 15.1 us against 13.4)
    const int64_t want = (16 * static_cast<int64_t>(sms) + p.T - 1) / p.T;
    p.splits = static_cast<int32_t>(want < 1 ? 1 : want > g ? g : want);
    const int64_t blocks = (p.T * p.splits + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffff) return BI_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(blocks));
    const bool norm = p.part[0].w || p.part[1].w;
    return launch_pdl(inter ? (norm ? heads_kernel<LANES, true, true> : heads_kernel<LANES, true, false>)
                            : (norm ? heads_kernel<LANES, false, true> : heads_kernel<LANES, false, false>),
                      grid, dim3(kThreads), 0, s, p);
}

}  // namespace

bi_status launch_heads(HeadsParams p, bool inter, cudaStream_t s) {
    int dev = 0;
    const DeviceInfo *info = nullptr;
    const bi_status st = current_device(&dev, &info);
    if (st != BI_OK) return st;
    p.status = device_status_word();
    if (p.D <= 64) return launch_lanes<4>(p, inter, info->sm_count, s);
    if (p.D <= 128) return launch_lanes<8>(p, inter, info->sm_count, s);
    return launch_lanes<16>(p, inter, info->sm_count, s);
}

}  // namespace bi
