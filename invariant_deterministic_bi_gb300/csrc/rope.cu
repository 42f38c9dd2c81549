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
// the frequency's own rounding (2^-65 turns a position), at any position, with
// no table of positions and no argument reduction. sincospif takes the top 32
// bits as a signed number of half turns.
//
// Layout: LANES lanes hold a row, 16 dimensions each as two 16-byte vectors:
// for the rotated part the two that hold eight pairs (vectors u and u + R/16, or
// 2u and 2u + 1), so a pair never leaves its lane and lane u always needs the
// frequencies 8u .. 8u + 7. The 32 / LANES rows of a warp are heads of one token:
// each computes a share of the token's sines and cosines and shuffles pass
// them round, once per warp for all its heads.
#include "bi_internal.h"
#include "bi_ptx.cuh"

namespace bi {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void unpack8(const uint4 &v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = pack_bf16x2(__float_as_uint(x[2 * k]), __float_as_uint(x[2 * k + 1]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Warp: token t and the groups of 32 / LANES heads s, s + splits, ... of its queries, keys and values.
template <int LANES, bool INTER>
__global__ void __launch_bounds__(kThreads)
heads_kernel(const HeadsParams p) {
    grid_dep_wait();      // earlier work of the stream is complete and visible
    grid_dep_launch();
    constexpr int ROWS = 32 / LANES, SHARE = 8 / ROWS;     // heads a warp takes at once; frequencies a lane computes
    const int lane = threadIdx.x & 31, u = lane % LANES, r = lane / LANES;
    const int64_t w = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = w / p.splits;
    if (t >= p.T) return;
    const bool holds = 16 * u < p.D, turns = 16 * u < p.R;
    int64_t pos = 0, slot = 0;
    if (p.R > 0) pos = p.pos[t];
    if (p.slots) slot = p.slots[t];
    uint64_t f[SHARE];
#pragma unroll
    for (int k = 0; k < SHARE; ++k) f[k] = turns ? p.turns[8 * u + r * SHARE + k] : 0;
    if (pos != static_cast<int32_t>(pos)) {                // the whole warp: one token
        if (lane == 0) atomicOr(p.status, kDevBadOffsets);
        return;
    }
    const bool kept = slot >= 0 && slot < p.cache_rows;    // (without a cache: slot 0 of 1)
    if (!kept && slot != -1 && lane == 0) atomicOr(p.status, kDevBadOffsets);

    float c[8], s[8];
    if (p.R > 0) {
        float cs[SHARE], sn[SHARE];
#pragma unroll
        for (int k = 0; k < SHARE; ++k) {
            const uint64_t phase = static_cast<uint64_t>(pos) * f[k];
            sincospif(__int2float_rn(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &sn[k], &cs[k]);
            cs[k] = __fmul_rn(cs[k], p.factor);
            sn[k] = __fmul_rn(sn[k], p.factor);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            c[k] = __shfl_sync(0xffffffffu, cs[k % SHARE], (k / SHARE) * LANES + u);
            s[k] = __shfl_sync(0xffffffffu, sn[k % SHARE], (k / SHARE) * LANES + u);
        }
    }
    // this lane's two vectors of a row
    const int v0 = turns && !INTER ? 8 * u : 16 * u;
    const int v1 = turns && !INTER ? 8 * u + p.R / 2 : 16 * u + 8;
    for (int j = static_cast<int>(w % p.splits); j < p.groups; j += p.splits) {
        const int part = j < p.first[1] ? 0 : j < p.first[2] ? 1 : 2;
        const Heads &h = p.part[part];
        const int head = (j - p.first[part]) * ROWS + r;
        const bool row = head < h.heads && holds && (kept || part == 0) && BI_IN_BOUNDS(v1 + 8 <= p.D && t < p.T, p.status);
        float x[16];
        uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
        if (row) {
            const uint16_t *src = h.src + t * h.lds + static_cast<int64_t>(head) * p.D;
            a = *reinterpret_cast<const uint4 *>(src + v0);
            b = *reinterpret_cast<const uint4 *>(src + v1);
        }
        if (part < 2) {
            unpack8(a, x);
            unpack8(b, x + 8);
            if (h.w) {
                float ss = 0.0f;
#pragma unroll
                for (int k = 0; k < 16; ++k) ss = __fmaf_rn(x[k], x[k], ss);
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float rs = rsqrtf(__fmaf_rn(ss, p.inv_d, p.eps));
                float wt[16];
                if (holds) {
                    unpack8(*reinterpret_cast<const uint4 *>(h.w + v0), wt);
                    unpack8(*reinterpret_cast<const uint4 *>(h.w + v1), wt + 8);
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] = __fmul_rn(__fmul_rn(x[k], rs), wt[k]);
            }
            if (turns) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int ia = INTER ? 2 * k : k, ib = INTER ? 2 * k + 1 : k + 8;
                    const float xa = x[ia], xb = x[ib];
                    x[ia] = __fmaf_rn(xa, c[k], -__fmul_rn(xb, s[k]));
                    x[ib] = __fmaf_rn(xb, c[k], __fmul_rn(xa, s[k]));
                }
            }
            a = pack8(x);
            b = pack8(x + 8);
        }
        if (row) {
            uint16_t *dst = h.dst + (h.cache ? slot : t) * h.ldd + static_cast<int64_t>(head) * p.D;
            *reinterpret_cast<uint4 *>(dst + v0) = a;
            *reinterpret_cast<uint4 *>(dst + v1) = b;
        }
    }
}

template <int LANES>
bi_status launch_lanes(HeadsParams p, bool inter, int sms, cudaStream_t s) {
    constexpr int ROWS = 32 / LANES;
    int g = 0;
    for (int i = 0; i < 3; ++i) {
        p.first[i] = g;
        g += (p.part[i].heads + ROWS - 1) / ROWS;
    }
    p.groups = g;
    // warps a token: all its groups in one where that fills the GPU, else a group each
    const int64_t want = (16 * static_cast<int64_t>(sms) + p.T - 1) / p.T;
    p.splits = static_cast<int32_t>(want < 1 ? 1 : want > g ? g : want);
    const int64_t blocks = (p.T * p.splits + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffff) return BI_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(blocks));
    return inter ? launch_pdl(heads_kernel<LANES, true>, grid, dim3(kThreads), 0, s, p)
                 : launch_pdl(heads_kernel<LANES, false>, grid, dim3(kThreads), 0, s, p);
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
