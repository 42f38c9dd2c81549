"""Plain 64-bit forms of the 4-bit operators (numpy, CPU): the cache format,
its packed layout, attention over held values and the int4-weight linear."""
import numpy as np

import bi_synth as syn

GROUP = 32


def held(bits):
    """bf16 bit patterns [..., 128] -> (n [..., 128], s [..., 4]) with value n * s; NaN scale for non-finite groups."""
    with np.errstate(invalid="ignore"):
        x = syn.bf16_bits_to_f32(bits).astype(np.float64).reshape(*bits.shape[:-1], 4, GROUP)
        amax = np.abs(x).max(-1)
        need = np.clip(amax / 7.0, 2.0 ** -100, 2.0 ** 120)
        m, e = np.frexp(need)
        s = np.ldexp(np.ceil(m * 16.0), e - 4)
        s = np.where(np.isfinite(amax), s, np.nan)
        n = np.clip(np.rint(x / s[..., None]), -7, 7)
        n = np.where(np.isfinite(s)[..., None], n, 0.0)
    return n.reshape(bits.shape), s


def values(n, s):
    return (n.reshape(*s.shape, GROUP) * s[..., None]).reshape(n.shape)


def pack(n, offset):
    """Codes of a token's rows [..., 128] at this offset of its block -> the cache's bytes [..., 64]."""
    words = np.zeros(n.shape[:-1] + (32,), np.uint16)
    u = (n + 8).astype(np.uint16)
    for d in range(128):
        i, q, r = d // 32, d // 8 % 4, d % 8
        words[..., 8 * (i ^ (offset // 2 % 4)) + r] |= u[..., d] << (4 * q)
    return words.view(np.uint8)


def attention(q, k, v, scale, causal_from=None):
    """softmax(scale q k^T) v in 64 bits: q [T, Hq, D], k, v [L, Hkv, D]; row t sees tokens 0 .. causal_from + t."""
    T, Hq, _ = q.shape
    L, Hkv, _ = k.shape
    out = np.empty(q.shape)
    for h in range(Hq):
        s = scale * (q[:, h] @ k[:, h // (Hq // Hkv)].T)
        if causal_from is not None:
            s = np.where(np.arange(L)[None] <= causal_from + np.arange(T)[:, None], s, -np.inf)
        p = np.exp(s - s.max(-1, keepdims=True))
        out[:, h] = (p / p.sum(-1, keepdims=True)) @ v[:, h // (Hq // Hkv)]
    return out


def gemm(x, W, S, Z):
    """(Y, sum |x w|) in 64 bits: x [M, K], W u8 [N, K/2], S [N, G], Z u8 [N, G] or None."""
    N, G = S.shape
    u = np.stack([W & 15, W >> 4], -1).reshape(N, G, -1).astype(np.float64)
    w = ((u - (8.0 if Z is None else Z.astype(np.float64)[..., None])) * S[..., None]).reshape(N, -1)
    return x @ w.T, np.abs(x) @ np.abs(w).T
