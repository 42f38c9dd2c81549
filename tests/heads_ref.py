"""Plain 64-bit forms of the operators between projection and attention, and of
windowed attention, for the tests (numpy)."""
import math

import numpy as np


def freqs(R, base=10000.0, scaling=None, s=1.0, L0=0.0, low=1.0, high=4.0):
    """Frequencies and the factor of cos and sin, from their definitions."""
    if scaling == "ntk":
        base = base * s ** (R / (R - 2))
    f = np.array([base ** (-2 * i / R) for i in range(R // 2)])
    if scaling == "linear":
        f = f / s
    if scaling == "bands":
        for i, n in enumerate(L0 * f / (2 * math.pi)):
            t = (n - low) / (high - low)
            f[i] *= 1.0 if n > high else 1 / s if n < low else t + (1 - t) / s
    if scaling == "yarn":
        dim = lambda n: R * math.log(L0 / (2 * math.pi * n)) / (2 * math.log(base))
        a, b = max(math.floor(dim(high)), 0), min(math.ceil(dim(low)), R - 1)
        for i in range(R // 2):
            t = min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
            f[i] *= 1 - t + t / s
        return f, 0.1 * math.log(s) + 1 if s > 1 else 1.0
    return f, 1.0


def angles(positions, turns):
    """p f_i of every position and frequency, reduced to one turn in whole numbers."""
    return np.array([[((int(p) * int(t)) % (1 << 64)) / 2.0 ** 64 for t in turns] for p in positions]) * (2 * math.pi)


def turn(x, angle, inter, factor):
    """x [T, H, D] turned, and the sum |a| + |b| of each element's pair (0 where nothing turns)."""
    R = 2 * angle.shape[1]
    c, s = np.cos(angle)[:, None] * factor, np.sin(angle)[:, None] * factor
    one, two = (slice(0, R, 2), slice(1, R, 2)) if inter else (slice(0, R // 2), slice(R // 2, R))
    y, size = x.copy(), np.zeros_like(x)
    a, b = x[..., one], x[..., two]
    y[..., one], y[..., two] = a * c - b * s, b * c + a * s
    size[..., one] = size[..., two] = (np.abs(a) + np.abs(b)) * abs(factor)
    return y, size


def norm(x, w, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def attention(q, k, v, n, W, S, scale):
    """The last len(q) of n tokens: q [t, Hq, D], k and v [n, Hkv, D] (float64)."""
    G = q.shape[1] // k.shape[1]
    out = np.zeros_like(q)
    for i in range(len(q)):
        p = n - len(q) + i
        j = np.arange(p + 1)
        j = j[(j > p - W) | (j < S)]
        for h in range(q.shape[1]):
            s = k[j, h // G] @ q[i, h] * scale
            e = np.exp(s - s.max())
            out[i, h] = e @ v[j, h // G] / e.sum()
    return out
