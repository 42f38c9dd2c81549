"""Rotary positions, norms of query and key heads, and appends to the paged bf16
cache on the GPU, against plain 64-bit forms; rows' bits alone and in batches,
in place, strided, padded; bad slots and positions; captured; on another stream.

Tolerances. One rounding to bf16: 2^-8 of the value. Before it, in fp32: the
angle is within pi 2^-25 (rounding) + pi 2^-31 (bits dropped) of the exact one,
sincospif within 2^-23, the factor and the two products add 2^-24 of a term
each: together below 2^-20 of factor (|a| + |b|). The norm: a sum of at most 256
squares in 16-term chains and a tree (20 roundings, half of which the root
keeps), the mean's 1 / D, rsqrtf (2^-22) and two products: below 2^-19 more."""
import numpy as np
import pytest

import bi_synth as syn
import heads_ref as ref
from util import bits_of, f64_of, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8


def heads(T, H, D, seed, std=1.0):
    return syn.to_bf16_bits(std * syn.normal_rows(seed, 0, T, H * D)).reshape(T, H, D)


def weight(D, seed):
    return syn.to_bf16_bits(0.4 + 1.6 * syn.rng(seed, 9).random(D).astype(np.float32))


def f64(bits):
    return syn.bf16_bits_to_f32(bits).astype(np.float64)


def turns_of(fr):
    return fr.turns.cpu().numpy().view(np.uint64)


def check(got, want, size, rel, what=""):
    err, lim = np.abs(got - want), HALF * (np.abs(want) + rel * size) + rel * size
    assert (err <= lim).all(), f"{what}: {(err > lim).sum()} of {err.size}, worst {np.max(err / np.maximum(lim, 1e-300)):.3f}"


POSITIONS = [0, 1, -1, 17, 4095, 131071, 1 << 20, (1 << 31) - 1, -(1 << 31), 123456789]


@pytest.mark.parametrize("D,R,inter", [(128, 128, False), (128, 128, True), (128, 64, False), (128, 48, True), (64, 64, False),
                                       (64, 16, True), (80, 32, False), (96, 96, True), (192, 64, False), (256, 256, True),
                                       (256, 240, False), (16, 16, False), (144, 144, False)])
@pytest.mark.parametrize("T,H", [(1, 1), (10, 5), (77, 9)])
def test_rope(bi, D, R, inter, T, H):
    x = heads(T, H, D, D + R + T)
    pos = np.array((POSITIONS * 8)[:T])
    fr = bi.rope_freqs(R, interleaved=inter, factor=1.25)
    got = f64_of(bi.rope(to_dev_bf16(x), to_dev(pos), fr))
    want, size = ref.turn(f64(x), ref.angles(pos, turns_of(fr)), inter, 1.25)
    check(got, want, size, 2.0 ** -20)
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", scale=4.0), dict(scaling="ntk", scale=8.0),
                                dict(scaling="bands", scale=8.0, original_length=8192, low=1.0, high=4.0),
                                dict(scaling="yarn", scale=16.0, original_length=4096, low=1.0, high=32.0)])
@pytest.mark.parametrize("R,base", [(128, 1e6), (64, 1e4), (32, 5e5)])
def test_frequencies(bi, kw, R, base):
    fr = bi.rope_freqs(R, base=base, **kw)
    f, m = ref.freqs(R, base, kw.get("scaling"), kw.get("scale", 1.0), kw.get("original_length", 0.0), kw.get("low", 1.0), kw.get("high", 4.0))
    got = turns_of(fr).astype(np.float64) / 2.0 ** 64 * 2 * np.pi
    assert np.allclose(got, f, rtol=2.0 ** -48, atol=2.0 ** -60)      # a few double roundings, and the unit of a turn
    assert fr.factor == np.float32(m)
    again = bi.rope_freqs(R, freqs=f, factor=m)
    assert np.allclose(turns_of(again).astype(np.float64), turns_of(fr).astype(np.float64), rtol=2.0 ** -48, atol=16)


def test_back_and_forth(bi):
    """Turned by p and by -p gives the row again, but for two roundings."""
    T, H, D = 12, 4, 128
    x = heads(T, H, D, 3)
    fr = bi.rope_freqs(D)
    pos = to_dev(np.arange(T) * 9999)
    y = bi.rope(bi.rope(to_dev_bf16(x), pos, fr), -pos, fr)
    size = np.abs(f64(x)) + np.abs(np.roll(f64(x), D // 2, axis=-1))
    # the first rounding, 2^-8 of each of the pair, turns with it: at most sqrt(2) 2^-8 of |a| + |b|; the second is 2^-8
    assert (np.abs(f64_of(y) - f64(x)) <= 2.0 ** -8 * 2.5 * size).all()


@pytest.mark.parametrize("D,R,inter,Hq,Hkv", [(128, 128, False, 32, 8), (128, 128, True, 32, 4), (128, 64, False, 5, 5), (64, 32, True, 3, 1),
                                              (96, 96, False, 4, 2), (256, 128, False, 7, 3), (80, 0, False, 6, 2)])
@pytest.mark.parametrize("T", [1, 19])
def test_qk_norm_rope(bi, D, R, inter, Hq, Hkv, T):
    q, k, qw, kw = heads(T, Hq, D, 1, 3.0), heads(T, Hkv, D, 2, 0.1), weight(D, 3), weight(D, 4)
    q[0, 0] = 0
    pos = np.array((POSITIONS * 8)[:T])
    fr = bi.rope_freqs(R, interleaved=inter) if R else None
    got = bi.qk_norm_rope(to_dev_bf16(q), to_dev_bf16(k), to_dev_bf16(qw), to_dev_bf16(kw), 1e-6, to_dev(pos) if R else None, fr)
    for g, x, w in zip(got, (q, k), (qw, kw)):
        n = ref.norm(f64(x), f64(w), 1e-6)
        want, size = ref.turn(n, ref.angles(pos, turns_of(fr)), inter, 1.0) if R else (n, np.zeros_like(n))
        check(f64_of(g), want, size + np.abs(n), 2.0 ** -18)
    assert bi.device_status() == bi.BI_OK


def test_rows_do_not_depend_on_the_batch(bi):
    """Few tokens (a warp a group of heads), many (a warp a token): the same bits; strides and places do not matter."""
    T, Hq, Hkv, D = 3000, 6, 3, 128
    fused = to_dev_bf16(heads(T, Hq + 2 * Hkv, D, 5))
    q, k = fused[:, :Hq], fused[:, Hq:Hq + Hkv]
    qw, kw, fr = to_dev_bf16(weight(D, 1)), to_dev_bf16(weight(D, 2)), bi.rope_freqs(D)
    import torch
    pos = torch.arange(T, device="cuda") * 41
    Q, K = bi.qk_norm_rope(q, k, qw, kw, 1e-6, pos, fr)
    for t in (0, 1, 1499, T - 1):
        a, b = bi.qk_norm_rope(q[t:t + 1], k[t:t + 1].clone(), qw, kw, 1e-6, pos[t:t + 1], fr)
        assert torch.equal(a[0], Q[t]) and torch.equal(b[0], K[t])
    again = bi.qk_norm_rope(q.flip(0), k.flip(0), qw, kw, 1e-6, pos.flip(0), fr)
    assert torch.equal(again[0].flip(0), Q) and torch.equal(again[1].flip(0), K)
    # in place, within the projection's rows; the values stay
    v = fused[:, Hq + Hkv:].clone()
    a, b = bi.qk_norm_rope(q, k, qw, kw, 1e-6, pos, fr, Q_out=q, K_out=k)
    assert a is q and b is k and torch.equal(q, Q) and torch.equal(k, K) and torch.equal(fused[:, Hq + Hkv:], v)
    x = Q.clone()
    assert torch.equal(bi.rope(x, pos, fr, Y=x), bi.rope(Q, pos, fr)) and not torch.equal(x, Q)


def test_values_that_are_not_finite_stay_in_their_head(bi):
    import torch
    x = heads(40, 8, 128, 6)
    clean = to_dev_bf16(x)
    bad = clean.clone()
    bad[3, 2, 7], bad[3, 5, 100], bad[20, 0, 127] = float("nan"), float("inf"), float("-inf")
    w, fr, pos = to_dev_bf16(weight(128, 1)), bi.rope_freqs(128), torch.arange(40, device="cuda")
    hit = torch.zeros((40, 8), dtype=torch.bool, device="cuda")
    hit[3, 2] = hit[3, 5] = hit[20, 0] = True
    for f in (lambda t: bi.rope(t, pos, fr), lambda t: bi.qk_norm_rope(t, t, w, w, 1e-6, pos, fr)[0]):
        a, b = f(clean), f(bad)
        assert torch.equal(a[~hit], b[~hit]) and not torch.isfinite(b[hit].float()).all(-1).any()


def pattern_cache(shape, value):
    import torch
    return torch.full(shape, value, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("T,Hq,Hkv,D,bs,R,inter,normed", [(1, 32, 8, 128, 16, 128, False, True), (61, 8, 2, 128, 24, 64, True, True),
                                                           (2600, 4, 4, 128, 16, 128, False, True), (33, 0, 5, 128, 1, 128, False, False),
                                                           (7, 3, 1, 64, 8, 64, True, False), (700, 0, 8, 128, 128, 0, False, True),
                                                           (50, 2, 3, 256, 16, 96, False, True)])
def test_append(bi, T, Hq, Hkv, D, bs, R, inter, normed):
    """Caches hold the bits of the separate calls, Q_out too; everything else stays; padding and bad slots store nothing."""
    import torch
    fused = to_dev_bf16(heads(T, Hq + 2 * Hkv, D, T))
    q, k, v = fused[:, :Hq] if Hq else None, fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    qw, kw = (to_dev_bf16(weight(D, s)) if normed else None for s in (1, 2))
    if not Hq:
        qw = None
    fr = bi.rope_freqs(R, interleaved=inter, factor=0.9) if R else None
    pos = torch.arange(T, device="cuda") * 7 + 3 if R else None
    blocks = -(-T // bs) + 3
    slots = torch.from_numpy(syn.rng(3, T).permutation(blocks * bs)[:T].astype(np.int64)).cuda()
    if T > 5:
        slots[1] = slots[T - 1] = -1
    Kc, Vc = pattern_cache((blocks, bs, Hkv, D), 3.0), pattern_cache((blocks, bs, Hkv, D), -5.0)
    out = bi.kv_append(k, v, slots, Kc, Vc, pos, fr, k_weight=kw, eps=1e-5, Q=q, q_weight=qw)
    assert bi.device_status() == bi.BI_OK
    if normed:
        wantQ, wantK = bi.qk_norm_rope(q if Hq else k, k, qw if Hq else kw, kw, 1e-5, pos, fr)
    elif fr is not None:
        wantQ, wantK = bi.rope(q, pos, fr) if Hq else None, bi.rope(k, pos, fr)
    assert (out is None) == (not Hq) and (not Hq or torch.equal(out, wantQ))
    good = slots >= 0
    for cache, rows, fill in ((Kc, wantK, 3.0), (Vc, v, -5.0)):
        want = pattern_cache((blocks * bs, Hkv, D), fill)
        want[slots[good]] = rows[good]
        assert torch.equal(cache.view(blocks * bs, Hkv, D), want)
    if normed and Hq:                                     # only the keys normed: the queries are turned alone
        K3, V3 = pattern_cache(Kc.shape, 3.0), pattern_cache(Kc.shape, -5.0)
        out3 = bi.kv_append(k, v, slots, K3, V3, pos, fr, k_weight=kw, eps=1e-5, Q=q)
        assert torch.equal(out3, bi.rope(q, pos, fr)) and torch.equal(K3, Kc) and torch.equal(V3, Vc)
    # slots outside: skipped and reported; a position that does not fit in 32 bits: nothing of the token
    if T > 5:
        slots[2], slots[3] = blocks * bs, -7
        if R:
            pos[4] = 1 << 31
        K2, V2 = pattern_cache(Kc.shape, 3.0), pattern_cache(Kc.shape, -5.0)
        out2 = torch.full_like(out, 9.0) if Hq else None
        bi.kv_append(k, v, slots, K2, V2, pos, fr, k_weight=kw, eps=1e-5, Q=q, q_weight=qw, Q_out=out2)
        assert bi.device_status() == bi.BI_ERR_INVALID_ARG
        good[2] = good[3] = False
        if R:
            good[4] = False
        want = pattern_cache((blocks * bs, Hkv, D), 3.0)
        want[slots[good]] = wantK[good]
        assert torch.equal(K2.view(blocks * bs, Hkv, D), want)
        if Hq:
            t = torch.arange(T, device="cuda") != (4 if R else -1)
            assert torch.equal(out2[t], wantQ[t]) and (not R or (out2[4] == 9.0).all())


def test_append_past_2_31(bi):
    """Slots and tokens whose offsets pass 32 bits."""
    import torch
    Hkv, D, bs = 8, 128, 16
    blocks = (1 << 31) // (Hkv * D * bs) + 40
    Kc = torch.zeros((blocks, bs, Hkv, D), dtype=torch.bfloat16, device="cuda")
    Vc = torch.zeros_like(Kc)
    T = 3
    x = to_dev_bf16(heads(T, 2 * Hkv, D, 8))
    wide = torch.zeros(((T - 1) * (1 << 30) + 2 * Hkv * D + 64), dtype=torch.bfloat16, device="cuda")
    far = wide.as_strided((T, 2 * Hkv, D), (1 << 30, D, 1))
    far.copy_(x)
    slots = torch.tensor([blocks * bs - 1, 5, (blocks - 1) * bs], device="cuda")
    fr, pos = bi.rope_freqs(D), torch.tensor([5, 1 << 30, 77], device="cuda")
    bi.kv_append(far[:, :Hkv], far[:, Hkv:], slots, Kc, Vc, pos, fr)
    want = bi.rope(x[:, :Hkv].contiguous(), pos, fr)
    assert torch.equal(Kc.view(-1, Hkv, D)[slots], want) and torch.equal(Vc.view(-1, Hkv, D)[slots], x[:, Hkv:])
    assert int((Kc.view(-1, Hkv * D)[:, 0] != 0).sum()) == T
    assert torch.equal(bi.rope(far, pos, fr, Y=far), bi.rope(x, pos, fr))
    assert bi.device_status() == bi.BI_OK


def test_captured_and_on_another_stream(bi):
    import torch
    T, Hq, Hkv, D, bs = 30, 8, 2, 128, 16
    fused = to_dev_bf16(heads(T, Hq + 2 * Hkv, D, 1))
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    w, fr = to_dev_bf16(weight(D, 1)), bi.rope_freqs(D)
    pos, slots = torch.arange(T, device="cuda"), torch.arange(T, device="cuda")
    Kc, Vc, out = pattern_cache((4, bs, Hkv, D), 0.0), pattern_cache((4, bs, Hkv, D), 0.0), torch.zeros_like(q)
    call = lambda **kw: bi.kv_append(k, v, slots, Kc, Vc, pos, fr, k_weight=w, Q=q, q_weight=w, Q_out=out, **kw)
    call()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call()
    for step in range(3):
        fused.copy_(to_dev_bf16(heads(T, Hq + 2 * Hkv, D, 10 + step)))
        pos.add_(100), slots.copy_(slots.flip(0))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (Kc, Vc, out)]
        call()
        assert all(torch.equal(a, b) for a, b in zip(got, (Kc, Vc, out)))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    y = bi.rope(q, pos, fr, stream=other)
    other.synchronize()
    assert torch.equal(y, bi.rope(q, pos, fr))
    assert bi.device_status() == bi.BI_OK


def test_empty(bi):
    import torch
    e = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    i = torch.empty(0, dtype=torch.int64, device="cuda")
    fr, w = bi.rope_freqs(128), torch.ones(128, dtype=torch.bfloat16, device="cuda")
    c = pattern_cache((2, 16, 4, 128), 1.0)
    assert bi.rope(e, i, fr).shape == (0, 4, 128)
    assert bi.qk_norm_rope(e, e, w, w, 1e-6, i, fr)[1].shape == (0, 4, 128)
    assert bi.kv_append(e, e, i, c, c.clone(), i, fr, Q=e).shape == (0, 4, 128)
    assert bi.rope(torch.empty((3, 0, 128), dtype=torch.bfloat16, device="cuda"), torch.arange(3, device="cuda"), fr).numel() == 0
    assert (c == 1.0).all() and bi.device_status() == bi.BI_OK


def test_refusals(bi):
    import torch
    x = torch.zeros((3, 4, 128), dtype=torch.bfloat16, device="cuda")
    pos, fr, w = torch.arange(3, device="cuda"), bi.rope_freqs(128), torch.ones(128, dtype=torch.bfloat16, device="cuda")
    c, c2 = (torch.zeros((2, 16, 4, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    f32 = torch.zeros((3, 4, 128), device="cuda")
    for name, call in (("X", lambda o: bi.rope(o, pos, fr)), ("positions", lambda o: bi.rope(x, o, fr)), ("Y", lambda o: bi.rope(x, pos, fr, Y=o)),
                       ("freqs", lambda o: bi.rope(x, pos, o)), ("K", lambda o: bi.qk_norm_rope(x, o, w, w, 1e-6, pos, fr)),
                       ("q_weight", lambda o: bi.qk_norm_rope(x, x, o, w, 1e-6, pos, fr)), ("slots", lambda o: bi.kv_append(x, x, o, c, c2)),
                       ("K_cache", lambda o: bi.kv_append(x, x, pos, o, c2)), ("V", lambda o: bi.kv_append(x, o, pos, c, c2)),
                       ("k_weight", lambda o: bi.kv_append(x, x, pos, c, c2, k_weight=o))):
        for other in ([1, 2], f32, x.cpu()):
            with pytest.raises(TypeError, match=name):
                call(other)
    for call in (lambda: bi.rope(x, pos[:2], fr), lambda: bi.rope(x.transpose(0, 1), pos, fr), lambda: bi.rope(x, pos, fr, Y=x[:, :2]),
                 lambda: bi.qk_norm_rope(x, x[:2], w, w, 1e-6, pos, fr), lambda: bi.qk_norm_rope(x, x, w[:64], w, 1e-6, pos, fr),
                 lambda: bi.qk_norm_rope(x, x, w, w, 1e-6, pos, None), lambda: bi.kv_append(x, x[:, :2], pos, c, c2),
                 lambda: bi.kv_append(x, x, pos, c, c2[:1]), lambda: bi.kv_append(x, x, pos, c, c2, q_weight=w),
                 lambda: bi.kv_append(x, x, pos[:2], c, c2), lambda: bi.kv_append(x, x, pos, c.transpose(0, 1), c2),
                 lambda: bi.rope_freqs(128, scaling="other"), lambda: bi.rope_freqs(128, freqs=[1.0]),
                 lambda: bi.RopeFreqs(fr.turns, 64)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: bi.rope(x[..., :64].contiguous(), pos, fr), lambda: bi.rope_freqs(24), lambda: bi.rope_freqs(512),
                 lambda: bi.rope_freqs(64, base=1.0), lambda: bi.rope_freqs(64, scaling="yarn", scale=4.0),
                 lambda: bi.rope_freqs(64, scaling="linear", scale=0.0), lambda: bi.rope_freqs(16, freqs=[float("nan")] * 8),
                 lambda: bi.rope(torch.zeros((3, 4, 40), dtype=torch.bfloat16, device="cuda"), pos, bi.rope_freqs(16)),
                 lambda: bi.qk_norm_rope(x, x, w, w, -1.0, pos, fr), lambda: bi.qk_norm_rope(x, x, w, w, float("nan"), pos, fr),
                 lambda: bi.rope(x[:1].expand(3, 4, 128), pos, fr)):
        with pytest.raises(bi.BiError):
            call()
    with pytest.raises(AttributeError):
        fr.factor = 2.0
    assert bi.device_status() == bi.BI_OK
