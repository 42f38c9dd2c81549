"""The calls over heads and the windowed calls of the C ABI reject bad arguments before touching a GPU, and the
frequencies of rotations, computed on the host (CPU only)."""
import ctypes

import numpy as np
import pytest

import heads_ref as ref

FAKE = 0x10000                    # never dereferenced: every call below fails validation first
f = ctypes.c_float


@pytest.fixture(scope="module")
def so():
    from invariant_deterministic_bi_gb300 import _build
    _build.build()
    import invariant_deterministic_bi_gb300 as m
    return m.load()


def rope_t(**kw):
    import invariant_deterministic_bi_gb300 as m
    a = dict(dict(turns=FAKE, rotary_dim=128, interleaved=0, factor=1.0), **kw)
    return ctypes.byref(m._Rope(a["turns"], a["rotary_dim"], a["interleaved"], a["factor"]))


BAD_ROPE = [(dict(rotary_dim=0), 1), (dict(rotary_dim=144), 1), (dict(rotary_dim=40), 2), (dict(turns=None), 1), (dict(turns=FAKE + 4), 3),
            (dict(factor=float("nan")), 1)]


@pytest.mark.parametrize("change,want", [(dict(T=-1), 1), (dict(T=1 << 31), 1), (dict(D=0), 1), (dict(D=264), 2), (dict(D=136), 2), (dict(D=272), 2),
                                         (dict(X=None), 1), (dict(Y=None), 1), (dict(pos=None), 1), (dict(H=-1), 1), (dict(ldx=504), 1),
                                         (dict(ldy=504), 1), (dict(ldx=516), 3), (dict(X=FAKE + 8), 3), (dict(pos=FAKE + 4), 3),
                                         (dict(H=(1 << 20) + 1, ldx=1 << 40, ldy=1 << 40), 2), (dict(rope=None), 1), (dict(T=0), 0), (dict(H=0), 0)]
                         + [(dict(rope=r), w) for r, w in BAD_ROPE])
def test_rope(so, change, want):
    a = dict(dict(X=FAKE, ldx=512, pos=FAKE, T=4, H=4, D=128, rope={}, Y=FAKE, ldy=512), **change)
    r = None if a["rope"] is None else rope_t(**a["rope"])
    assert so.bi_rope(a["X"], a["ldx"], a["pos"], a["T"], a["H"], a["D"], r, a["Y"], a["ldy"], None) == want


@pytest.mark.parametrize("change,want", [(dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(qw=None), 1), (dict(kw=None), 1), (dict(Q=None), 1),
                                         (dict(Ko=None), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(ldk=120), 1), (dict(kw=FAKE + 8), 3),
                                         (dict(ldqo=516), 3), (dict(pos=None), 1), (dict(T=0), 0)] + [(dict(rope=r), w) for r, w in BAD_ROPE])
def test_qk_norm_rope(so, change, want):
    a = dict(dict(Q=FAKE, ldq=512, K=FAKE, ldk=256, qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE, T=4, Hq=4, Hkv=2, D=128, rope={}, Qo=FAKE, ldqo=512,
                  Ko=FAKE, ldko=256), **change)
    assert so.bi_qk_norm_rope(a["Q"], a["ldq"], a["K"], a["ldk"], a["qw"], a["kw"], f(a["eps"]), a["pos"], a["T"], a["Hq"], a["Hkv"], a["D"],
                              rope_t(**a["rope"]), a["Qo"], a["ldqo"], a["Ko"], a["ldko"], None) == want


@pytest.mark.parametrize("change,want", [(dict(T=-1), 1), (dict(nb=0), 1), (dict(bs=0), 1), (dict(Hkv=0), 1), (dict(Hq=-1), 1), (dict(eps=-1.0), 1),
                                         (dict(slots=None), 1), (dict(slots=FAKE + 4), 3), (dict(nb=1 << 38, bs=16), 2), (dict(Kc=None), 1),
                                         (dict(Vc=FAKE + 8), 3), (dict(V=None), 1), (dict(ldv=120), 1), (dict(D=100), 2), (dict(Qo=None), 1),
                                         (dict(Hq=0), 1), (dict(Hq=0, Q=None, Qo=None), 1), (dict(ldq=520, qw=FAKE + 2), 3), (dict(T=0), 0)]
                         + [(dict(rope=r), w) for r, w in BAD_ROPE])
def test_kv_append(so, change, want):
    a = dict(dict(K=FAKE, ldk=256, V=FAKE, ldv=256, T=4, slots=FAKE, kw=FAKE, eps=1e-6, pos=FAKE, rope={}, Kc=FAKE, Vc=FAKE, nb=64, Hkv=2, D=128,
                  bs=16, Q=FAKE, ldq=512, qw=FAKE, Hq=4, Qo=FAKE, ldqo=512), **change)
    assert so.bi_kv_append(a["K"], a["ldk"], a["V"], a["ldv"], a["T"], a["slots"], a["kw"], f(a["eps"]), a["pos"], rope_t(**a["rope"]), a["Kc"],
                           a["Vc"], a["nb"], a["Hkv"], a["D"], a["bs"], a["Q"], a["ldq"], a["qw"], a["Hq"], a["Qo"], a["ldqo"], None) == want


def attn(**kw):
    a = dict(dict(Q=FAKE, cu=FAKE, T=9, K=FAKE, V=FAKE, table=FAKE, mb=8, nb=64, lens=FAKE, B=4, Hq=32, Hkv=8, D=128, bs=16, L=1024, q=4,
                  scale=f(0.1), W=100, S=4, ws=FAKE, wsb=1 << 30, O=FAKE), **kw)
    mid = (a["K"], a["V"], a["table"], a["mb"], a["nb"], a["lens"], a["B"], a["Hq"], a["Hkv"], a["D"], a["bs"], a["L"])
    tail = (a["scale"], a["W"], a["S"], a["ws"], a["wsb"], a["O"], None)
    return (a["Q"], *mid, *tail), (a["Q"], a["cu"], a["T"], *mid, a["q"], *tail)


@pytest.mark.parametrize("change,want", [
    (dict(W=0), 1), (dict(W=-5), 1), (dict(S=-1), 1), (dict(B=-1), 1), (dict(B=65536), 1), (dict(L=0), 1), (dict(L=(1 << 30) + 1), 1), (dict(mb=0), 1),
    (dict(nb=0), 1), (dict(bs=0), 1), (dict(scale=f(float("nan"))), 1), (dict(Q=None), 1), (dict(V=None), 1), (dict(lens=None), 1), (dict(D=64), 2),
    (dict(Hkv=3), 2), (dict(Hq=24), 2), (dict(Q=FAKE + 8), 3), (dict(V=FAKE + 8), 3), (dict(table=FAKE + 2), 3), (dict(ws=FAKE + 8), 3), (dict(B=0), 0)])
def test_attention(so, change, want):
    decode, extend = attn(**change)
    assert so.bi_attention_decode_window(*decode) == want
    assert so.bi_attention_extend_window(*extend) == want


def test_attention_own_arguments_and_workspaces(so):
    size, plain = so.bi_attention_decode_window_workspace_size, so.bi_attention_decode_workspace_size
    assert size(4, 32, 1024, 2000, 0) == plain(4, 32, 1024) == size(4, 32, 1024, 1, 1024)
    assert size(4, 32, 100000, 1, 0) == plain(4, 32, 128) and size(4, 32, 100000, 2, 0) == plain(4, 32, 256)
    assert size(4, 32, 100000, 128, 0) == plain(4, 32, 256) and size(4, 32, 100000, 130, 129) == plain(4, 32, 5 * 128)
    assert size(4, 32, 0, 1, 0) == size(4, 32, 128, 0, 0) == size(4, 32, 128, 1, -1) == size(-1, 32, 128, 1, 0) == -1
    assert size(4, 32, 1 << 30, 0x7FFFFFFF, 0x7FFFFFFF) == plain(4, 32, 1 << 30)
    need = size(4, 32, 1024, 100, 4)
    assert so.bi_attention_decode_window(*attn(wsb=need - 1)[0]) == 1
    assert so.bi_attention_decode_window(*attn(ws=None)[0]) == 1
    assert so.bi_attention_extend_window(*attn(q=0)[1]) == so.bi_attention_extend_window(*attn(wsb=-1)[1]) == 1
    assert so.bi_attention_extend_window(*attn(cu=FAKE + 2)[1]) == 3
    assert so.bi_attention_extend_window(*attn(T=0)[1]) == 0
    size = so.bi_attention_extend_window_workspace_size
    assert size(-1, 32, 8, 128, 1, 5, 0) == size(4, 32, 5, 128, 1, 5, 0) == size(4, 32, 8, 128, 1, 0, 0) == size(4, 32, 8, 128, 0, 5, 0) == -1


@pytest.mark.parametrize("R,base,kind,s,L0,low,high", [(128, 1e6, 0, 1, 0, 1, 4), (64, 1e4, 1, 4, 0, 1, 4), (32, 1e4, 2, 8, 0, 1, 4), (16, 2.0, 2, 0.5, 0, 1, 4),
                                                       (128, 5e5, 3, 8, 8192, 1, 4), (128, 1e6, 4, 16, 4096, 1, 32), (256, 1e4, 4, 0.5, 100, 1, 2)])
def test_frequencies(so, R, base, kind, s, L0, low, high):
    turns, m = np.zeros(R // 2 + 1, np.uint64), f()
    turns[-1] = 77
    assert so.bi_rope_freqs(R, kind, base, s, L0, low, high, None, turns.ctypes.data, ctypes.byref(m)) == 0
    want, factor = ref.freqs(R, base, [None, "linear", "ntk", "bands", "yarn"][kind], s, L0, low, high)
    # double precision throughout: pow, and a few products
    assert np.allclose(turns[:-1].astype(np.float64) / 2.0 ** 64 * 2 * np.pi, want % (2 * np.pi), rtol=2.0 ** -46, atol=2.0 ** -60)
    assert turns[-1] == 77 and m.value == np.float32(factor)


def test_given_frequencies(so):
    given = (ctypes.c_double * 8)(0.0, 1.0, -1.0, 2 * np.pi * 1e6, 1e-9, 2 * np.pi * 0.75, -1e-300, 5.0)
    turns, m = np.zeros(8, np.uint64), f()
    assert so.bi_rope_freqs(16, 5, 0, 0, 0, 0, 0, given, turns.ctypes.data, ctypes.byref(m)) == 0 and m.value == 1.0
    back = turns.astype(np.float64) / 2.0 ** 64
    want = np.array(list(given)) / (2 * np.pi) % 1.0
    assert (np.minimum(np.abs(back - want), 1 - np.abs(back - want)) < 2.0 ** -30).all()      # (a million turns keep 33 bits of their fraction)
    for bad in (float("nan"), float("inf"), 2.0 ** 41):
        given[3] = bad
        assert so.bi_rope_freqs(16, 5, 0, 0, 0, 0, 0, given, turns.ctypes.data, ctypes.byref(m)) == 1


@pytest.mark.parametrize("a,want", [((0, 0, 1e4, 1, 0, 1, 4), 1), ((24, 0, 1e4, 1, 0, 1, 4), 2), ((512, 0, 1e4, 1, 0, 1, 4), 2), ((64, 6, 1e4, 1, 0, 1, 4), 1),
                                    ((64, -1, 1e4, 1, 0, 1, 4), 1), ((64, 0, 1.0, 1, 0, 1, 4), 1), ((64, 0, float("inf"), 1, 0, 1, 4), 1),
                                    ((64, 1, 1e4, 0, 0, 1, 4), 1), ((64, 2, 1e4, float("nan"), 0, 1, 4), 1), ((64, 3, 1e4, 2, 0, 1, 4), 1),
                                    ((64, 4, 1e4, 2, 100, 4, 4), 1), ((64, 3, 1e4, 2, 100, 0, 4), 1), ((64, 5, 1e4, 2, 100, 1, 4), 1)])
def test_frequencies_refused(so, a, want):
    turns, m = np.zeros(256, np.uint64), f()
    assert so.bi_rope_freqs(*a, None, turns.ctypes.data, ctypes.byref(m)) == want
    assert not turns.any()
