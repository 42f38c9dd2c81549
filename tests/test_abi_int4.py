"""The 4-bit calls of the C ABI reject bad arguments before touching a GPU (CPU only)."""
import ctypes

import pytest

FAKE = 0x10000                    # never dereferenced: every call below fails validation first
f = ctypes.c_float


@pytest.fixture(scope="module")
def so():
    from invariant_deterministic_bi_gb300 import _build
    _build.build()
    import invariant_deterministic_bi_gb300 as m
    return m.load()


def kv(**kw):
    a = dict(dict(K=FAKE, ldk=1024, V=FAKE, ldv=1024, T=4, slots=FAKE, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, nb=64, Hkv=8, D=128,
                  bs=16), **kw)
    return (a["K"], a["ldk"], a["V"], a["ldv"], a["T"], a["slots"], a["kc"], a["ks"], a["vc"], a["vs"], a["nb"], a["Hkv"],
            a["D"], a["bs"], None), (a["kc"], a["ks"], a["vc"], a["vs"], a["nb"], a["Hkv"], a["D"], a["bs"], a["slots"], a["T"],
                                     a["K"], a["ldk"], a["V"], a["ldv"], None)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), 1), (dict(T=1 << 31), 1), (dict(K=None), 1), (dict(slots=None), 1), (dict(vs=None), 1), (dict(nb=0), 1),
    (dict(Hkv=0), 1), (dict(bs=0), 1), (dict(ldk=1016), 1), (dict(D=64), 2), (dict(nb=1 << 40), 2),
    (dict(nb=1 << 25, bs=16, Hkv=8), 2), (dict(nb=1, bs=1, Hkv=(1 << 20) + 1, ldk=1 << 28, ldv=1 << 28), 2), (dict(ldv=1028), 3), (dict(V=FAKE + 8), 3), (dict(kc=FAKE + 8), 3),
    (dict(ks=FAKE + 8), 3), (dict(slots=FAKE + 4), 3), (dict(T=0), 0)])
def test_append_and_read(so, change, want):
    append, read = kv(**change)
    assert so.bi_kv_int4_append(*append) == want
    assert so.bi_kv_int4_read(*read) == want


def attn(**kw):
    a = dict(dict(Q=FAKE, cu=FAKE, T=9, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, table=FAKE, mb=8, nb=64, lens=FAKE, B=4, Hq=32, Hkv=8,
                  D=128, bs=16, L=128, q=4, scale=f(0.1), ws=FAKE, wsb=1 << 30, O=FAKE), **kw)
    cache = (a["kc"], a["ks"], a["vc"], a["vs"])
    mid = (a["table"], a["mb"], a["nb"], a["lens"], a["B"], a["Hq"], a["Hkv"], a["D"], a["bs"], a["L"])
    return ((a["Q"], *cache, *mid, a["scale"], a["ws"], a["wsb"], a["O"], None),
            (a["Q"], a["cu"], a["T"], *cache, *mid, a["q"], a["scale"], a["ws"], a["wsb"], a["O"], None))


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), 1), (dict(B=65536), 1), (dict(L=0), 1), (dict(L=(1 << 30) + 1), 1), (dict(mb=0), 1), (dict(nb=0), 1),
    (dict(scale=f(float("nan"))), 1), (dict(Q=None), 1), (dict(kc=None), 1), (dict(lens=None), 1), (dict(D=64), 2),
    (dict(Hkv=3), 2), (dict(Hq=48, Hkv=4), 2), (dict(Hq=24), 2), (dict(nb=1 << 40), 2), (dict(Q=FAKE + 8), 3),
    (dict(vc=FAKE + 8), 3), (dict(vs=FAKE + 8), 3), (dict(table=FAKE + 2), 3), (dict(B=0), 0)])
def test_attention(so, change, want):
    decode, extend = attn(**change)
    assert so.bi_attention_decode_int4(*decode) == want
    assert so.bi_attention_extend_int4(*extend) == want


def test_attention_own_arguments(so):
    assert so.bi_attention_decode_int4(*attn(wsb=100)[0]) == 1
    assert so.bi_attention_decode_int4(*attn(ws=FAKE + 8)[0]) == 3
    assert so.bi_attention_decode_int4(*attn(B=65535, Hq=1 << 30, Hkv=1 << 27, L=1 << 30, nb=1, bs=1)[0]) == 1
    assert so.bi_attention_extend_int4(*attn(q=0)[1]) == 1
    assert so.bi_attention_extend_int4(*attn(cu=FAKE + 2)[1]) == 3
    assert so.bi_attention_extend_int4(*attn(T=0)[1]) == 0
    assert so.bi_attention_extend_int4(*attn(ws=FAKE + 8)[1]) == 3
    size = so.bi_attention_extend_int4_workspace_size
    assert size(80, 32, 8, 4000, 5) == so.bi_attention_decode_workspace_size(80, 32, 4000)
    assert size(4096, 32, 8, 8192, 4096) == 0             # many rows: the tiled kernel
    assert size(4, 32, 5, 128, 1) == size(4, 8, 32, 128, 1) == size(-1, 32, 8, 128, 1) == size(4, 32, 8, 0, 1) == -1
    assert size(1 << 60, 32, 8, 1 << 30, 1) == -1


@pytest.mark.parametrize("change,want", [
    (dict(M=-1), 1), (dict(K=0), 1), (dict(g=0), 1), (dict(X=None), 1), (dict(S=None), 1), (dict(ldx=100), 1), (dict(ldy=100), 1),
    (dict(g=16), 2), (dict(g=96), 2), (dict(g=192), 2), (dict(N=500), 2), (dict(ldx=260), 3), (dict(W=FAKE + 8), 3),
    (dict(X=FAKE + 8), 3), (dict(S=FAKE + 8), 3), (dict(Z=FAKE + 4), 3), (dict(M=0), 0), (dict(N=0), 0)])
def test_gemm(so, change, want):
    a = dict(dict(X=FAKE, ldx=256, W=FAKE, S=FAKE, Z=None, Y=FAKE, ldy=512, M=4, N=512, K=256, g=64), **change)
    assert so.bi_gemm_int4(a["X"], a["ldx"], a["W"], a["S"], a["Z"], a["Y"], a["ldy"], a["M"], a["N"], a["K"], a["g"], None) == want
