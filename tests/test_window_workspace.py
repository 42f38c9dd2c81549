"""The workspace of windowed extend: room for the tokens that are split over the chunks, and for no others. Sizes on
the CPU; on the GPU that a call uses what its size says, in the batches that a server makes (single tokens beside a
prompt), with the bits of the tiles."""
import numpy as np
import pytest

from test_attention_window import Case

RECORD = 130 * 4                          # (m, l, o[128]) of a head and chunk, fp32
MOST = 512 << 20


@pytest.fixture(scope="module")
def size():
    from invariant_deterministic_bi_gb300 import _build
    _build.build()
    import invariant_deterministic_bi_gb300 as m
    return m.attention_extend_window_workspace_size


def place(W, S, Hq, most):
    """Bytes of one token's results: the chunks that it can see."""
    chunks = min((W + 126) // 128 + 1 + -(-S // 128), -(-most // 128))
    return Hq * chunks * RECORD


@pytest.mark.parametrize("T,most,W,S", [(1024, 1024, 1024, 0), (1500, 8192, 2000, 16), (4096, 8192, 4096, 4), (700, 32768, 4096, 0), (100000, 1 << 30, 1, 0)])
@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (64, 8), (8, 8)])
def test_a_prompt_asks_for_nothing(size, T, most, W, S, Hq, Hkv):
    """But where its tiles would leave SMs idle (one query head a KV head here): then all of it is split."""
    got = size(T, Hq, Hkv, most, T, W, S, B=1)
    assert got == 0 or (Hq == Hkv and got == T * place(W, S, Hq, most))


@pytest.mark.parametrize("W", [1024, 2048, 4096])
@pytest.mark.parametrize("Hq,Hkv,few", [(32, 8, 16), (64, 8, 8)])
@pytest.mark.parametrize("prompt", [512, 1500])
def test_single_tokens_beside_a_prompt(size, W, Hq, Hkv, few, prompt):
    """63 single tokens and a prompt: the split is on, with room for `few` tokens of every sequence at most."""
    got, one = size(63 + prompt, Hq, Hkv, 9000, prompt, W, 4, B=64), place(W, 4, Hq, 9000)
    assert 64 * one <= got <= min(MOST, 64 * few * one) and got % one == 0


def test_sizes(size):
    assert size(64, 32, 8, 9000, 1, 1024, 4, B=64) == 64 * place(1024, 4, 32, 9000) == size(64, 32, 8, 9000, 100000, 1024, 4, B=64)
    assert size(0, 32, 8, 9000, 1, 1024, 4, B=64) == size(64, 32, 8, 9000, 1, 1024, 4, B=0) == 0
    for bad in (dict(B=-1), dict(B=65536), dict(W=0), dict(S=-1), dict(T=-1), dict(T=1 << 31), dict(Hkv=5), dict(L=0), dict(L=(1 << 30) + 1), dict(q=0)):
        a = dict(dict(T=64, Hkv=8, L=9000, q=1, W=1024, S=4, B=64), **bad)
        assert size(a["T"], 32, a["Hkv"], a["L"], a["q"], a["W"], a["S"], B=a["B"]) == -1, bad
    r = np.random.default_rng(1)
    some = 0
    for _ in range(3000):
        B, most = int(2 ** r.uniform(0, 12)), int(2 ** r.uniform(0, 12))
        T = int(r.integers(B, B * most + 1))
        G, Hkv, W, S, L = int(r.choice([1, 2, 4, 8])), int(r.choice([1, 2, 8])), int(2 ** r.uniform(0, 14)), int(r.choice([0, 4, 200])), int(2 ** r.uniform(0, 20))
        got, any_b = size(T, G * Hkv, Hkv, L, most, W, S, B=B), size(T, G * Hkv, Hkv, L, most, W, S)
        one = place(W, S, G * Hkv, L)
        assert 0 <= got <= min(MOST, T * one) and got % one == 0
        assert any_b == 0 or got <= any_b
        some += got > 0
    assert some > 300


def run(bi, c, W, S, bytes_, touched=True):
    """The call with a workspace of exactly these bytes, and what follows it left alone; it writes to it or not."""
    import torch
    ws = torch.full((bytes_ + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    got = c.extend(bi, W, S, ws=ws[:bytes_])
    assert (ws[bytes_:] == 0xFF).all()
    assert bool((ws[:bytes_] != 0xFF).any()) == touched
    assert torch.equal(got, c.tiled(bi, W, S))
    assert bi.device_status() == bi.BI_OK
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("q,Hq,Hkv,bs,W,S", [
    ([1] * 30 + [700] + [1] * 33, 32, 8, 16, 300, 4),                   # a place for `few` tokens of every sequence
    ([1] * 20 + [300, 3, 0, 16, 17, 8, 2], 16, 4, 24, 200, 130),
    ([5, 1, 90, 8, 2, 64, 3], 16, 2, 16, 1000, 0),
    ([3] * 40, 32, 8, 16, 150, 4),                                      # a place for every row
    ([40] * 6, 8, 2, 16, 90, 0),
])
def test_exactly_its_room(bi, q, Hq, Hkv, bs, W, S):
    c = Case([x + 7 * (i % 90) + (x == 0) for i, x in enumerate(q)], q, Hq, Hkv, bs, seed=len(q))
    need = bi.attention_extend_window_workspace_size(sum(q), Hq, Hkv, c.max_len, max(q), W, S, B=len(q))
    assert need > 0
    got = run(bi, c, W, S, need)
    run(bi, c, W, S, need - 16, touched=False)
    rows = np.unique(np.concatenate([np.arange(0, sum(q), 17), np.arange(min(sum(q), 40))]))
    import torch
    assert torch.equal(got[torch.from_numpy(rows).cuda()], c.cut(bi, W, S, tokens=rows))


@pytest.mark.gpu
def test_where_every_row_would_not_fit(bi):
    """Single tokens and a few drafts beside a prompt whose rows would take more than 512 MB: those are split all the
    same, also where there is room for fewer places a sequence than a tile has."""
    import torch
    W, S, Hq, Hkv = 4096, 4, 32, 8
    q = [1] * 40 + [1100] + [1] * 12 + [13, 14, 15, 16, 2, 5] + [1] * 5
    c = Case([x + 60 * (i % 70) for i, x in enumerate(q)], q, Hq, Hkv, 16, seed=3)
    c.max_len = 5000                                                    # (a generous most: 34 chunks a token)
    assert bi.attention_extend_window_workspace_size(sum(q), Hq, Hkv, 5000, max(q), W, S) == 0
    need = bi.attention_extend_window_workspace_size(sum(q), Hq, Hkv, 5000, max(q), W, S, B=len(q))
    assert 0 < need < 16 * len(q) * place(W, S, Hq, 5000) <= 2 * MOST
    got = run(bi, c, W, S, need)
    assert torch.equal(got, c.extend(bi, W, S))


@pytest.mark.gpu
def test_a_call_for_one_prompt_allocates_its_output_alone(bi):
    import torch
    c = Case([1100], [1024], 32, 8, 16, seed=4)
    c.extend(bi, 1024, 0)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    O = c.extend(bi, 1024, 0)
    assert torch.cuda.max_memory_allocated() - before <= O.numel() * 2 + (1 << 20)
    assert bi.device_status() == bi.BI_OK
