"""Decode and extend attention with a sliding window and first tokens that stay
visible, on the GPU: parity with a plain 64-bit form, the bits of the calls
without a window where it holds every token, extend = decode of the cut
sequence, and what stands out of sight (blocks given back, infinities and NaN)
without effect. Tolerance: that of the calls without a window, 1e-2 |ref| + 2e-3
on values of size 1 (bf16 rounding 2^-8 and an absolute floor for cancellation;
leaving out tokens changes no step of it)."""
import numpy as np
import pytest

import bi_synth as syn
import heads_ref as ref
from util import assert_close_rel, bits_of, f64_of, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu
D = 128
SCALE = D ** -0.5
RTOL, ATOL = 1e-2, 2e-3


def normal(seed, stream, *shape):
    return syn.to_bf16_bits(syn.normal_rows(seed, stream, int(np.prod(shape[:-1])), shape[-1])).reshape(shape)


class Case:
    """Sequences of lens tokens, the last q of each new, in a paged cache."""

    def __init__(self, lens, q, Hq, Hkv, bs, seed=0):
        import torch
        self.lens, self.q = [int(x) for x in lens], [int(x) for x in q]
        nb = -(-max(self.lens) // bs)
        blocks = len(lens) * nb + 3
        self.table_np = syn.rng(seed, 2).permutation(blocks)[:len(lens) * nb].astype(np.int32).reshape(len(lens), nb)
        self.Kb, self.Vb = normal(seed, 3, blocks, bs, Hkv, D), normal(seed, 4, blocks, bs, Hkv, D)
        self.Qb = normal(seed, 5, sum(q), Hq, D)
        self.K, self.V, self.Q = to_dev_bf16(self.Kb), to_dev_bf16(self.Vb), to_dev_bf16(self.Qb)
        self.table, self.len_t = to_dev(self.table_np), torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.cu_np = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
        self.cu, self.bs, self.max_len = to_dev(self.cu_np), bs, max(self.lens)

    def rows(self, b):
        j = np.arange(self.lens[b])
        at = self.table_np[b][j // self.bs], j % self.bs
        return tuple(syn.bf16_bits_to_f32(x[at]).astype(np.float64) for x in (self.Kb, self.Vb))

    def reference(self, W, S):
        out = []
        for b in range(len(self.lens)):
            q = syn.bf16_bits_to_f32(self.Qb[self.cu_np[b]:self.cu_np[b + 1]]).astype(np.float64)
            out.append(ref.attention(q, *self.rows(b), self.lens[b], W, S, SCALE))
        return np.concatenate(out)

    def decode(self, bi, W, S, **kw):
        a = dict(dict(Q=self.Q, K=self.K, V=self.V, table=self.table, lens=self.len_t, max_len=self.max_len), **kw)
        return bi.attention_decode_window(a["Q"], a["K"], a["V"], a["table"], a["lens"], a["max_len"], SCALE, W, S,
                                          O=a.get("O"), workspace=a.get("ws"))

    def extend(self, bi, W, S, **kw):
        a = dict(dict(Q=self.Q, cu=self.cu, K=self.K, V=self.V, table=self.table, lens=self.len_t, max_len=self.max_len,
                      max_q=max(1, max(self.q))), **kw)
        return bi.attention_extend_window(a["Q"], a["cu"], a["K"], a["V"], a["table"], a["lens"], a["max_len"], a["max_q"], SCALE,
                                          W, S, O=a.get("O"), workspace=a.get("ws"))

    def tiled(self, bi, W, S, **kw):
        """Without room for the split over chunks."""
        import torch
        return self.extend(bi, W, S, ws=torch.empty(16, dtype=torch.uint8, device="cuda"), **kw)

    def cut(self, bi, W, S, tokens=None, **kw):
        """Every new token (or these) decoded over its cut sequence."""
        import torch
        seq = np.repeat(np.arange(len(self.q)), self.q)
        n = np.concatenate([np.arange(l - q + 1, l + 1) for l, q in zip(self.lens, self.q)])
        at = np.arange(len(n)) if tokens is None else np.asarray(tokens)
        return self.decode(bi, W, S, Q=self.Q[torch.from_numpy(at).cuda()].contiguous(), table=self.table[torch.from_numpy(seq[at]).cuda()].contiguous(),
                           lens=torch.from_numpy(n[at].astype(np.int32)).cuda(), **kw)


WINDOWS = [(1, 0), (1, 1), (3, 130), (127, 0), (128, 4), (129, 128), (200, 300), (1000, 1), (1 << 30, 0)]


@pytest.mark.parametrize("W,S", WINDOWS)
@pytest.mark.parametrize("Hq,Hkv,bs", [(8, 2, 16), (8, 1, 24), (4, 4, 128), (6, 3, 64), (8, 1, 1), (8, 2, 192)])
def test_decode(bi, Hq, Hkv, bs, W, S):
    c = Case([1, 2, 127, 128, 129, 255, 257, 384, 700, 1300], [1] * 10, Hq, Hkv, bs, seed=W + S)
    assert_close_rel(f64_of(c.decode(bi, W, S)), c.reference(W, S), RTOL, ATOL, f"W={W} S={S}")
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("B", [1, 3, 40])                               # chunks in clusters, an item a CTA, the ring
@pytest.mark.parametrize("W,S", [(1920, 0), (1900, 5), (4000, 0), (6000, 300)])
def test_decode_long(bi, B, W, S):
    """Sixteen chunks and more (a cluster holds sixteen); the sequences' bits are those of each alone."""
    import torch
    c = Case([6000, 4100, 2049][:B] + [130] * (B - 3), [1] * B, 8, 2, 16, seed=W + S)
    got = c.decode(bi, W, S)
    for b in range(min(B, 4)):
        one = c.decode(bi, W, S, Q=c.Q[b:b + 1], table=c.table[b:b + 1].contiguous(), lens=c.len_t[b:b + 1], max_len=c.lens[b])
        assert torch.equal(one[0], got[b])
    if B < 40:
        assert_close_rel(f64_of(got), c.reference(W, S), RTOL, ATOL)
        cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        assert torch.equal(got, c.tiled(bi, W, S, cu=cu)) and torch.equal(got, c.extend(bi, W, S, cu=cu))
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("W,S", WINDOWS)
@pytest.mark.parametrize("Hq,Hkv,bs", [(8, 2, 16), (8, 1, 24), (8, 2, 20), (4, 4, 128), (6, 3, 64)])
def test_extend(bi, Hq, Hkv, bs, W, S):
    c = Case([1, 128, 300, 513, 40], [1, 128, 200, 33, 0], Hq, Hkv, bs, seed=W + S + 1)
    got = c.extend(bi, W, S)
    assert_close_rel(f64_of(got), c.reference(W, S), RTOL, ATOL, f"W={W} S={S}")
    import torch
    assert torch.equal(got, c.cut(bi, W, S))                            # and decode's bits, token by token
    assert torch.equal(got, c.tiled(bi, W, S))
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("B", [3, 60])                                  # one item a CTA, the ring
def test_a_window_that_holds_everything_changes_no_bit(bi, B):
    import torch
    r = syn.rng(B, 0)
    c = Case(r.integers(1, 900, B), [1] * B, 32, 8, 16, seed=B)
    plain = bi.attention_decode(c.Q, c.K, c.V, c.table, c.len_t, c.max_len, SCALE)
    for W, S in ((max(c.lens), 0), (1 << 30, 5), (1, c.max_len), (40, 1 << 30), (1 << 40, 1 << 40)):
        assert torch.equal(c.decode(bi, W, S), plain)
    c = Case([700, 130, 64], [400, 1, 64], 32, 8, 16, seed=1)
    plain = bi.attention_extend(c.Q, c.cu, c.K, c.V, c.table, c.len_t, c.max_len, 400, SCALE)
    for W, S in ((700, 0), (1 << 31, 7), (1, 700)):
        assert torch.equal(c.extend(bi, W, S), plain) and torch.equal(c.tiled(bi, W, S), plain)
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("Hq,Hkv,bs", [(16, 4, 16), (4, 4, 24), (16, 2, 64), (8, 2, 12)])
@pytest.mark.parametrize("W,S", [(200, 5), (1000, 0)])
def test_prompts_and_single_tokens_in_one_batch(bi, Hq, Hkv, bs, W, S):
    """Sequences of a few tokens go to the split, the others to the tiles, in one call (all to one of them by other
    numbers); a generous most costs nothing."""
    import torch
    r = syn.rng(W, 7)
    for q in ([1] * 30 + [1000, 3, 0, 8] + [1] * 27, [700, 1, 900, 3, 1, 0, 64, 17], [2, 90, 1]):
        c = Case([int(x) + int(r.integers(0, 300)) + (x == 0) for x in q], q, Hq, Hkv, bs, seed=W)
        got = c.extend(bi, W, S)
        assert torch.equal(got, c.tiled(bi, W, S)) and torch.equal(got, c.extend(bi, W, S, max_q=100000))
        rows = np.unique(np.concatenate([np.arange(0, len(got), 29), np.arange(min(len(got), 40)), np.arange(max(0, len(got) - 40), len(got))]))
        assert torch.equal(got[torch.from_numpy(rows).cuda()], c.cut(bi, W, S, tokens=rows))
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("W,S", [(100, 4), (300, 0), (128, 200)])
def test_tokens_do_not_depend_on_the_batch(bi, W, S):
    import torch
    c = Case([900, 33, 400, 1, 777, 640], [500, 33, 7, 1, 130, 64], 16, 4, 16, seed=5)
    whole = c.extend(bi, W, S)
    for b, (n, q) in enumerate(zip(c.lens, c.q)):
        rows = slice(int(c.cu_np[b]), int(c.cu_np[b + 1]))
        done = 0
        for piece in (1, q // 3, q - 1 - q // 3):                       # in pieces, alone, with another maximum length
            piece = min(piece, q - done)
            if piece <= 0:
                continue
            got = c.extend(bi, W, S, Q=c.Q[rows][done:done + piece].contiguous(), cu=torch.tensor([0, piece], dtype=torch.int32, device="cuda"),
                           table=c.table[b:b + 1].contiguous(), lens=torch.tensor([n - q + done + piece], dtype=torch.int32, device="cuda"),
                           max_q=piece, max_len=n + 5000 * b if b < 2 else n)
            assert torch.equal(got, whole[rows][done:done + piece]), (b, done)
            done += piece
    many = Case([c.lens[0]] * 50, [1] * 50, 16, 4, 16, seed=6)
    out = many.decode(bi, W, S)
    for b in (0, 17, 49):
        one = many.decode(bi, W, S, Q=many.Q[b:b + 1], table=many.table[b:b + 1].contiguous(), lens=many.len_t[b:b + 1])
        assert torch.equal(one[0], out[b])
    assert torch.equal(many.decode(bi, W, S, max_len=100000), out)      # a generous maximum length
    assert bi.device_status() == bi.BI_OK


def hide(c, W, S, value):
    """The caches with `value` wherever no new token looks, and the table with -1 for blocks that hold nothing in sight."""
    seen = np.zeros(c.Kb.shape[:2], bool)
    table = c.table_np.copy()
    for b, (n, q) in enumerate(zip(c.lens, c.q)):
        j = np.arange(n)
        live = (j > n - q - W) | (j < S) if q else np.zeros(n, bool)
        seen[c.table_np[b][j[live] // c.bs], j[live] % c.bs] = True
        for i in range(table.shape[1]):
            if not live[i * c.bs:(i + 1) * c.bs].any():
                table[b, i] = -1 - i
    import torch
    m = to_dev(seen)[:, :, None, None]
    v = torch.tensor(value, dtype=torch.bfloat16, device="cuda")
    return torch.where(m, c.K, v), torch.where(m, c.V, v), to_dev(table)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3.0e38])
@pytest.mark.parametrize("W,S,bs", [(100, 4, 16), (300, 0, 24), (200, 5, 20), (130, 129, 128), (17, 3, 256), (64, 5, 8)])
def test_what_is_out_of_sight_has_no_effect(bi, value, W, S, bs):
    import torch
    for lens, q in (([700, 129, 3, 1290], [1] * 4), ([700, 129, 3, 1290] * 30, [1] * 120), ([700, 129, 3, 1290], [150, 2, 3, 1])):
        c = Case(lens, q, 8, 2, bs, seed=W)
        K, V, table = hide(c, W, S, value)
        call = c.decode if max(q) == 1 else c.extend
        assert torch.equal(call(bi, W, S, K=K, V=V, table=table), call(bi, W, S))
        if max(q) > 1:
            assert torch.equal(c.tiled(bi, W, S, K=K, V=V, table=table), c.tiled(bi, W, S))
        assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (8, 4), (8, 2), (8, 1)])
def test_values_that_are_not_finite_reach_only_tokens_that_see_them(bi, Hq, Hkv):
    """Infinities and NaN among the tokens of an extend call: each token is what decode of its cut sequence gives; the
    ones that do not see them have the clean bits."""
    import torch
    W, S = 140, 6
    c = Case([500, 90], [330, 90], Hq, Hkv, 16, seed=Hkv)
    clean = c.extend(bi, W, S)
    K, V = c.K.clone(), c.V.clone()
    at = [(0, 2, V, 5, "nan"), (0, 260, V, 77, "inf"), (0, 261, V, 127, "-inf"), (0, 388, K, 3, "nan"), (1, 0, V, 64, "inf"), (1, 40, K, 9, "nan")]
    hit = np.zeros((len(clean), Hkv), bool)
    for b, j, t, d, x in at:
        h = (j + d) % Hkv
        t[c.table_np[b, j // 16], j % 16, h, d] = float(x)
        p = np.arange(c.lens[b] - c.q[b], c.lens[b])
        hit[c.cu_np[b]:c.cu_np[b + 1], h] |= (j <= p) & ((j > p - W) | (j < S))
    cut = c.cut(bi, W, S, K=K, V=V).float()
    rows = torch.from_numpy(np.repeat(hit, Hq // Hkv, axis=1)).cuda()
    for got in (c.extend(bi, W, S, K=K, V=V), c.tiled(bi, W, S, K=K, V=V)):
        assert torch.equal(torch.nan_to_num(got.float(), nan=123.0), torch.nan_to_num(cut, nan=123.0))
        assert torch.equal(got[~rows], clean[~rows])
        assert not torch.isfinite(got.float()[rows]).all(-1).any()
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("Hq,bs", [(8, 16), (16, 64), (32, 16), (64, 128), (32, 24), (32, 20), (8, 1)])
@pytest.mark.parametrize("W,S", [(130, 5), (1 << 30, 0)])
def test_many_sequences_of_drafts(bi, Hq, bs, W, S):
    """Up to 32 query rows a KV head and more than 40 (sequence, 16 rows, KV head, chunk) an SM: two tiles of 16 rows at
    once. Every token has decode's bits, also where some of its neighbours see values that are not finite."""
    import torch
    most = 32 // (Hq // 8)
    c = Case([300, 129, 40, 256, 299] * 20, [most, most - 1, 1, most // 2 + 1, 0] * 20, Hq, 8, bs, seed=Hq)
    for value in (None, "nan", "-inf"):
        V = c.V.clone()
        if value:
            for b, j in ((0, 297), (1, 128), (3, 120), (5, 299), (10, 0), (10, 170), (15, 299 - W % 128)):
                j = min(j, c.lens[b] - 1)
                V[c.table_np[b, j // bs], j % bs, b % 8, (37 * j) % D] = float(value)
        cut = torch.nan_to_num(c.cut(bi, W, S, V=V).float(), nan=123.0)
        for got in (c.extend(bi, W, S, V=V, max_len=20000), c.extend(bi, W, S, V=V), c.tiled(bi, W, S, V=V)):
            assert torch.equal(torch.nan_to_num(got.float(), nan=123.0), cut)
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("bs", [16, 24, 20])
def test_blocks_outside_the_cache(bi, bs):
    """A block in sight that lies outside: its tokens count nothing, also where it holds all that a token sees of a chunk."""
    import torch
    W, S = 150, 5
    c = Case([600, 600, 40], [40, 1, 2], 8, 2, bs, seed=bs)
    table = c.table_np.copy()
    bad = [(0, 0), (0, 580 // bs), (1, 0), (2, 0)] + [(1, i) for i in range(-(-512 // bs) * 0 + 460 // bs, 512 // bs)]
    for n, (b, i) in enumerate(bad):
        table[b, i] = [-1, 1 << 30, c.K.shape[0]][n % 3]
    got = c.extend(bi, W, S, table=to_dev(table))
    assert bi.device_status() == bi.BI_ERR_INVALID_ARG
    assert torch.equal(torch.nan_to_num(c.tiled(bi, W, S, table=to_dev(table)).float(), nan=9.0), torch.nan_to_num(got.float(), nan=9.0))
    assert bi.device_status() == bi.BI_ERR_INVALID_ARG
    old, c.table = c.table, to_dev(table)
    cut = c.cut(bi, W, S)
    c.table = old
    assert bi.device_status() == bi.BI_ERR_INVALID_ARG
    assert torch.equal(torch.nan_to_num(got.float(), nan=9.0), torch.nan_to_num(cut.float(), nan=9.0))
    out = 0
    for b in range(3):
        k, v = c.rows(b)
        for i in range(c.q[b]):
            p = c.lens[b] - c.q[b] + i
            j = np.arange(p + 1)
            j = j[((j > p - W) | (j < S)) & ~np.isin(j // bs, [x for s, x in bad if s == b])]
            row = f64_of(got[out])
            if len(j) == 0:
                assert np.isnan(row).all()
            else:
                q = syn.bf16_bits_to_f32(c.Qb[out]).astype(np.float64)
                s = np.einsum("jhd,hgd->hgj", k[j], q.reshape(2, 4, D)) * SCALE
                e = np.exp(s - s.max(-1, keepdims=True))
                want = (np.einsum("hgj,jhd->hgd", e, v[j]) / e.sum(-1, keepdims=True)).reshape(8, D)
                assert_close_rel(row, want, RTOL, ATOL, f"{b} {i}")
            out += 1


def test_sequences_out_of_range_are_left_as_they_were(bi):
    import torch
    c = Case([300, 200, 100, 64], [1, 1, 1, 1], 8, 2, 16, seed=3)
    want = c.decode(bi, 50, 4)
    lens = torch.tensor([300, 0, 301, 64], dtype=torch.int32, device="cuda")
    O = torch.full_like(want, 7.0)
    c.decode(bi, 50, 4, lens=lens, O=O)
    assert bi.device_status() == bi.BI_ERR_INVALID_ARG
    assert torch.equal(O[[0, 3]], want[[0, 3]]) and (O[[1, 2]] == 7.0).all()
    c = Case([300, 200, 100], [20, 30, 5], 8, 2, 16, seed=4)
    want = c.extend(bi, 50, 4)
    Q = torch.cat([c.Q, c.Q[:5]])
    keep = torch.tensor(list(range(20)) + list(range(50, 55)), device="cuda")
    for call in (c.extend, c.tiled):
        O = torch.full((60, 8, D), 7.0, dtype=torch.bfloat16, device="cuda")
        call(bi, 50, 4, Q=Q, O=O, lens=torch.tensor([300, 29, 100], dtype=torch.int32, device="cuda"))
        assert bi.device_status() == bi.BI_ERR_INVALID_ARG
        assert torch.equal(O[keep], want[keep]) and (O[20:50] == 7.0).all() and (O[55:] == 7.0).all()   # rows behind the last one stay


def test_a_cache_past_2_31(bi):
    """Blocks whose offsets pass 32 bits."""
    import torch
    Hkv, bs = 8, 16
    blocks = (1 << 31) // (Hkv * bs * D) + 200
    c = Case([500, 260], [40, 1], 8, Hkv, bs, seed=9)
    K = torch.zeros((blocks, bs, Hkv, D), dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    n = c.K.shape[0]
    K[blocks - n:], V[blocks - n:] = c.K, c.V
    table = c.table + (blocks - n)
    assert torch.equal(c.extend(bi, 200, 3, K=K, V=V, table=table), c.extend(bi, 200, 3))
    assert torch.equal(c.tiled(bi, 200, 3, K=K, V=V, table=table), c.extend(bi, 200, 3))
    assert torch.equal(c.cut(bi, 200, 3), c.extend(bi, 200, 3))
    old, c.table = c.table, table
    assert torch.equal(c.cut(bi, 200, 3, K=K, V=V), c.extend(bi, 200, 3, K=K, V=V))
    c.table = old
    assert bi.device_status() == bi.BI_OK


def test_captured_on_streams_and_with_workspaces(bi):
    import torch
    c = Case([700, 300, 9], [1, 1, 1], 8, 2, 16, seed=2)
    W, S = 200, 4
    size = bi.attention_decode_window_workspace_size(3, 8, 700, W, S)
    assert 0 < size <= bi.attention_decode_workspace_size(3, 8, 700)
    assert size == bi.attention_decode_window_workspace_size(3, 8, 70000, W, S)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    want, O = c.decode(bi, W, S), torch.zeros_like(c.Q)
    c.decode(bi, W, S, ws=ws, O=O)
    assert torch.equal(O, want) and (ws[size:] == 0xFF).all()
    with pytest.raises(bi.BiError):
        c.decode(bi, W, S, ws=ws[:size - 16])
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        c.decode(bi, W, S, ws=ws, O=O)
        c.extend(bi, W, S, O=O, Q=O.clone())
    O.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(O, c.extend(bi, W, S, Q=want))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = bi.attention_decode_window(c.Q, c.K, c.V, c.table, c.len_t, 700, SCALE, W, S, stream=other)
    other.synchronize()
    assert torch.equal(got, want) and bi.device_status() == bi.BI_OK


def test_two_streams_and_a_capture_that_forks(bi):
    """Calls of both forms on two streams at once, with their own workspaces, eager and from a captured graph."""
    import torch
    W, S = 180, 3
    cases = [Case([700, 50, 1300], [1, 1, 1], 8, 2, 16, seed=1), Case([900, 400, 64], [300, 5, 1], 8, 2, 16, seed=2)]
    want = [cases[0].decode(bi, W, S), cases[1].extend(bi, W, S)]
    sizes = [bi.attention_decode_window_workspace_size(3, 8, 1300, W, S), bi.attention_extend_window_workspace_size(306, 8, 2, 900, 300, W, S)]
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    outs = [torch.zeros_like(w) for w in want]
    side = [torch.cuda.Stream() for _ in range(2)]

    def both():
        here = torch.cuda.current_stream()
        for s, call, c, w, o in zip(side, (Case.decode, Case.extend), cases, ws, outs):
            s.wait_stream(here)
            with torch.cuda.stream(s):
                for _ in range(3):
                    call(c, bi, W, S, ws=w, O=o)
            here.wait_stream(s)

    both()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        both()
    for _ in range(3):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert bi.device_status() == bi.BI_OK


def test_from_projection_to_attention(bi):
    """A model's layer as it is served: projection, append with norms and rotation, attention; a prompt in two chunks, then
    single tokens, against the plain form of the whole in 64 bits."""
    import torch
    Hq, Hkv, bs, W, S, T = 8, 2, 16, 60, 3, 150
    H, R = 256, 64
    x = to_dev_bf16(syn.to_bf16_bits(syn.normal_rows(1, 0, T, H)))
    Wqkv = to_dev_bf16(syn.to_bf16_bits(0.06 * syn.normal_rows(1, 1, (Hq + 2 * Hkv) * D, H)))
    qw, kw = (to_dev_bf16(syn.to_bf16_bits(0.5 + syn.rng(1, s).random(D).astype(np.float32))) for s in (5, 6))
    fr = bi.rope_freqs(R, base=10000.0, interleaved=True, scaling="linear", scale=2.0)
    K = torch.zeros((14, bs, Hkv, D), dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    table = torch.randperm(14, device="cuda")[:10].to(torch.int32).view(1, 10)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    outs = []
    for lo, hi in [(0, 70), (70, 140)] + [(t, t + 1) for t in range(140, T)]:
        pos = torch.arange(lo, hi, device="cuda")
        qkv = bi.gemm_bf16(x[lo:hi], Wqkv).view(hi - lo, Hq + 2 * Hkv, D)
        slots = table[0].long()[pos // bs] * bs + pos % bs
        q = bi.kv_append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], slots, K, V, pos, fr, k_weight=kw, Q=qkv[:, :Hq], q_weight=qw)
        if hi - lo > 1:
            outs.append(bi.attention_extend_window(q, i32(0, hi - lo), K, V, table, i32(hi), T, hi - lo, SCALE, W, S))
        else:
            outs.append(bi.attention_decode_window(q, K, V, table, i32(hi), T, SCALE, W, S))
    got = torch.cat(outs)
    assert bi.device_status() == bi.BI_OK
    # one call over the whole prompt: the same bits
    qkv = bi.gemm_bf16(x, Wqkv).view(T, Hq + 2 * Hkv, D)
    Q, Kr = bi.qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qw, kw, 1e-6, torch.arange(T, device="cuda"), fr)
    assert torch.equal(K.view(-1, Hkv, D)[table[0].long()[torch.arange(T) // bs] * bs + torch.arange(T, device="cuda") % bs], Kr)
    assert torch.equal(bi.attention_extend_window(Q, i32(0, T), K, V, table, i32(T), T, T, SCALE, W, S), got)
    # plain, from the projection's bf16 rows, the cache rounded to bf16 as it is held
    rows = f64_of(qkv)
    angle = np.outer(np.arange(T), ref.freqs(R, 10000.0, "linear", 2.0)[0])
    bf = lambda a: syn.bf16_bits_to_f32(syn.to_bf16_bits(a.astype(np.float32))).astype(np.float64)
    q = bf(ref.turn(ref.norm(rows[:, :Hq], f64_of(qw), 1e-6), angle, True, 1.0)[0])
    k = bf(ref.turn(ref.norm(rows[:, Hq:Hq + Hkv], f64_of(kw), 1e-6), angle, True, 1.0)[0])
    want = ref.attention(q, k, rows[:, Hq + Hkv:], T, W, S, SCALE)
    # a rounding of q or k to the other side (2^-8 of one element) moves a score by at most 2^-8 |q_d k_d| SCALE: on top
    # of the attention's own tolerance 2^-8 * max|q| max|k| * SCALE * (max|v| + |out|)
    extra = 2.0 ** -8 * np.abs(q).max() * np.abs(k).max() * SCALE * (np.abs(rows[:, Hq + Hkv:]).max() + np.abs(want).max())
    assert_close_rel(f64_of(got), want, RTOL, ATOL + extra)


def test_refusals(bi):
    import torch
    c = Case([64, 32], [1, 1], 8, 2, 16)
    for name, call in (("Q", lambda o: c.decode(bi, 5, 0, Q=o)), ("K_cache", lambda o: c.decode(bi, 5, 0, K=o)), ("V_cache", lambda o: c.extend(bi, 5, 0, V=o)),
                       ("block_table", lambda o: c.decode(bi, 5, 0, table=o)), ("seq_lens", lambda o: c.extend(bi, 5, 0, lens=o)),
                       ("cu_q", lambda o: c.extend(bi, 5, 0, cu=o)), ("workspace", lambda o: c.decode(bi, 5, 0, ws=o)), ("O", lambda o: c.extend(bi, 5, 0, O=o))):
        for other in ([1], torch.zeros((2, 8, 128), device="cuda"), c.Q.cpu()):
            with pytest.raises(TypeError, match=name):
                call(other)
    for W, S in ((0, 0), (-1, 0), (1, -1), (-(1 << 40), 0), (5, -(1 << 40))):
        for call in (c.decode, c.extend):
            with pytest.raises(bi.BiError):
                call(bi, W, S)
        assert bi.attention_decode_window_workspace_size(2, 8, 64, W, S) == -1 == bi.attention_extend_window_workspace_size(2, 8, 2, 64, 1, W, S)
    with pytest.raises(TypeError):
        c.decode(bi, 5.0, 0)
    for n in (0, -1, (1 << 30) + 1, 1 << 31, (1 << 32) + 64):
        for call in (c.decode, c.extend):
            with pytest.raises(bi.BiError):
                call(bi, 5, 0, max_len=n)
    assert torch.equal(c.extend(bi, 5, 0, max_q=(1 << 32) + 1), c.extend(bi, 5, 0))
    with pytest.raises(ValueError):
        c.decode(bi, 5, 0, V=c.V[:2])
    with pytest.raises(ValueError):
        c.decode(bi, 5, 0, lens=c.len_t[:1], table=c.table[:1].contiguous())
    with pytest.raises(ValueError):
        c.extend(bi, 5, 0, cu=c.cu[:2].contiguous())
    with pytest.raises(ValueError):
        c.decode(bi, 5, 0, K=c.K.transpose(1, 2))
    empty = torch.empty((0, 8, 128), dtype=torch.bfloat16, device="cuda")
    zero = torch.empty(0, dtype=torch.int32, device="cuda")
    assert c.decode(bi, 5, 0, Q=empty, table=c.table[:0], lens=zero).shape == (0, 8, 128)
    assert c.extend(bi, 5, 0, Q=empty, cu=torch.zeros(3, dtype=torch.int32, device="cuda")).shape == (0, 8, 128)
    assert bi.device_status() == bi.BI_OK
