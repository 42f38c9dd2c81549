"""Attention over the 4-bit cache where scores leave the ordinary range: products that overflow, scores next to the
largest number, and blocks outside the cache beside them. Decode, extend split over the chunks, extend tiled and the
bf16 calls over the held values give the same bits, and a chunk counts nothing only for a row that sees no token of it
in the cache."""
import numpy as np
import pytest

import bi_synth as syn
from util import bits_of

pytestmark = pytest.mark.gpu
D = 128
Q0 = -34.5                           # times 7 * 2^120 (the largest held number): -3.21e38, a number; twice that is not
BIG = 7.0 * 2.0 ** 120


def make(bi, lens, bs, Hq, Hkv, special, seed):
    """Sequences of small keys, but for `special`: (sequence, token) -> how many of dimensions 0 and 32 hold BIG (1: a
    score of -3.21e38, 2: minus infinity). Every query is Q0 in those two dimensions and 0 elsewhere; the scale is 1."""
    import torch
    nb = -(-max(lens) // bs)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = len(lens) * nb * bs
    K = torch.randn((rows, Hkv, D), device="cuda", generator=g).mul_(0.05).bfloat16()
    V = torch.randn((rows, Hkv, D), device="cuda", generator=g).bfloat16()
    table = torch.randperm(len(lens) * nb, device="cuda", generator=g).int().view(len(lens), nb)
    for (b, j), n in special.items():
        slot = int(table[b, j // bs]) * bs + j % bs
        K[slot, :, 0] = BIG
        K[slot, :, 32] = BIG if n == 2 else 0.0
    cache = bi.kv_int4_cache(len(lens) * nb, bs, Hkv)
    every = torch.arange(rows, device="cuda")
    bi.kv_int4_append(K, V, every, cache)
    Kh, Vh = (t.view(-1, bs, Hkv, D) for t in bi.kv_int4_read(cache, every))
    return cache, Kh, Vh, table


def queries(n, Hq):
    import torch
    Q = torch.zeros((n, Hq, D), dtype=torch.bfloat16, device="cuda")
    Q[:, :, 0] = Q0
    Q[:, :, 32] = Q0
    return Q


def extend_forms(bi, Q, cu, cache, table, lens, top, most):
    """Extend split over the chunks and tiled."""
    import torch
    split = torch.empty(bi.attention_decode_workspace_size(Q.shape[0], Q.shape[1], top), dtype=torch.uint8, device="cuda")
    assert bi.attention_extend_int4_workspace_size(Q.shape[0], Q.shape[1], cache.k_codes.shape[1], top, most) > 0
    return [bi.attention_extend_int4(Q, cu, cache, table, lens, top, most, 1.0, workspace=ws)
            for ws in (split, torch.empty(16, dtype=torch.uint8, device="cuda"))]


@pytest.mark.parametrize("Hq,Hkv,bs", [(4, 4, 16), (4, 2, 24), (8, 2, 128), (16, 2, 1)])
def test_overflowing_scores_are_the_bf16_calls(bi, Hq, Hkv, bs):
    import torch
    # a last chunk of one token that overflows; a sole token that does; a sole token with a score of -3.21e38; three of
    # them; a last chunk of them; an ordinary sequence; an overflowing token among ordinary ones
    lens = [129, 1, 1, 3, 131, 140, 130]
    special = {(0, 128): 2, (1, 0): 2, (2, 0): 1, (3, 0): 1, (3, 1): 1, (3, 2): 1, (4, 128): 1, (4, 129): 1, (4, 130): 1,
               (6, 128): 2}
    cache, Kh, Vh, table = make(bi, lens, bs, Hq, Hkv, special, seed=bs)
    ld, Q, top = torch.tensor(lens, dtype=torch.int32, device="cuda"), queries(len(lens), Hq), max(lens)
    want = bi.attention_decode(Q, Kh, Vh, table, ld, top, 1.0)
    nan = torch.isnan(want).flatten(1)
    assert nan.all(1).tolist() == [True, True] + [False] * 5 and nan.any(1).tolist() == nan.all(1).tolist()
    assert np.array_equal(bits_of(bi.attention_decode_int4(Q, cache, table, ld, top, 1.0)), bits_of(want))
    cu = torch.arange(len(lens) + 1, dtype=torch.int32, device="cuda")
    for got in extend_forms(bi, Q, cu, cache, table, ld, top, 1):
        assert np.array_equal(bits_of(got), bits_of(want))
    # two or three new tokens of each sequence that has them: the bf16 extend, and decode of the cut sequences
    qlens = [2, 1, 1, 3, 3, 2, 3]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(qlens)]), dtype=torch.int32, device="cuda")
    Q = queries(sum(qlens), Hq)
    want = bi.attention_extend(Q, cu, Kh, Vh, table, ld, top, 3, 1.0)
    assert bool(torch.isnan(want[1]).all()) and not bool(torch.isnan(want[0]).any())
    for got in extend_forms(bi, Q, cu, cache, table, ld, top, 3):
        assert np.array_equal(bits_of(got), bits_of(want))
    assert bi.device_status() == bi.BI_OK


def test_blocks_outside_the_cache_beside_extreme_scores(bi):
    """A chunk counts nothing for a row that sees only blocks outside the cache, and as it would in the bf16 calls for
    one that sees a token of the cache, whatever its score."""
    import torch
    bs, Hq, Hkv = 16, 8, 2
    lens = [150, 145, 129, 145, 40]
    # 0: chunk 1 has a bad block, and its valid tokens overflow. 1: of chunk 1, token 144 is the only one in the cache,
    # with a score of -3.21e38. 2: chunk 0 lies outside the cache, the one token of chunk 1 has a score of -3.21e38.
    # 3: an ordinary token 144 after the bad block. 4: no block in the cache.
    special = {(0, j): 2 for j in range(144, 150)} | {(1, 144): 1, (2, 128): 1}
    cache, Kh, Vh, table = make(bi, lens, bs, Hq, Hkv, special, seed=5)
    slot = table[2, 8].long() * bs
    lone = Vh.view(-1, Hkv, D)[slot].repeat_interleave(Hq // Hkv, 0)
    table[0, 8] = table[1, 8] = table[3, 8] = -1
    table[2, :8] = 1 << 30
    table[4] = -1
    ld, top = torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens)
    Q = queries(5, Hq)
    O = bi.attention_decode_int4(Q, cache, table, ld, top, 1.0)
    same = bi.attention_decode(Q, Kh, Vh, table, ld, top, 1.0)
    assert np.array_equal(bits_of(O[[0, 1, 3]]), bits_of(same[[0, 1, 3]]))
    assert bool(torch.isnan(O[[0, 4]]).all()) and not bool(torch.isnan(O[1:4]).any())
    assert torch.equal(O[2], lone)                       # one token: its value
    # new tokens before and behind the bad blocks' end: rows of one tile that see none or some of a chunk in the cache
    qlens = [8, 4, 3, 5, 2]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(qlens)]), dtype=torch.int32, device="cuda")
    Q = queries(sum(qlens), Hq)
    want = torch.empty_like(Q)
    for b, n in enumerate(qlens):
        for i in range(n):
            r = int(cu[b]) + i
            cut = torch.tensor([lens[b] - n + i + 1], dtype=torch.int32, device="cuda")
            want[r:r + 1] = bi.attention_decode_int4(Q[r:r + 1], cache, table[b:b + 1].contiguous(), cut, top, 1.0)
    for got in extend_forms(bi, Q, cu, cache, table, ld, top, max(qlens)):
        assert np.array_equal(bits_of(got), bits_of(want))
    assert bi.device_status() == bi.BI_ERR_INVALID_ARG
