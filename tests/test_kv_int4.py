"""The paged 4-bit K/V cache on the GPU: append against the format's definition
in 64 bits (codes, scales and packed layout exactly), read, padding and bad
slots, and decode and extend attention over it: the same bits as the bf16
calls over a bf16 cache of the held values, and parity with a plain 64-bit
form."""
import ctypes

import numpy as np
import pytest

import bi_synth as syn
import int4_ref as ref
from util import bits_of, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu
D = 128
SCALE = D ** -0.5


def rows(T, Hkv, seed, std=1.0):
    return syn.to_bf16_bits(std * syn.normal_rows(seed, 0, T, Hkv * D)).reshape(T, Hkv, D)


def special_rows(Hkv):
    """Rows at the format's edges: zeros, ties, one loud value, extremes, subnormals, infinities and NaN."""
    x = np.zeros((12, Hkv, D), np.float32)
    x[1] = np.tile(np.arange(-16, 16) * 0.5, 4)[None]              # amax 8: ties against s = 1.25 among them
    x[2] = np.tile(np.concatenate([[7.0], np.arange(31) * 0.25 - 4]), 4)[None]   # s = 1: every x.5 is a tie
    x[3, :, 5] = 1e4
    x[4] = 3.0e38
    x[5] = 1e-39
    x[6] = 2.0 ** -101
    x[7] = -0.0
    x[8, :, 40] = np.inf
    x[9, :, 70] = np.nan
    x[10] = 7.0 * 2.0 ** 120
    x[11] = np.tile(2.0 ** np.arange(-16.0, 16.0), 4)[None]
    return syn.to_bf16_bits(x)


def new_cache(bi, blocks, bs, Hkv):
    """A cache whose every byte is a pattern, so that a stray write shows."""
    c = bi.kv_int4_cache(blocks, bs, Hkv)
    c.k_codes.fill_(0x5A), c.v_codes.fill_(0xA5), c.k_scales.fill_(3.0), c.v_scales.fill_(-5.0)
    return c


@pytest.mark.parametrize("T,Hkv,bs", [(1, 1, 1), (7, 8, 16), (33, 5, 24), (300, 2, 128)])
def test_append_matches_the_definition_and_touches_nothing_else(bi, T, Hkv, bs):
    K, V = rows(T, Hkv, 1), rows(T, Hkv, 2, std=0.3)
    K[: min(T, 12)] = special_rows(Hkv)[: min(T, 12)]
    V[-min(T, 12):] = special_rows(Hkv)[: min(T, 12)]
    blocks = -(-T // bs) + 2
    slots = syn.rng(3, T).permutation(blocks * bs)[:T].astype(np.int64)
    if T > 2:
        slots[1] = -1                                     # padding
    c = new_cache(bi, blocks, bs, Hkv)
    before = [t.clone() for t in c]
    assert bi.kv_int4_append(to_dev_bf16(K), to_dev_bf16(V), to_dev(slots), c) is c
    assert bi.device_status() == bi.BI_OK
    want = [t.cpu() for t in before]
    codes = [want[0].numpy(), want[2].numpy()]
    scales = [bits_of(want[1]).copy(), bits_of(want[3]).copy()]
    for which, x in enumerate((K, V)):
        n, s = ref.held(x)
        sb = syn.to_bf16_bits(np.nan_to_num(s, nan=0.0).astype(np.float32))
        sb = np.where(np.isnan(s), np.uint16(0x7FFF), sb)
        for t in range(T):
            if slots[t] >= 0:
                codes[which][slots[t] // bs, :, slots[t] % bs] = ref.pack(n[t], int(slots[t] % bs))
                scales[which][slots[t] // bs, :, slots[t] % bs] = sb[t]
    assert np.array_equal(c.k_codes.cpu().numpy(), codes[0]) and np.array_equal(c.v_codes.cpu().numpy(), codes[1])
    assert np.array_equal(bits_of(c.k_scales), scales[0]) and np.array_equal(bits_of(c.v_scales), scales[1])
    # and back: exact bf16 numbers, zeros for padding, repeated slots allowed
    again = np.concatenate([slots, slots[:1]])
    Kr, Vr = bi.kv_int4_read(c, to_dev(again))
    for got, x in ((Kr, K), (Vr, V)):
        v = ref.values(*ref.held(x))
        v[slots < 0] = 0.0
        g = got.float().cpu().numpy().astype(np.float64)
        assert np.array_equal(g[:T], v, equal_nan=True) and np.array_equal(g[T], v[0], equal_nan=True)


def test_append_takes_strided_rows_and_read_writes_them(bi):
    import torch
    T, Hkv, bs = 21, 4, 8
    qkv = to_dev_bf16(rows(T, 3 * Hkv, 5))
    K, V = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
    slots = torch.arange(T, device="cuda") + 3
    a, b = new_cache(bi, 4, bs, Hkv), new_cache(bi, 4, bs, Hkv)
    bi.kv_int4_append(K, V, slots, a)
    bi.kv_int4_append(K.contiguous(), V.contiguous(), slots, b)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))
    out = torch.full_like(qkv, 9.0)
    Kr, Vr = bi.kv_int4_read(a, slots)
    bi.kv_int4_read(a, slots, K=out[:, Hkv:2 * Hkv], V=out[:, 2 * Hkv:])
    assert torch.equal(out[:, Hkv:2 * Hkv], Kr) and torch.equal(out[:, 2 * Hkv:], Vr) and bool((out[:, :Hkv] == 9.0).all())


def test_bad_slots_are_reported_and_skipped(bi):
    import torch
    c = new_cache(bi, 2, 8, 2)
    before = [t.clone() for t in c]
    K = to_dev_bf16(rows(3, 2, 6))
    slots = torch.tensor([-1, 16, -7], device="cuda")
    bi.kv_int4_append(K, K, slots, c)
    assert bi.device_status() == bi.BI_ERR_INVALID_ARG
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(c, before))
    Kr, Vr = bi.kv_int4_read(c, slots)
    assert bi.device_status() == bi.BI_ERR_INVALID_ARG
    assert not Kr.any() and not Vr.any()
    bi.kv_int4_read(c, torch.full((5,), -1, device="cuda"))
    assert bi.device_status() == bi.BI_OK


# ---------------------------------------------------------------- attention ---

def make(bi, lens, bs, Hq, Hkv, seed, q_rows=None, max_len=None):
    """A 4-bit cache and a bf16 cache of the same held values, in blocks in a random order."""
    import torch
    lens = np.asarray(lens, np.int32)
    nb = max(1, int(-(-int(max_len or lens.max()) // bs)))
    blocks = len(lens) * nb + 2
    K, V = to_dev_bf16(rows(blocks * bs, Hkv, seed, 1.5)), to_dev_bf16(rows(blocks * bs, Hkv, seed + 1, 0.5))
    cache = bi.kv_int4_cache(blocks, bs, Hkv)
    every = torch.arange(blocks * bs, device="cuda")
    bi.kv_int4_append(K, V, every, cache)
    Kh, Vh = (t.view(blocks, bs, Hkv, D) for t in bi.kv_int4_read(cache, every))
    table = syn.rng(seed, 2).permutation(blocks)[: len(lens) * nb].astype(np.int32).reshape(len(lens), nb)
    Q = syn.to_bf16_bits(syn.normal_rows(seed, 3, (q_rows or len(lens)) * Hq, D)).reshape(-1, Hq, D)
    return to_dev_bf16(Q), cache, Kh, Vh, to_dev(table), to_dev(lens)


def host_seq(Kh, Vh, table, b, L):
    """Held keys and values of sequence b in 64 bits."""
    bs = Kh.shape[1]
    t = table.cpu().numpy()[b]
    at = [(t[j // bs], j % bs) for j in range(L)]
    k, v = Kh.float().cpu().numpy().astype(np.float64), Vh.float().cpu().numpy().astype(np.float64)
    return np.stack([k[a] for a in at]), np.stack([v[a] for a in at])


def tolerance(want, v):
    """bf16 output: one rounding (2^-8 of the value); the fp32 sums and the probabilities' 16 bits add less
    than 2^-13 of the largest value each."""
    return 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * np.abs(v).max()


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (4, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("bs", [1, 16, 24, 256])
def test_decode_is_bf16_decode_of_the_held_values(bi, Hq, Hkv, bs):
    lens = [1, 2, 127, 128, 129, 700, 16, 33]
    Q, c, Kh, Vh, table, ld = make(bi, lens, bs, Hq, Hkv, seed=10 + bs)
    got = bi.attention_decode_int4(Q, c, table, ld, 700, SCALE)
    same = bi.attention_decode(Q, Kh, Vh, table, ld, 700, SCALE)
    assert np.array_equal(bits_of(got), bits_of(same))
    for b, L in enumerate(lens):
        k, v = host_seq(Kh, Vh, table, b, L)
        want = ref.attention(Q[b:b + 1].float().cpu().numpy().astype(np.float64), k, v, SCALE)[0]
        err = np.abs(got[b].float().cpu().numpy() - want)
        assert (err <= tolerance(want, v)).all(), (b, float(err.max()))
    assert bi.device_status() == bi.BI_OK


def test_decode_long_and_many(bi):
    """More chunks than the merge takes at once, and more items than warps fit."""
    for lens, Hq, Hkv in (([5000, 8193, 40], 32, 8), ([900] * 70, 32, 8)):
        Q, c, Kh, Vh, table, ld = make(bi, lens, 16, Hq, Hkv, seed=40)
        got = bi.attention_decode_int4(Q, c, table, ld, max(lens), SCALE)
        assert np.array_equal(bits_of(got), bits_of(bi.attention_decode(Q, Kh, Vh, table, ld, max(lens), SCALE)))
        one = bi.attention_decode_int4(Q[2:3], c, table[2:3], ld[2:3], int(lens[2]), SCALE)
        assert np.array_equal(bits_of(one), bits_of(got[2:3])), "a sequence alone differs"


@pytest.mark.parametrize("Hq,Hkv,bs", [(4, 4, 16), (4, 2, 24), (32, 8, 16), (16, 2, 1)])
@pytest.mark.parametrize("lens,qlens", [([1, 40, 300], [1, 40, 17]), ([129, 513, 128, 20], [1, 200, 128, 0]),
                                        ([700, 5, 131, 4500], [5, 5, 3, 1])])     # few rows: split over the chunks
def test_extend_is_bf16_extend_and_decode_of_cut_sequences(bi, Hq, Hkv, bs, lens, qlens):
    cu = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    Q, c, Kh, Vh, table, ld = make(bi, lens, bs, Hq, Hkv, seed=60 + bs, q_rows=int(cu[-1]) + 3)
    import torch
    O = torch.full_like(Q, 7.0)
    args = (table, ld, max(lens), max(qlens), SCALE)
    bi.attention_extend_int4(Q, to_dev(cu), c, *args, O=O)
    same = bi.attention_extend(Q, to_dev(cu), Kh, Vh, *args)
    tiled = bi.attention_extend_int4(Q, to_dev(cu), c, *args, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert np.array_equal(bits_of(tiled[:cu[-1]]), bits_of(same[:cu[-1]]))
    assert np.array_equal(bits_of(O[:cu[-1]]), bits_of(same[:cu[-1]]))
    assert bool((O[cu[-1]:] == 7.0).all()), "rows behind the last sequence were written"
    for b in range(len(lens)):
        for i in sorted({0, qlens[b] // 2, qlens[b] - 1}):
            if 0 <= i < qlens[b]:
                cut = torch.tensor([lens[b] - qlens[b] + i + 1], dtype=torch.int32, device="cuda")
                row = int(cu[b]) + i
                one = bi.attention_decode_int4(Q[row:row + 1], c, table[b:b + 1], cut, max(lens), SCALE)
                assert np.array_equal(bits_of(one), bits_of(O[row:row + 1])), (b, i)
        if qlens[b]:
            k, v = host_seq(Kh, Vh, table, b, lens[b])
            q = Q[int(cu[b]):int(cu[b + 1])].float().cpu().numpy().astype(np.float64)
            want = ref.attention(q, k, v, SCALE, causal_from=lens[b] - qlens[b])
            err = np.abs(O[int(cu[b]):int(cu[b + 1])].float().cpu().numpy() - want)
            assert (err <= tolerance(want, v)).all(), (b, float(err.max()))
    assert bi.device_status() == bi.BI_OK


def test_bad_lengths_and_blocks(bi):
    """Lengths out of range leave their rows as they were; blocks outside the cache, even a whole chunk of them,
    count nothing; both are reported, and the other sequences keep their bits."""
    import torch
    lens = [300, 200, 40, 300]
    Q, c, Kh, Vh, table, ld = make(bi, lens, 128, 8, 2, seed=80)
    good = bi.attention_decode_int4(Q, c, table, ld, 300, SCALE)
    bad_len, bad_tab = ld.clone(), table.clone()
    bad_len[2] = 0
    bad_tab[0, 0] = -1                                    # the first chunk of sequence 0
    bad_tab[3, 1] = 1 << 30                               # the second of sequence 3
    O = torch.full_like(Q, 7.0)
    bi.attention_decode_int4(Q, c, bad_tab, bad_len, 300, SCALE, O=O)
    assert bi.device_status() == bi.BI_ERR_INVALID_ARG
    assert np.array_equal(bits_of(O[1]), bits_of(good[1])) and bool((O[2] == 7.0).all())
    for b, keep in ((0, range(128, 300)), (3, [*range(128), *range(256, 300)])):
        k, v = host_seq(Kh, Vh, table, b, 300)
        k, v = k[list(keep)], v[list(keep)]
        want = ref.attention(Q[b:b + 1].float().cpu().numpy().astype(np.float64), k, v, SCALE)[0]
        assert (np.abs(O[b].float().cpu().numpy() - want) <= tolerance(want, v)).all()
    cu = torch.arange(5, dtype=torch.int32, device="cuda")
    E = torch.full_like(Q, 7.0)
    for ws in (None, torch.empty(16, dtype=torch.uint8, device="cuda")):      # split over the chunks, and tiled
        E.fill_(7.0)
        bi.attention_extend_int4(Q, cu, c, bad_tab, bad_len, 300, 1, SCALE, workspace=ws, O=E)
        assert bi.device_status() == bi.BI_ERR_INVALID_ARG
        assert np.array_equal(bits_of(E), bits_of(O))


def test_non_finite_rows_show(bi):
    """A key or value group with an infinity or a NaN reads as NaN, and reaches the outputs that see it."""
    import torch
    lens = [50, 50]
    Q, c, Kh, Vh, table, ld = make(bi, lens, 16, 4, 2, seed=90)
    x = torch.zeros((1, 2, D), dtype=torch.bfloat16, device="cuda")
    x[0, 1, 3] = float("inf")
    slot = table[0, 1].long() * 16 + 2
    zero = torch.zeros_like(x)
    bi.kv_int4_append(zero, x, slot.reshape(1), c)
    O = bi.attention_decode_int4(Q, c, table, ld, 50, SCALE)
    nan = torch.isnan(O)
    assert bool(nan[0, 2:, :32].all()) and not bool(nan[0, 2:, 32:].any()) and not bool(nan[0, :2].any())
    assert not bool(nan[1].any())


def test_refusals():
    """Binding and ABI refuse what the kernels do not take (before any launch)."""
    import invariant_deterministic_bi_gb300 as bi
    import torch
    c = bi.kv_int4_cache(4, 16, 2)
    K = torch.zeros((3, 2, D), dtype=torch.bfloat16, device="cuda")
    s = torch.arange(3, device="cuda")
    with pytest.raises(TypeError):
        bi.kv_int4_append(K.float(), K, s, c)
    with pytest.raises(TypeError):
        bi.kv_int4_append(K, K, s.int(), c)
    with pytest.raises(ValueError):
        bi.kv_int4_append(K[:2], K, s, c)
    with pytest.raises(ValueError):
        bi.kv_int4_append(K.transpose(0, 1).contiguous().transpose(0, 1), K, s, c)     # heads apart
    with pytest.raises(ValueError):
        bi.KVInt4Cache(c.k_codes[..., :32].contiguous(), c.k_scales, c.v_codes, c.v_scales)
    with pytest.raises((TypeError, ValueError)):
        bi.kv_int4_append(K.cpu(), K, s, c)
    with pytest.raises(TypeError):
        bi.kv_int4_append(K, K, s, tuple(c))
    with pytest.raises(AttributeError):
        c.k_codes = c.v_codes
    base = torch.zeros(3 * 2 * D + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(bi.BiError) as e:
        bi.kv_int4_append(base[4:].view(3, 2, D), K, s, c)                           # 8-byte aligned rows
    assert e.value.status == bi.BI_ERR_MISALIGNED
    Q = torch.zeros((2, 6, D), dtype=torch.bfloat16, device="cuda")
    t, ln = torch.zeros((2, 1), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    with pytest.raises(bi.BiError) as e:
        bi.attention_decode_int4(Q, c, t, ln, 16, SCALE)                             # three heads a KV head
    assert e.value.status == bi.BI_ERR_UNSUPPORTED
    with pytest.raises(bi.BiError) as e:
        bi.attention_decode_int4(Q[:, :4].contiguous(), c, t, ln, 16, SCALE,
                                 workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == bi.BI_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        bi.attention_decode_int4(Q[:, :4], c, t, ln, 16, SCALE)                      # not contiguous
    with pytest.raises(ValueError):
        bi.attention_extend_int4(Q, ln, c, t, ln, 16, 1, SCALE)                      # cu_q of B entries
    assert bi.device_status() == bi.BI_OK


def test_step_in_a_graph_and_on_a_side_stream(bi):
    """qkv projection -> append -> decode -> output projection as a captured step, replayed with new inputs, and the
    same calls on another stream: the eager bits."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    B, Hq, Hkv, bs, H = 3, 8, 2, 16, 256
    W1 = torch.randint(0, 256, ((Hq + 2 * Hkv) * D, H // 2), dtype=torch.uint8, device="cuda", generator=g)
    S1 = (0.02 * torch.rand((W1.shape[0], H // 64), device="cuda", generator=g)).bfloat16()
    W2 = torch.randint(0, 256, (H, Hq * D // 2), dtype=torch.uint8, device="cuda", generator=g)
    S2 = (0.02 * torch.rand((H, Hq * D // 128), device="cuda", generator=g)).bfloat16()
    table = torch.arange(B * 4, dtype=torch.int32, device="cuda").view(B, 4)
    ws = torch.empty(bi.attention_decode_workspace_size(B, Hq, 64), dtype=torch.uint8, device="cuda")
    x = torch.empty((B, H), dtype=torch.bfloat16, device="cuda")
    lens = torch.ones(B, dtype=torch.int32, device="cuda")

    def step(cache, stream=None):
        qkv = bi.gemm_int4(x, W1, S1, stream=stream).view(B, -1, D)
        slots = table.long().gather(1, ((lens - 1) // bs).long()[:, None])[:, 0] * bs + (lens - 1) % bs
        bi.kv_int4_append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], slots, cache, stream=stream)
        o = bi.attention_decode_int4(qkv[:, :Hq].contiguous(), cache, table, lens, 64, SCALE, workspace=ws, stream=stream)
        return bi.gemm_int4(o.view(B, -1), W2, S2, stream=stream)

    xs = [torch.randn((B, H), device="cuda", generator=g).bfloat16() for _ in range(20)]
    cache = bi.kv_int4_cache(B * 4, bs, Hkv)
    want = []
    for i, xi in enumerate(xs):
        x.copy_(xi), lens.fill_(i + 1)
        want.append(step(cache).clone())
    side = torch.cuda.Stream()
    cache = bi.kv_int4_cache(B * 4, bs, Hkv)
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph):
        out = step(cache)
    torch.cuda.current_stream().wait_stream(side)
    for i, xi in enumerate(xs):
        x.copy_(xi), lens.fill_(i + 1)
        graph.replay()
        assert torch.equal(out, want[i]), i
    cache = bi.kv_int4_cache(B * 4, bs, Hkv)
    torch.cuda.synchronize()
    for i, xi in enumerate(xs[:4]):
        with torch.cuda.stream(side):
            x.copy_(xi), lens.fill_(i + 1)
            got = step(cache, stream=side)
        side.synchronize()
        assert torch.equal(got, want[i]), i
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("Hq,Hkv,bs", [(4, 4, 16), (4, 2, 24), (8, 2, 1), (16, 2, 8)])
def test_non_finite_rows_reach_only_the_tokens_that_see_them(bi, Hq, Hkv, bs):
    """Among the new tokens some values and keys are infinite or NaN: every token still has the bits of decode of the
    sequence cut after it, split over the chunks or tiled."""
    import torch
    lens, qlens = [50, 300, 260, 9, 129], [20, 130, 7, 9, 3]
    Q, c, Kh, Vh, table, ld = make(bi, lens, bs, Hq, Hkv, seed=91, q_rows=sum(qlens))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(qlens)]), dtype=torch.int32, device="cuda")
    bad = float("nan"), float("inf"), -float("inf")
    for b, (L, n) in enumerate(zip(lens, qlens)):      # new tokens 1, 4, 5 and, where there are more, 17, 100 and the last
        for i, j in enumerate(t for t in (1, 4, 5, 17, 100, n - 1) if t < n):
            j += L - n
            k = torch.ones((1, Hkv, D), dtype=torch.bfloat16, device="cuda")
            v = k.clone()
            v[0, i % Hkv, 32 * (i % 4) + 5] = bad[i % 3]
            if i == 2:
                k[0, 0, 70] = bad[b % 3]
            bi.kv_int4_append(k, v, (table[b, j // bs].long() * bs + j % bs).reshape(1), c)
    want = torch.empty_like(Q)
    for b, (L, n) in enumerate(zip(lens, qlens)):
        for i in range(n):
            cut = torch.tensor([L - n + i + 1], dtype=torch.int32, device="cuda")
            r = int(cu[b]) + i
            want[r:r + 1] = bi.attention_decode_int4(Q[r:r + 1], c, table[b:b + 1].contiguous(), cut, 300, SCALE)
    assert bool(torch.isnan(want).any()) and bool(torch.isfinite(want).any())
    need = bi.attention_decode_workspace_size(sum(qlens), Hq, 300)
    for ws in (torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty(16, dtype=torch.uint8, device="cuda")):
        got = bi.attention_extend_int4(Q, cu, c, table, ld, 300, max(qlens), SCALE, workspace=ws)
        assert np.array_equal(bits_of(got), bits_of(want))
    # the few new tokens of sequences 2 and 4 alone, which are split
    few = [2, 4]
    rows = torch.cat([torch.arange(int(cu[b]), int(cu[b + 1]), device="cuda") for b in few])
    cu2 = torch.tensor([0, 7, 10], dtype=torch.int32, device="cuda")
    q2, t2, l2 = Q[rows].contiguous(), table[few].contiguous(), ld[few].contiguous()
    assert bi.attention_extend_int4_workspace_size(10, Hq, Hkv, 300, 7) > 0
    got = bi.attention_extend_int4(q2, cu2, c, t2, l2, 300, 7, SCALE)
    assert np.array_equal(bits_of(got), bits_of(want[rows]))
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("exponent", [127, 127 - 98, 127 + 122])
def test_every_quotient_is_rounded_exactly(bi, exponent):
    """For each of the 128 significands of the largest magnitude, all numbers of the six binades up to it, of both signs:
    the codes and scales of the definition (ordinary magnitudes, and where the scale reaches its least and largest)."""
    groups = []
    for m in range(128):
        top = exponent << 7 | m
        below = np.arange(top - 6 * 128 + 1, top + 1).astype(np.uint16)
        below = np.concatenate([below, below | 0x8000, np.zeros(-2 * below.size % 31, np.uint16)]).reshape(-1, 31)
        groups.append(np.concatenate([np.full((below.shape[0], 1), top | (0x8000 if m & 1 else 0), np.uint16), below], 1))
    x = np.concatenate(groups)
    x = np.concatenate([x, np.zeros((-x.shape[0] % 4, 32), np.uint16)]).reshape(-1, 1, D)
    T = x.shape[0]
    c = bi.kv_int4_cache(T, 1, 1)
    slots = to_dev(np.arange(T, dtype=np.int64))
    bi.kv_int4_append(to_dev_bf16(x), to_dev_bf16(x ^ 0x8000), slots, c)
    n, s = ref.held(x)
    assert np.array_equal(bits_of(c.k_scales).reshape(T, 1, 4), syn.to_bf16_bits(s.astype(np.float32)))
    assert np.array_equal(c.k_codes.cpu().numpy().reshape(T, 1, 64), ref.pack(n, 0))
    assert np.array_equal(c.v_codes.cpu().numpy().reshape(T, 1, 64), ref.pack(-n, 0))
    assert bi.device_status() == bi.BI_OK
