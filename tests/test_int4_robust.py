"""The 4-bit operators under the conditions of a serving process: the bounds-checked debug build, first launches
inside a graph capture, caches and weights past 2^31 bytes, a generous maximum length, two streams at once, empty
calls, and a layer run as it is used."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest

import bi_synth as syn
import int4_ref as ref
from util import bits_of, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
D = 128
SCALE = D ** -0.5


def run_ops(debug):
    env = dict(os.environ)
    env.pop("BI_LIBRARY", None)
    if debug:
        env["BI_LIBRARY"] = "debug"
    r = subprocess.run([sys.executable, os.path.join(HERE, "_debug_int4_ops.py")], capture_output=True, text=True, env=env, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


def test_debug_and_release_builds_give_the_same_bits():
    from invariant_deterministic_bi_gb300 import _build
    _build.build(debug=True)
    rel, dbg = run_ops(False), run_ops(True)
    assert rel.pop("debug_build") is False and dbg.pop("debug_build") is True
    assert dbg["status"] == "BI_OK", "a bounds check failed on valid inputs"
    assert dbg == rel
    for bs in (16, 24):                                   # the split and the tiled form of extend agree
        for most in (40, 16):
            assert rel[f"extend{bs}_True_{most}"] == rel[f"extend{bs}_False_{most}"]
        assert rel[f"extend_status{bs}_True_40"] == "BI_OK" and rel[f"extend_status{bs}_True_16"] == "BI_ERR_INVALID_ARG"


_FIRST_CALLS = r"""
import sys
import torch
sys.path.insert(0, sys.argv[1])
import invariant_deterministic_bi_gb300 as bi

g = torch.Generator(device="cuda").manual_seed(5)
bf = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)
x, q, Q = bf(4, 2048), bf(2, 8, 128), bf(7, 8, 128)
W = torch.randint(0, 256, (512, 1024), dtype=torch.uint8, device="cuda", generator=g)
S = torch.rand((512, 16), device="cuda", generator=g).to(torch.bfloat16)
K, V = bf(64, 2, 128), bf(64, 2, 128)
table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
lens = torch.tensor([32, 20], dtype=torch.int32, device="cuda")
cu = torch.tensor([0, 3, 7], dtype=torch.int32, device="cuda")
slots = torch.arange(64, device="cuda")
c = bi.kv_int4_cache(4, 16, 2)


def calls():
    y = bi.gemm_int4(x, W, S)
    bi.kv_int4_append(K, V, slots, c)
    return [y, bi.gemm_int4(x.repeat(10, 1), W, S), *bi.kv_int4_read(c, slots), bi.attention_decode_int4(q, c, table, lens, 32, 0.1),
            bi.attention_extend_int4(Q, cu, c, table, lens, 32, 4, 0.1)]


graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
side.wait_stream(torch.cuda.current_stream())
with torch.cuda.stream(side), torch.cuda.graph(graph):
    a = calls()                        # the library's first launches
torch.cuda.current_stream().wait_stream(side)
graph.replay()
graph.replay()
torch.cuda.synchronize()
b = calls()
torch.cuda.synchronize()
assert all(torch.equal(u.view(torch.int16), v.view(torch.int16)) for u, v in zip(a, b))
assert bi.device_status() == bi.BI_OK
print("ok")
"""


def test_first_calls_of_a_process_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", _FIRST_CALLS, os.path.dirname(HERE)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-3000:]


def test_cache_past_two_gigabytes(bi):
    """Rows whose byte offsets pass 2^31 (keys and values 2.5 GB each): the same results as in a small cache."""
    import torch
    blocks, bs, Hkv, L = 300_000, 16, 8, 700
    big, small = bi.kv_int4_cache(blocks, bs, Hkv), bi.kv_int4_cache(64, bs, Hkv)
    K = to_dev_bf16(syn.to_bf16_bits(syn.normal_rows(1, 0, L, Hkv * D)).reshape(L, Hkv, D))
    j = torch.arange(L, device="cuda")
    nb = -(-L // bs)
    far = blocks - 1 - 3 * torch.arange(nb, device="cuda")
    bi.kv_int4_append(K, K, far[j // bs] * bs + j % bs, big)
    bi.kv_int4_append(K, K, j, small)
    q = to_dev_bf16(syn.to_bf16_bits(syn.normal_rows(2, 0, 32, D)).reshape(1, 32, D))
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    near = torch.arange(nb, dtype=torch.int32, device="cuda").view(1, -1)
    a = bi.attention_decode_int4(q, big, far.int().view(1, -1), lens, L, SCALE)
    assert torch.equal(a, bi.attention_decode_int4(q, small, near, lens, L, SCALE))
    Q, cu = q.repeat(200, 1, 1).contiguous(), torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    e = bi.attention_extend_int4(Q, cu, big, far.int().view(1, -1), lens, L, 200, SCALE)
    assert torch.equal(e, bi.attention_extend_int4(Q, cu, small, near, lens, L, 200, SCALE))
    for u, v in zip(bi.kv_int4_read(big, far[j // bs] * bs + j % bs), bi.kv_int4_read(small, j)):
        assert torch.equal(u, v)
    assert bi.device_status() == bi.BI_OK


def test_weights_past_two_gigabytes(bi):
    """The last rows of a 2.3 GB weight matrix equal the same rows on their own, for few and for many rows of X."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(2)
    N, K = 72_000, 65_536
    W = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    S = torch.rand((N, K // 128), device="cuda", generator=g).to(torch.bfloat16)
    for M in (2, 20):
        X = torch.randn((M, K), device="cuda", generator=g).to(torch.bfloat16)
        y = bi.gemm_int4(X, W, S)
        assert torch.equal(y[:, -64:], bi.gemm_int4(X, W[-64:].contiguous(), S[-64:].contiguous()))
    assert bi.device_status() == bi.BI_OK


def test_generous_maximum_length(bi):
    """Short sequences under a large maximum length, in a table with room for it: the same bits."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    c = bi.kv_int4_cache(40, 16, 2)
    K = torch.randn((640, 2, D), device="cuda", generator=g).to(torch.bfloat16)
    bi.kv_int4_append(K, K, torch.arange(640, device="cuda"), c)
    lens = torch.tensor([1, 130, 300], dtype=torch.int32, device="cuda")
    table = torch.arange(60, dtype=torch.int32, device="cuda").view(3, 20) % 40
    wide = torch.zeros((3, 6250), dtype=torch.int32, device="cuda")
    wide[:, :20] = table
    q = torch.randn((3, 8, D), device="cuda", generator=g).to(torch.bfloat16)
    a = bi.attention_decode_int4(q, c, table, lens, 300, SCALE)
    assert torch.equal(a, bi.attention_decode_int4(q, c, wide, lens, 100_000, SCALE))
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    assert torch.equal(a, bi.attention_extend_int4(q, cu, c, wide, lens, 100_000, 1, SCALE))
    assert torch.equal(a, bi.attention_extend_int4(q, cu, c, wide, lens, 100_000, 5000, SCALE))
    assert bi.device_status() == bi.BI_OK


def test_two_streams_at_once(bi):
    """Calls of two streams that overlap on the GPU, each with its own cache and workspace, give the bits of either alone."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(6)
    lens = torch.full((16,), 1000, dtype=torch.int32, device="cuda")
    table = torch.arange(16 * 63, dtype=torch.int32, device="cuda").view(16, 63)
    W = torch.randint(0, 256, (4096, 1024), dtype=torch.uint8, device="cuda", generator=g)
    S = torch.rand((4096, 32), device="cuda", generator=g).to(torch.bfloat16)
    jobs = []
    for _ in range(2):
        K = torch.randn((16 * 63 * 16, 8, D), device="cuda", generator=g).to(torch.bfloat16)
        jobs.append((K, torch.randn((16, 32, D), device="cuda", generator=g).to(torch.bfloat16),
                     torch.randn((24, 2048), device="cuda", generator=g).to(torch.bfloat16), bi.kv_int4_cache(16 * 63, 16, 8)))
    slots = torch.arange(16 * 63 * 16, device="cuda")

    def job(K, q, x, c, stream=None):
        bi.kv_int4_append(K, K, slots, c, stream=stream)
        return [bi.attention_decode_int4(q, c, table, lens, 1000, SCALE, stream=stream), bi.gemm_int4(x, W, S, stream=stream),
                bi.gemm_int4(x[:3], W, S, stream=stream)]

    want = [job(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for k in range(2):
            got[k].append(job(*jobs[k], stream=streams[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for out in got[k]:
            assert all(torch.equal(u, v) for u, v in zip(out, want[k]))
    assert bi.device_status() == bi.BI_OK


def test_empty_calls(bi):
    import torch
    c = bi.kv_int4_cache(2, 16, 2)
    none = torch.empty((0, 2, D), dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    assert bi.kv_int4_append(none, none, slots, c) is c
    assert bi.kv_int4_read(c, slots)[0].shape == (0, 2, D)
    q = torch.empty((0, 4, D), dtype=torch.bfloat16, device="cuda")
    table, lens = torch.empty((0, 1), dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    assert bi.attention_decode_int4(q, c, table, lens, 16, SCALE).shape == (0, 4, D)
    assert bi.attention_extend_int4(q, torch.zeros(1, dtype=torch.int32, device="cuda"), c, table, lens, 16, 1, SCALE).shape == (0, 4, D)
    assert bi.device_status() == bi.BI_OK


def test_prefill_then_decode_equals_decode_alone(bi):
    """The use of the set: a prompt's keys and values appended and attended to in pieces, then tokens decoded, against
    the same tokens decoded one by one from an empty cache: the same bits at every step, and parity with 64 bits."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(7)
    T, H, Hq, Hkv, bs = 150, 512, 8, 2, 16
    Wq = torch.randint(0, 256, ((Hq + 2 * Hkv) * D, H // 2), dtype=torch.uint8, device="cuda", generator=g)
    Sq = (0.02 * torch.rand((Wq.shape[0], H // 64), device="cuda", generator=g)).bfloat16()
    x = torch.randn((T, H), device="cuda", generator=g).bfloat16()
    table = torch.randperm(12, device="cuda", generator=g).int()[:10].view(1, 10)
    at = lambda j: table[0].long()[j // bs] * bs + j % bs

    def piece(cache, a, b, decode):
        j = torch.arange(a, b, device="cuda")
        qkv = bi.gemm_int4(x[a:b], Wq, Sq).view(b - a, -1, D)
        bi.kv_int4_append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], at(j), cache)
        q, lens = qkv[:, :Hq].contiguous(), torch.tensor([b], dtype=torch.int32, device="cuda")
        if decode:
            return bi.attention_decode_int4(q, cache, table, lens, 160, SCALE), qkv
        cu = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        return bi.attention_extend_int4(q, cu, cache, table, lens, 160, b - a, SCALE), qkv

    one = bi.kv_int4_cache(12, bs, Hkv)
    alone = [piece(one, t, t + 1, True) for t in range(T)]
    many = bi.kv_int4_cache(12, bs, Hkv)
    rows, at_once = [], []
    for a, b in ((0, 100), (100, 105), (105, 140)):
        o, qkv = piece(many, a, b, False)
        rows.append(o), at_once.append(qkv)
    for t in range(140, T):
        o, qkv = piece(many, t, t + 1, True)
        rows.append(o), at_once.append(qkv)
    assert torch.equal(torch.cat(at_once), torch.cat([p[1] for p in alone]))
    got = torch.cat(rows)
    assert torch.equal(got, torch.cat([p[0] for p in alone]))
    qkv = torch.cat(at_once).float().cpu().numpy()
    k, v = (ref.values(*ref.held(syn.to_bf16_bits(qkv[:, s]))) for s in (slice(Hq, Hq + Hkv), slice(Hq + Hkv, None)))
    want = ref.attention(qkv[:, :Hq].astype(np.float64), k, v, SCALE, causal_from=0)
    # one bf16 rounding (2^-8 of the value); the fp32 sums and the probabilities' 16 bits add less than 2^-13 of the
    # largest value each
    assert (np.abs(got.float().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * np.abs(v).max()).all()
    assert bi.device_status() == bi.BI_OK


def test_block_past_2_31_tokens_ahead(bi):
    """Blocks so large that the places of the next 31 blocks pass 31 bits: a chunk still lies in its one block."""
    import torch
    if torch.cuda.get_device_properties(0).total_memory < 64 << 30:
        pytest.skip("needs a cache of 10 GB")
    bs = 69273672                                      # 31 blocks on: past 2^31
    c = bi.KVInt4Cache(*(torch.empty((1, 1, bs, w), dtype=d, device="cuda")
                         for w, d in ((64, torch.uint8), (4, torch.bfloat16)) * 2))
    g = torch.Generator(device="cuda").manual_seed(7)
    K = torch.randn((300, 1, D), device="cuda", generator=g).to(torch.bfloat16)
    V = torch.randn((300, 1, D), device="cuda", generator=g).to(torch.bfloat16)
    small = bi.kv_int4_cache(20, 16, 1)
    for cache in (c, small):
        bi.kv_int4_append(K, V, torch.arange(300, device="cuda"), cache)
    q = torch.randn((1, 8, D), device="cuda", generator=g).to(torch.bfloat16)
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    one, many = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.arange(20, dtype=torch.int32, device="cuda").view(1, 20)
    want = bi.attention_decode_int4(q, small, many, lens, 300, SCALE)
    assert torch.equal(bi.attention_decode_int4(q, c, one, lens, 300, SCALE), want)
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for ws in (None, torch.empty(16, dtype=torch.uint8, device="cuda")):
        assert torch.equal(bi.attention_extend_int4(q, cu, c, one, lens, 300, 1, SCALE, workspace=ws), want)
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("most", [5, 4096, 2 ** 31 - 1])
def test_extend_with_a_generous_most_new_tokens(bi, most):
    """max_q_len bounds a sequence's new tokens from above; however far above, the call is the same."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(11)
    B, Hq = 6, 16
    c = bi.kv_int4_cache(8 * B, 16, 4)
    K = torch.randn((128 * B, 4, D), device="cuda", generator=g).to(torch.bfloat16)
    bi.kv_int4_append(K, K, torch.arange(128 * B, device="cuda"), c)
    table = torch.arange(8 * B, dtype=torch.int32, device="cuda").view(B, 8)
    lens = torch.tensor([100, 5, 128, 77, 0, 33], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 5, 10, 11, 13, 13, 17], dtype=torch.int32, device="cuda")
    q = torch.randn((17, Hq, D), device="cuda", generator=g).to(torch.bfloat16)
    assert bi.attention_extend_int4_workspace_size(17, Hq, 4, 128, most) > 0
    want = bi.attention_extend_int4(q, cu, c, table, lens, 128, 5, SCALE, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert torch.equal(bi.attention_extend_int4(q, cu, c, table, lens, 128, most, SCALE), want)
    assert bi.device_status() == bi.BI_OK


def test_generous_maximum_length_of_many(bi):
    """Enough room under the maximum length that the lengths are read first; among them one of 0 and one past it."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    B, top = 40, 200_000
    c = bi.kv_int4_cache(64, 16, 2)
    K = torch.randn((1024, 2, D), device="cuda", generator=g).to(torch.bfloat16)
    bi.kv_int4_append(K, K, torch.arange(1024, device="cuda"), c)
    lens = torch.randint(1, 520, (B,), device="cuda", generator=g).int()
    lens[0], lens[39] = 1, 520
    wide = torch.zeros((B, top // 16), dtype=torch.int32, device="cuda")
    wide[:, :33] = torch.randint(0, 64, (B, 33), device="cuda", generator=g).int()
    table = wide[:, :33].contiguous()
    q = torch.randn((B, 8, D), device="cuda", generator=g).to(torch.bfloat16)
    a = bi.attention_decode_int4(q, c, table, lens, 520, SCALE)
    assert torch.equal(a, bi.attention_decode_int4(q, c, wide, lens, top, SCALE))
    assert bi.device_status() == bi.BI_OK
    lens[7], lens[8] = 0, top + 1
    o = torch.full_like(a, 7.0)
    bi.attention_decode_int4(q, c, wide, lens, top, SCALE, O=o)
    assert bi.device_status() == bi.BI_ERR_INVALID_ARG
    assert bool((o[7:9] == 7).all())
    keep = [b for b in range(B) if b not in (7, 8)]
    assert torch.equal(o[keep], a[keep])


def test_results_made_on_another_stream(bi):
    """Outputs and workspaces that a call on another stream allocates: not the memory of work still queued on the
    current stream, and not reused before the current stream has read them."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(6)
    X = torch.randn((64, 4096), device="cuda", generator=g).bfloat16()
    W = torch.randint(0, 256, (2048, 2048), dtype=torch.uint8, device="cuda", generator=g)
    S = torch.rand((2048, 32), device="cuda", generator=g).bfloat16()
    S_neg = S.neg()
    want = bi.gemm_int4(X, W, S)
    side = torch.cuda.Stream()
    big = torch.randn((8192, 8192), device="cuda")
    torch.cuda.synchronize()
    for _ in range(4):
        before = torch.full((64, 2048), 3.0, device="cuda", dtype=torch.bfloat16)
        (big @ big)                                        # keeps the current stream busy
        copy = before + 1
        del before                                         # free for the current stream, still to be read there
        y = bi.gemm_int4(X, W, S, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        (big @ big)
        got = y + 0
        del y                                              # free, still to be read by the current stream
        z = bi.gemm_int4(X, W, S_neg, stream=side)
        torch.cuda.synchronize()
        assert bool((copy == 4).all()) and torch.equal(got, want) and torch.equal(z, -want)


def test_another_stream_inside_a_capture(bi):
    """A call on a stream forked from the captured one, its output and workspace allocated for that stream: replays give
    the eager bits."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(9)
    X = torch.randn((24, 1024), device="cuda", generator=g).bfloat16()
    W = torch.randint(0, 256, (512, 512), dtype=torch.uint8, device="cuda", generator=g)
    S = torch.rand((512, 8), device="cuda", generator=g).bfloat16()
    c = bi.kv_int4_cache(24, 16, 2)
    K = torch.randn((384, 2, D), device="cuda", generator=g).bfloat16()
    bi.kv_int4_append(K, K, torch.arange(384, device="cuda"), c)
    q = torch.randn((1, 8, D), device="cuda", generator=g).bfloat16()
    table, lens = torch.arange(24, dtype=torch.int32, device="cuda").view(1, 24), torch.tensor([380], dtype=torch.int32, device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        y = bi.gemm_int4(X, W, S, stream=side)
        o = bi.attention_decode_int4(q, c, table, lens, 384, SCALE, stream=side)
        z = bi.gemm_int4(X, W, S)
        torch.cuda.current_stream().wait_stream(side)
        both = y + z
    for _ in range(2):
        X.normal_(generator=g), q.normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, bi.gemm_int4(X, W, S)) and torch.equal(z, y) and torch.equal(both, y + z)
        assert torch.equal(o, bi.attention_decode_int4(q, c, table, lens, 384, SCALE))
    assert bi.device_status() == bi.BI_OK
