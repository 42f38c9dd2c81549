"""Workloads of the 4-bit serving operators: a paged K/V cache held in 4 bits
(append, read), decode and extend attention over it, and linear layers with
4-bit weights and group scales.

Each case is one pass through an operator. `run` computes it either through the
framework (`own` true) or in plain torch operations in 32 bits.

The cache format: every 32 consecutive dimensions of one token's K (or V) row of
one KV head share a scale s, the smallest number with four significant bits that
is at least amax / 7 (kept in [2^-100, 2^120]); each value is held as the integer
round(x / s) in -7 .. 7 (ties to even). The weights: W[n][k] = (u - z) * s with
4-bit u, and s, z per row and group of g consecutive k (z = 8 without zeros).
"""
import math
import random

import numpy as np
import torch

own = False

D = 128          # head dimension
GROUP = 32       # dimensions of a cache row that share a scale


def _gen(seed, stream):
    return torch.Generator(device="cuda").manual_seed(1000003 * (int(seed) % (1 << 30)) + stream)


def _bf16(shape, seed, stream, std=1.0):
    x = torch.randn(shape, device="cuda", generator=_gen(seed, stream))
    return (x * std).to(torch.bfloat16)


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one decode step of a batch of 64: each sequence's new token goes to its own slot
        dict(name="kv_step_64", op="kv", tokens=64, padded=0, Hkv=8, bs=16),
        # a chunk of prompt tokens, its batch padded at the end (slot -1)
        dict(name="kv_prompt_8155", op="kv", tokens=8155, padded=37, Hkv=8, bs=16),
        # one user: latency counts
        dict(name="decode_1x4096", op="decode", B=1, len_min=4096, len_max=4096, Hq=32, Hkv=8, bs=16),
        # a full decode batch
        dict(name="decode_64x4096", op="decode", B=64, len_min=4096, len_max=4096, Hq=32, Hkv=8, bs=16),
        # a ragged batch without shared heads, blocks that end inside a 128-token chunk
        dict(name="decode_7_ragged_mha", op="decode", B=7, len_min=1, len_max=9000, Hq=8, Hkv=8, bs=24),
        # two long contexts, eight query heads a KV head
        dict(name="decode_2x131072_g8", op="decode", B=2, len_min=131072, len_max=131072, Hq=64, Hkv=8, bs=128),
        # a few drafted tokens a sequence checked at once
        dict(name="extend_16x5_drafts", op="extend", B=16, q_min=5, q_max=5, past_min=100, past_max=4000, Hq=32, Hkv=8, bs=16),
        # chunked prefill and decode mixed in one batch
        dict(name="extend_8_mixed_g8", op="extend", B=8, q_min=1, q_max=512, past_min=0, past_max=2500, Hq=32, Hkv=4, bs=32),
        # the second half of an 8192-token prompt
        dict(name="extend_1x4096_over_8192", op="extend", B=1, q_min=4096, q_max=4096, past_min=4096, past_max=4096, Hq=32, Hkv=8, bs=16),
        # one token's qkv projection
        dict(name="gemm_m1_qkv", op="gemm", M=1, N=6144, K=4096, g=128, zeros=False),
        # gate_up of a batch of 16, asymmetric codes
        dict(name="gemm_m16_gate_up", op="gemm", M=16, N=24576, K=4096, g=64, zeros=True),
        # down projection of a short prompt
        dict(name="gemm_m200_down", op="gemm", M=200, N=4096, K=12288, g=32, zeros=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["kv", "decode", "decode", "extend", "gemm", "gemm"])
    heads = [(32, 8), (32, 4), (16, 8), (8, 8), (64, 8), (4, 1), (5, 5)]
    blocks = [1, 8, 16, 16, 24, 32, 48, 64, 128, 256]
    if op == "kv":
        return dict(op=op, tokens=_log_int(rng, 1, 8000), padded=rng.choice([0, 0, 1, 30]), Hkv=rng.choice([1, 2, 4, 5, 8]),
                    bs=rng.choice(blocks))
    Hq, Hkv = rng.choice(heads)
    if op == "decode":
        B = _log_int(rng, 1, 64)
        most = max(2, min(131072, (64 * 4096 * 8) // (B * max(Hkv, Hq // 4))))
        len_max = _log_int(rng, 2, most)
        return dict(op=op, B=B, len_min=rng.choice([1, len_max, max(1, len_max // 3)]), len_max=len_max, Hq=Hq, Hkv=Hkv,
                    bs=rng.choice(blocks))
    if op == "extend":
        B = _log_int(rng, 1, 16)
        q_max = _log_int(rng, 2, max(2, min(2000, 8000 // B)))
        return dict(op=op, B=B, q_min=rng.choice([1, q_max]), q_max=q_max, past_min=0, past_max=_log_int(rng, 1, 3500), Hq=min(Hq, 32),
                    Hkv=min(Hkv, 8) if Hq <= 32 else 8, bs=rng.choice(blocks))
    g = rng.choice([32, 64, 128, 256])
    K = g * _log_int(rng, 1, 12288 // g)
    return dict(op=op, M=_log_int(rng, 1, 200), N=8 * _log_int(rng, 1, 3000 if K <= 4096 else 512), K=K, g=g,
                zeros=rng.choice([False, True]))


def _spread(case, what, lo, hi, n):
    """n sizes between lo and hi, fixed by the case; the first is the largest."""
    r = random.Random("%s %s %s %s" % (what, lo, hi, n))
    return [hi] + [r.randint(lo, hi) for _ in range(n - 1)]


def _lens(case):
    """(new tokens, cached length with them) of each sequence of an attention case."""
    B = case["B"]
    if case["op"] == "decode":
        L = _spread(case, "len", case["len_min"], case["len_max"], B)
        return [1] * B, L
    q = _spread(case, "q", case["q_min"], case["q_max"], B)
    past = _spread(case, "past", case["past_min"], case["past_max"], B)[::-1]
    return q, [a + b for a, b in zip(q, past)]


def work(case):
    row = D // 2 + D // GROUP * 2                       # bytes of one cache row (codes and scales)
    if case["op"] == "kv":
        T, H = case["tokens"], case["Hkv"]
        once = T * H * 2 * (2 * D + row) + 8 * (T + case["padded"])
        return dict(bytes=2 * once + case["padded"] * H * 2 * 2 * D, flops=T * H * 2 * D * 4)
    if case["op"] == "gemm":
        M, N, K, g = case["M"], case["N"], case["K"], case["g"]
        return dict(bytes=N * K // 2 + N * (K // g) * (3 if case["zeros"] else 2) + 2 * M * (K + N), flops=2 * M * N * K)
    q, L = _lens(case)
    Hq, Hkv, bs = case["Hq"], case["Hkv"], case["bs"]
    pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(q, L))
    table = sum(4 * -(-b // bs) for b in L)
    return dict(bytes=sum(L) * Hkv * 2 * row + sum(q) * Hq * D * 4 + table + 8 * len(L), flops=4 * D * Hq * pairs)


# ----------------------------------------------------------------- inputs ---

def _kv_rows(T, Hkv, seed, stream):
    """Keys with a few strong channels a head, values without."""
    loud = 1.0 + 7.0 * (torch.rand((1, Hkv, D), device="cuda", generator=_gen(seed, stream)) > 0.96).float()
    K = torch.randn((T, Hkv, D), device="cuda", generator=_gen(seed, stream + 1)).mul_(loud).to(torch.bfloat16)
    V = torch.randn((T, Hkv, D), device="cuda", generator=_gen(seed, stream + 2)).mul_(0.4).to(torch.bfloat16)
    return K, V


def _slots(case, seed):
    T, bs = case["tokens"], case["bs"]
    blocks = -(-T // bs) + 5
    order = torch.randperm(blocks, device="cuda", generator=_gen(seed, 3))
    if T <= 256:                                        # a decode step: one slot a sequence, anywhere
        s = torch.randperm(blocks * bs, device="cuda", generator=_gen(seed, 4))[:T]
    else:                                               # a prompt: its blocks filled in order
        t = torch.arange(T, device="cuda")
        s = order[t // bs] * bs + t % bs
    return torch.cat([s, torch.full((case["padded"],), -1, device="cuda", dtype=s.dtype)]), blocks


def _kv_inputs(case, seed):
    T = case["tokens"] + case["padded"]
    K, V = _kv_rows(T, case["Hkv"], seed, 10)
    slots, blocks = _slots(case, seed)
    return K, V, slots, blocks


def _attn_inputs(case, seed):
    """Q, cu_q, K and V rows of the whole cache by slot, block table, lengths."""
    q, L = _lens(case)
    B, bs, Hq, Hkv = case["B"], case["bs"], case["Hq"], case["Hkv"]
    per = [-(-n // bs) for n in L]
    blocks = sum(per) + 3
    order = torch.randperm(blocks, device="cuda", generator=_gen(seed, 20)).to(torch.int32)
    table = torch.zeros((B, max(per)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    K, V = _kv_rows(blocks * bs, Hkv, seed, 21)
    Q = _bf16((sum(q), Hq, D), seed, 25)
    cu = torch.tensor([0] + list(np.cumsum(q)), dtype=torch.int32, device="cuda")
    lens = torch.tensor(L, dtype=torch.int32, device="cuda")
    return Q, cu, K, V, table, lens, blocks


def _gemm_inputs(case, seed):
    M, N, K, g = case["M"], case["N"], case["K"], case["g"]
    X = _bf16((M, K), seed, 30)
    u = torch.randn((N, K), device="cuda", generator=_gen(seed, 31)).mul_(2.5).round_().add_(8).clamp_(0, 15).to(torch.uint8)
    W = u[:, 0::2] | (u[:, 1::2] << 4)
    S = (0.004 + 0.012 * torch.rand((N, K // g), device="cuda", generator=_gen(seed, 32))).to(torch.bfloat16)
    Z = torch.randint(5, 12, (N, K // g), device="cuda", generator=_gen(seed, 33), dtype=torch.uint8) if case["zeros"] else None
    return X, W.contiguous(), S, Z


# ------------------------------------------------------------- plain forms ---

def _quantise(x):
    """x [.., D] bf16 -> packed codes uint8 [.., D/2] (value + 8, low nibble first), scales [.., D/GROUP] fp32."""
    g = x.float().reshape(*x.shape[:-1], D // GROUP, GROUP)
    amax = g.abs().amax(-1)
    need = (amax / torch.full_like(amax, 7.0)).clamp(2.0 ** -100, 2.0 ** 120)   # a tensor divisor: a scalar one is a product on the GPU
    cut = (1 << 20) - 1                                 # of the 23 fraction bits, three stay (rounded up)
    s = ((need.view(torch.int32) + cut) & ~cut).view(torch.float32)
    u = (torch.round(g / s[..., None]).clamp(-7, 7) + 8).to(torch.uint8).reshape(x.shape)
    return u[..., 0::2] | (u[..., 1::2] << 4), s


def _dequantise(codes, s):
    u = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(*codes.shape[:-1], D).float() - 8.0
    return (u.reshape(*s.shape, GROUP) * s[..., None]).reshape(u.shape)


def _plain_cache(K, V):
    return [t for x in (K, V) for t in _quantise(x)]


def _plain_kv(st):
    kc, ks, vc, vs = st["cache"]
    at = st["slots"]
    good = at >= 0
    for x, codes, scales in ((st["K"], kc, ks), (st["V"], vc, vs)):
        c, s = _quantise(x)
        codes[at[good]] = c[good]
        scales[at[good]] = s[good]
    rows = at.clamp(min=0)
    keep = good[:, None, None]
    return tuple((_dequantise(c[rows], s[rows]) * keep).to(torch.bfloat16) for c, s in ((kc, ks), (vc, vs)))


def _plain_attention(st):
    case, Q, (kc, ks, vc, vs) = st["case"], st["Q"], st["cache"]
    bs, G = case["bs"], case["Hq"] // case["Hkv"]
    qn, L = _lens(case)
    out = torch.empty_like(Q)
    at = 0
    for b in range(case["B"]):
        n, q = L[b], qn[b]
        j = torch.arange(n, device="cuda")
        slot = st["table"][b].long()[j // bs] * bs + j % bs
        K = _dequantise(kc[slot], ks[slot]).permute(1, 2, 0)                       # [Hkv, D, n]
        V = _dequantise(vc[slot], vs[slot]).permute(1, 0, 2)                       # [Hkv, n, D]
        x = Q[at:at + q].float().reshape(q, case["Hkv"], G, D).permute(1, 2, 0, 3).reshape(case["Hkv"], G * q, D)
        s = torch.matmul(x, K).mul_(st["scale"]).view(case["Hkv"], G, q, n)
        s.masked_fill_(j[None, :] > (n - q + torch.arange(q, device="cuda"))[:, None], float("-inf"))
        s = torch.exp(s.sub_(s.amax(-1, keepdim=True)))
        l = s.sum(-1, keepdim=True)
        o = torch.matmul(s.view(case["Hkv"], G * q, n), V).view(case["Hkv"], G, q, D) / l
        out[at:at + q] = o.permute(2, 0, 1, 3).reshape(q, case["Hq"], D).to(torch.bfloat16)
        at += q
    return out


def _plain_gemm(st):
    W, S, Z = st["W"], st["S"], st["Z"]
    u = torch.stack([W & 15, W >> 4], dim=-1).reshape(W.shape[0], S.shape[1], -1).float()
    w = (u - (8.0 if Z is None else Z.float()[..., None])) * S.float()[..., None]
    return torch.matmul(st["X"].float(), w.reshape(W.shape[0], -1).t()).to(torch.bfloat16)


# --------------------------------------------------------------------- run ---

def prepare(case, seed):
    if own:
        import invariant_deterministic_bi_gb300 as bi
    if case["op"] == "kv":
        K, V, slots, blocks = _kv_inputs(case, seed)
        st = dict(case=case, K=K, V=V, slots=slots)
        if own:
            st["cache"] = bi.kv_int4_cache(blocks, case["bs"], case["Hkv"])
        else:
            zero = torch.zeros((blocks * case["bs"], case["Hkv"], D), dtype=torch.bfloat16, device="cuda")
            st["cache"] = _plain_cache(zero, zero)
        return st
    if case["op"] == "gemm":
        X, W, S, Z = _gemm_inputs(case, seed)
        return dict(case=case, X=X, W=W, S=S, Z=Z)
    Q, cu, K, V, table, lens, blocks = _attn_inputs(case, seed)
    q, L = _lens(case)
    st = dict(case=case, Q=Q, cu=cu, table=table, lens=lens, max_len=max(L), max_q=max(q), scale=D ** -0.5)
    if own:
        st["cache"] = bi.kv_int4_cache(blocks, case["bs"], case["Hkv"])
        bi.kv_int4_append(K, V, torch.arange(K.shape[0], device="cuda"), st["cache"])
        if case["op"] == "decode":
            st["workspace"] = torch.empty(bi.attention_decode_workspace_size(case["B"], case["Hq"], st["max_len"]),
                                          dtype=torch.uint8, device="cuda")
    else:
        st["cache"] = _plain_cache(K, V)
    return st


def run(state):
    case = state["case"]
    if not own:
        return {"kv": _plain_kv, "decode": _plain_attention, "extend": _plain_attention, "gemm": _plain_gemm}[case["op"]](state)
    import invariant_deterministic_bi_gb300 as bi
    if case["op"] == "kv":
        bi.kv_int4_append(state["K"], state["V"], state["slots"], state["cache"])
        return bi.kv_int4_read(state["cache"], state["slots"])
    if case["op"] == "gemm":
        return bi.gemm_int4(state["X"], state["W"], state["S"], zeros=state["Z"])
    if case["op"] == "decode":
        return bi.attention_decode_int4(state["Q"], state["cache"], state["table"], state["lens"], state["max_len"], state["scale"],
                                        workspace=state["workspace"])
    return bi.attention_extend_int4(state["Q"], state["cu"], state["cache"], state["table"], state["lens"], state["max_len"],
                                    state["max_q"], state["scale"])


# ------------------------------------------------------------------- exact ---

def _held(x):
    """The values that the cache holds for rows x, in 64 bits, from the format's definition."""
    x = x.double()
    y = x.reshape(-1, GROUP)
    need = y.abs().max(dim=1).values
    need = need / torch.full_like(need, 7.0)                                   # true division
    need = torch.minimum(torch.maximum(need, torch.full_like(need, 2.0 ** -100)), torch.full_like(need, 2.0 ** 120))
    part = torch.frexp(need).mantissa                                          # in [0.5, 1), and need / part a power of two
    s = torch.ceil(part * 16) * (need / part) / 16                             # four significant bits
    return (torch.clamp(torch.round(y / s[:, None]), -7, 7) * s[:, None]).reshape(x.shape)


def exact(case, seed):
    if case["op"] == "kv":
        K, V, slots, _ = _kv_inputs(case, seed)
        live = (slots >= 0).double().reshape(-1, 1, 1)
        return _held(K) * live, _held(V) * live
    if case["op"] == "gemm":
        X, W, S, Z = _gemm_inputs(case, seed)
        N, K, g = case["N"], case["K"], case["g"]
        out = torch.empty((case["M"], N), dtype=torch.float64, device="cuda")
        step = max(1, (1 << 26) // K)
        for n0 in range(0, N, step):
            w = torch.empty((min(N, n0 + step) - n0, K), dtype=torch.float64, device="cuda")
            w[:, 0::2] = (W[n0:n0 + step] % 16).double()
            w[:, 1::2] = (W[n0:n0 + step] // 16).double()
            z = 8.0 if Z is None else Z[n0:n0 + step].double().repeat_interleave(g, dim=1)
            w = (w - z) * S[n0:n0 + step].double().repeat_interleave(g, dim=1)
            out[:, n0:n0 + step] = X.double() @ w.T
        return out
    Q, cu, K, V, table, lens, _ = _attn_inputs(case, seed)
    qn, L = _lens(case)
    bs, Hkv, G = case["bs"], case["Hkv"], case["Hq"] // case["Hkv"]
    out = torch.empty(Q.shape, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        a0, a1, n = int(cu[b]), int(cu[b + 1]), L[b]
        rows = (table[b, :-(-n // bs)].long()[:, None] * bs + torch.arange(bs, device="cuda")[None, :]).reshape(-1)[:n]
        seen = torch.arange(n, device="cuda")[None, :] <= torch.arange(n - (a1 - a0), n, device="cuda")[:, None]
        for h in range(Hkv):
            k, v = _held(K[rows, h]), _held(V[rows, h])
            for i in range(h * G, (h + 1) * G):
                s = (Q[a0:a1, i].double() @ k.T) * (D ** -0.5)
                s = torch.where(seen, s, torch.full_like(s, -math.inf))
                out[a0:a1, i] = torch.softmax(s, dim=-1) @ v
    return out
