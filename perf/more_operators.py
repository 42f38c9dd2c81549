"""Workloads of the operators between a qkv projection and its attention, and of
attention with a sliding window: rotary positions, norms of query and key heads
with the rotation in the same pass, appending to the paged bf16 K/V cache, and
decode and extend attention over it with a window and first tokens that stay
visible.

Each case is one pass through an operator. `run` computes it either through the
framework (`own` true) or in plain torch operations in 32 bits.

Rotation at position p: the pair (a, b) of frequency f_i becomes
m (a cos p f_i - b sin p f_i, b cos p f_i + a sin p f_i); pairs are dimensions
(i, i + R/2) or, interleaved, (2i, 2i + 1) of the first R of a head. Norm:
x / sqrt(mean x^2 + eps) * w over a head, before the rotation. Window: the token
at position p sees position j <= p if j > p - window or j < sinks.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6


def _gen(seed, stream):
    return torch.Generator(device="cuda").manual_seed(1000003 * (int(seed) % (1 << 30)) + stream)


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # queries of one decode step of a batch of 64, far apart in their sequences
        dict(name="rope_step_64", op="rope", T=64, H=32, extra=0, D=128, R=128, inter=False, scaling="none", s=1.0, start=-1),
        # query and key heads of a prompt chunk, slices of the projection's rows; half of each head turns, positions
        # far beyond the trained length
        dict(name="rope_prompt_8155", op="rope", T=8155, H=40, extra=8, D=128, R=64, inter=True, scaling="yarn", s=8.0, start=100000),
        # one user's decode step: latency counts
        dict(name="qk_norm_rope_1", op="qk", T=1, Hq=32, Hkv=8, D=128, R=128, inter=False, scaling="none", s=1.0, start=-1),
        # a prompt chunk, eight query heads a KV head
        dict(name="qk_norm_rope_8155", op="qk", T=8155, Hq=32, Hkv=4, D=128, R=128, inter=False, scaling="none", s=1.0, start=0),
        # everything between projection and attention of a decode step: 61 sequences padded to 64
        dict(name="kv_append_step_64", op="kv", T=61, padded=3, Hq=32, Hkv=8, norm=True, bs=16, R=128, inter=False,
             scaling="none", s=1.0, start=-1),
        # a prompt chunk's keys and values, its batch padded at the end
        dict(name="kv_append_prompt_8155", op="kv", T=8155, padded=37, Hq=0, Hkv=8, norm=False, bs=16, R=128, inter=False,
             scaling="bands", s=8.0, start=20000),
        # one long conversation
        dict(name="decode_window_1x32768", op="decode", B=1, len_min=32768, len_max=32768, Hq=32, Hkv=8, bs=16, W=1024, S=4),
        # a full decode batch, most sequences longer than the window
        dict(name="decode_window_64x16000", op="decode", B=64, len_min=3000, len_max=16000, Hq=32, Hkv=8, bs=16, W=4096, S=0),
        # a ragged batch without shared heads, blocks and window that end inside a 128-token chunk
        dict(name="decode_window_7_ragged_mha", op="decode", B=7, len_min=1, len_max=9000, Hq=8, Hkv=8, bs=24, W=300, S=5),
        # a few drafted tokens a sequence checked at once
        dict(name="extend_window_16x5_drafts", op="extend", B=16, q_min=5, q_max=5, past_min=100, past_max=4000, Hq=32, Hkv=8,
             bs=16, W=1024, S=4),
        # chunked prefill and decode mixed in one batch
        dict(name="extend_window_8_mixed_g8", op="extend", B=8, q_min=1, q_max=512, past_min=0, past_max=2500, Hq=32, Hkv=4,
             bs=32, W=512, S=4),
        # the second half of an 8192-token prompt
        dict(name="extend_window_1x4096_over_8192", op="extend", B=1, q_min=4096, q_max=4096, past_min=4096, past_max=4096,
             Hq=32, Hkv=8, bs=16, W=2000, S=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "qk", "kv", "decode", "decode", "extend"])
    blocks = [1, 8, 16, 16, 24, 32, 48, 64, 128, 256]
    turn = dict(inter=rng.choice([False, True]), scaling=rng.choice(["none", "linear", "ntk", "bands", "yarn"]),
                s=rng.choice([2.0, 4.0, 8.0, 32.0]), start=rng.choice([-1, 0, 0, 4000, 130000]))
    if op in ("rope", "qk"):
        T = _log_int(rng, 1, 8155)
        D = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
        R = rng.choice([D, D, 16 * rng.randint(1, D // 16)])
        most = max(1, min(64, 8155 * 36 * 128 // (T * D)))
        if op == "rope":
            return dict(op=op, T=T, H=_log_int(rng, 1, most), extra=rng.choice([0, 3, 8]), D=D, R=R, **turn)
        Hkv = _log_int(rng, 1, max(1, most // 4))
        return dict(op=op, T=T, Hq=Hkv * rng.choice([1, 2, 3]), Hkv=Hkv, D=D, R=R, **turn)
    if op == "kv":
        T, Hkv = _log_int(rng, 1, 8000), rng.choice([1, 2, 4, 5, 8])
        return dict(op=op, T=T, padded=rng.choice([0, 0, 1, 30]), Hq=rng.choice([0, Hkv, 4 * Hkv]) if T <= 3000 else 0, Hkv=Hkv,
                    norm=rng.choice([False, True]), bs=rng.choice(blocks), R=rng.choice([32, 64, 128, 128]), **turn)
    Hq, Hkv = rng.choice([(32, 8), (32, 4), (16, 8), (8, 8), (64, 8), (4, 1), (5, 5)])
    W, S = _log_int(rng, 1, 4096), rng.choice([0, 0, 1, 4, 16, 64, 200])
    if op == "decode":
        B = _log_int(rng, 1, 64)
        len_max = _log_int(rng, 2, 131072)
        return dict(op=op, B=B, len_min=rng.choice([1, len_max, max(1, len_max // 3)]), len_max=len_max, Hq=Hq, Hkv=Hkv,
                    bs=rng.choice(blocks), W=W, S=S)
    B = _log_int(rng, 1, 16)
    q_max = _log_int(rng, 2, max(2, min(2000, 8000 // B)))
    return dict(op=op, B=B, q_min=rng.choice([1, q_max]), q_max=q_max, past_min=0, past_max=_log_int(rng, 1, 30000),
                Hq=min(Hq, 32), Hkv=min(Hkv, 8) if Hq <= 32 else 8, bs=rng.choice(blocks), W=min(W, 2000), S=S)


def _spread(case, what, lo, hi, n):
    """n sizes between lo and hi, fixed by the case; the first is the largest."""
    r = random.Random("%s %s %s %s" % (what, lo, hi, n))
    return [hi] + [r.randint(lo, hi) for _ in range(n - 1)]


def _lens(case):
    """(new tokens, cached length with them) of each sequence of an attention case."""
    B = case["B"]
    if case["op"] == "decode":
        return [1] * B, _spread(case, "len", case["len_min"], case["len_max"], B)
    q = _spread(case, "q", case["q_min"], case["q_max"], B)
    past = _spread(case, "past", case["past_min"], case["past_max"], B)[::-1]
    return q, [a + b for a, b in zip(q, past)]


def _seen(case, q, n):
    """(first tokens, start of the rest) that any of the last q of n tokens sees."""
    lo = max(0, n - q + 1 - case["W"])
    return min(case["S"], lo), lo


def work(case):
    op = case["op"]
    if op in ("rope", "qk"):
        rows = case["T"] * (case["H"] if op == "rope" else case["Hq"] + case["Hkv"])
        return dict(bytes=4 * rows * case["D"] + 8 * case["T"], flops=rows * (3 * case["R"] + (0 if op == "rope" else 4 * case["D"])))
    if op == "kv":
        T, P = case["T"], case["padded"]
        q, kv = (T + P) * case["Hq"], T * case["Hkv"]
        return dict(bytes=4 * 128 * (q + 2 * kv) + 16 * (T + P), flops=(q + kv) * (3 * case["R"] + (512 if case["norm"] else 0)))
    q, L = _lens(case)
    Hq, Hkv, W, S = case["Hq"], case["Hkv"], case["W"], case["S"]
    pairs = seen = 0
    for a, n in zip(q, L):
        first, lo = _seen(case, a, n)
        seen += first + n - lo
        p = np.arange(n - a, n, dtype=np.int64)
        pairs += int((np.minimum(p + 1, W) + np.clip(p + 1 - W, 0, S)).sum())
    return dict(bytes=seen * Hkv * 512 + sum(q) * Hq * 512 + 8 * len(L), flops=512 * Hq * pairs)


# ----------------------------------------------------------------- inputs ---

def _freq_args(case):
    """What a user gives for the case's frequencies."""
    kw = dict(base=1000000.0, interleaved=case["inter"])
    if case["scaling"] != "none":
        kw.update(scaling=case["scaling"], scale=case["s"])
    if case["scaling"] in ("bands", "yarn"):
        kw.update(original_length=8192)
    return kw


def _positions(case, T, seed):
    if case["start"] < 0:                               # a decode step: a position a sequence
        return torch.randint(0, 131072, (T,), device="cuda", generator=_gen(seed, 1))
    return case["start"] + torch.arange(T, device="cuda")


def _heads(T, H, D, seed, stream):
    """Heads of a projection: a few strong channels each, tokens of different size."""
    g = _gen(seed, stream)
    loud = 1.0 + 7.0 * (torch.rand((1, H, D), device="cuda", generator=g) > 0.96).float()
    size = 0.5 + torch.rand((T, 1, 1), device="cuda", generator=g)
    return torch.randn((T, H, D), device="cuda", generator=g).mul_(loud).mul_(size).to(torch.bfloat16)


def _weight(D, seed, stream):
    return (0.4 + 1.6 * torch.rand(D, device="cuda", generator=_gen(seed, stream))).to(torch.bfloat16)


def _slots(case, seed):
    T, bs = case["T"], case["bs"]
    blocks = -(-T // bs) + 5
    order = torch.randperm(blocks, device="cuda", generator=_gen(seed, 3))
    if T <= 256:                                        # a decode step: one slot a sequence, anywhere
        s = torch.randperm(blocks * bs, device="cuda", generator=_gen(seed, 4))[:T]
    else:                                               # a prompt: its blocks filled in order
        t = torch.arange(T, device="cuda")
        s = order[t // bs] * bs + t % bs
    return torch.cat([s, torch.full((case["padded"],), -1, device="cuda", dtype=s.dtype)]), blocks


def _attn_inputs(case, seed):
    """Q, cu_q, K and V caches, block table, lengths. Blocks that no token sees any more were given back."""
    q, L = _lens(case)
    B, bs, Hq, Hkv = case["B"], case["bs"], case["Hq"], case["Hkv"]
    table = np.full((B, max(-(-n // bs) for n in L)), -1, dtype=np.int64)
    live = np.zeros(table.shape, dtype=bool)
    for b, (a, n) in enumerate(zip(q, L)):
        first, lo = _seen(case, a, n)
        i = np.arange(-(-n // bs)) * bs
        live[b, :i.size] = (i < first) | (i + bs > lo)
    blocks = int(live.sum()) + 3
    table[live] = np.random.RandomState(int(seed) % (1 << 30)).permutation(blocks)[:blocks - 3]
    K = _heads(blocks * bs, Hkv, 128, seed, 21).view(blocks, bs, Hkv, 128)
    V = _heads(blocks * bs, Hkv, 128, seed, 22).mul_(0.4).view(blocks, bs, Hkv, 128)
    Q = torch.randn((sum(q), Hq, 128), device="cuda", generator=_gen(seed, 25)).to(torch.bfloat16)
    cu = torch.tensor([0] + list(np.cumsum(q)), dtype=torch.int32, device="cuda")
    lens = torch.tensor(L, dtype=torch.int32, device="cuda")
    return Q, cu, K, V, torch.tensor(table, dtype=torch.int32, device="cuda"), lens


def _row_inputs(case, seed):
    """The tensors of a case without attention."""
    if case["op"] == "rope":
        T = case["T"]
        X = _heads(T, case["H"] + case["extra"], case["D"], seed, 10)[:, :case["H"]]     # a slice of the projection
        return dict(X=X, pos=_positions(case, T, seed))
    if case["op"] == "qk":
        T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
        X = _heads(T, Hq + 2 * Hkv, D, seed, 10)
        return dict(Q=X[:, :Hq], K=X[:, Hq:Hq + Hkv], pos=_positions(case, T, seed), qw=_weight(D, seed, 11), kw=_weight(D, seed, 12))
    T, Hq, Hkv = case["T"] + case["padded"], case["Hq"], case["Hkv"]
    X = _heads(T, Hq + 2 * Hkv, 128, seed, 10)
    slots, blocks = _slots(case, seed)
    return dict(Q=X[:, :Hq] if Hq else None, K=X[:, Hq:Hq + Hkv], V=X[:, Hq + Hkv:], pos=_positions(case, T, seed),
                qw=_weight(128, seed, 11) if case["norm"] and Hq else None, kw=_weight(128, seed, 12) if case["norm"] else None,
                slots=slots, blocks=blocks)


# ------------------------------------------------------------- plain forms ---

def _plain_freqs(case):
    """Frequencies in 64 bits, and what cos and sin are multiplied by."""
    R, s, base = case["R"], case["s"], 1000000.0
    kind, i = case["scaling"], torch.arange(case["R"] // 2, dtype=torch.float64)
    if kind == "ntk" and R > 2:
        base *= s ** (R / (R - 2))
    f, m = torch.exp(-2.0 * i / R * math.log(base)), 1.0
    if kind == "linear":
        f = f / s
    elif kind == "bands":
        t = ((8192 * f / (2 * math.pi) - 1.0) / 3.0).clamp(0, 1)
        f = f * (t + (1 - t) / s)
    elif kind == "yarn":
        ends = [R * math.log(8192 / (2 * math.pi * n)) / (2 * math.log(base)) for n in (32.0, 1.0)]
        lo, hi = max(math.floor(ends[0]), 0), min(math.ceil(ends[1]), R - 1)
        t = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f, m = f * (1 - t + t / s), 0.1 * math.log(s) + 1.0
    return f.cuda(), m


def _plain_turn(x, pos, freqs, inter):
    f, m = freqs
    R = 2 * f.numel()
    angle = pos.double()[:, None, None] * f
    c, s = (torch.cos(angle) * m).float(), (torch.sin(angle) * m).float()
    y = x.clone()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., :R // 2], x[..., R // 2:R])
    u, v = a * c - b * s, b * c + a * s
    if inter:
        y[..., 0:R:2], y[..., 1:R:2] = u, v
    else:
        y[..., :R // 2], y[..., R // 2:R] = u, v
    return y


def _plain_norm(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _plain_rope(st):
    return _plain_turn(st["X"].float(), st["pos"], st["freqs"], st["case"]["inter"]).to(torch.bfloat16)


def _plain_qk(st):
    return tuple(_plain_turn(_plain_norm(st[x].float(), st[w]), st["pos"], st["freqs"], st["case"]["inter"]).to(torch.bfloat16)
                 for x, w in (("Q", "qw"), ("K", "kw")))


def _plain_kv(st):
    keep = st["slots"] >= 0
    at, shape = st["slots"][keep], (-1,) + st["Kc"].shape[2:]
    k = _plain_turn(_plain_norm(st["K"].float(), st["kw"]), st["pos"], st["freqs"], st["case"]["inter"]).to(torch.bfloat16)
    st["Kc"].view(shape)[at] = k[keep]
    st["Vc"].view(shape)[at] = st["V"][keep]
    if st["Q"] is None:
        return st["Kc"], st["Vc"]
    q = _plain_turn(_plain_norm(st["Q"].float(), st["qw"]), st["pos"], st["freqs"], st["case"]["inter"]).to(torch.bfloat16)
    return st["Kc"], st["Vc"], q


def _plain_attention(st):
    case, Q = st["case"], st["Q"]
    bs, Hkv, G, W, S = case["bs"], case["Hkv"], case["Hq"] // case["Hkv"], case["W"], case["S"]
    qn, L = _lens(case)
    out = torch.empty_like(Q)
    at = 0
    for b in range(case["B"]):
        n, q = L[b], qn[b]
        first, lo = _seen(case, q, n)
        j = torch.cat([torch.arange(first, device="cuda"), torch.arange(lo, n, device="cuda")])
        slot = st["table"][b].long()[j // bs] * bs + j % bs
        K = st["K"].view(-1, Hkv, 128)[slot].float().permute(1, 2, 0)              # [Hkv, D, n]
        V = st["V"].view(-1, Hkv, 128)[slot].float().permute(1, 0, 2)              # [Hkv, n, D]
        x = Q[at:at + q].float().reshape(q, Hkv, G, 128).permute(1, 2, 0, 3).reshape(Hkv, G * q, 128)
        s = torch.matmul(x, K).mul_(st["scale"]).view(Hkv, G, q, j.numel())
        p = (n - q + torch.arange(q, device="cuda"))[:, None]
        s.masked_fill_((j[None, :] > p) | ((j[None, :] <= p - W) & (j[None, :] >= S)), float("-inf"))
        s = torch.exp(s.sub_(s.amax(-1, keepdim=True)))
        l = s.sum(-1, keepdim=True)
        o = torch.matmul(s.view(Hkv, G * q, j.numel()), V).view(Hkv, G, q, 128) / l
        out[at:at + q] = o.permute(2, 0, 1, 3).reshape(q, case["Hq"], 128).to(torch.bfloat16)
        at += q
    return out


# --------------------------------------------------------------------- run ---

def prepare(case, seed):
    if own:
        import invariant_deterministic_bi_gb300 as bi
    if case["op"] in ("rope", "qk", "kv"):
        st = dict(_row_inputs(case, seed), case=case)
        st["freqs"] = bi.rope_freqs(case["R"], **_freq_args(case)) if own else _plain_freqs(case)
        if case["op"] == "kv":
            shape = (st["blocks"], case["bs"], case["Hkv"], 128)
            st["Kc"], st["Vc"] = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return st
    Q, cu, K, V, table, lens = _attn_inputs(case, seed)
    q, L = _lens(case)
    st = dict(case=case, Q=Q, cu=cu, K=K, V=V, table=table, lens=lens, max_len=max(L), max_q=max(q), scale=128 ** -0.5)
    if own:
        W, S = case["W"], case["S"]
        size = (bi.attention_decode_window_workspace_size(case["B"], case["Hq"], max(L), W, S) if case["op"] == "decode" else
                bi.attention_extend_window_workspace_size(sum(q), case["Hq"], case["Hkv"], max(L), max(q), W, S))
        st["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size > 0 else None
    return st


def run(state):
    case = state["case"]
    if not own:
        return {"rope": _plain_rope, "qk": _plain_qk, "kv": _plain_kv, "decode": _plain_attention, "extend": _plain_attention}[case["op"]](state)
    import invariant_deterministic_bi_gb300 as bi
    if case["op"] == "rope":
        return bi.rope(state["X"], state["pos"], state["freqs"])
    if case["op"] == "qk":
        return bi.qk_norm_rope(state["Q"], state["K"], state["qw"], state["kw"], EPS, state["pos"], state["freqs"])
    if case["op"] == "kv":
        q = bi.kv_append(state["K"], state["V"], state["slots"], state["Kc"], state["Vc"], positions=state["pos"],
                         freqs=state["freqs"], k_weight=state["kw"], eps=EPS, Q=state["Q"], q_weight=state["qw"])
        return (state["Kc"], state["Vc"]) if q is None else (state["Kc"], state["Vc"], q)
    if case["op"] == "decode":
        return bi.attention_decode_window(state["Q"], state["K"], state["V"], state["table"], state["lens"], state["max_len"],
                                          state["scale"], case["W"], case["S"], workspace=state["workspace"])
    return bi.attention_extend_window(state["Q"], state["cu"], state["K"], state["V"], state["table"], state["lens"],
                                      state["max_len"], state["max_q"], state["scale"], case["W"], case["S"],
                                      workspace=state["workspace"])


# ------------------------------------------------------------------- exact ---

def _angles(case, pos):
    """cos and sin (with the factor) of every position and pair, from the definition."""
    R, s, b = case["R"], case["s"], 1e6
    if case["scaling"] == "ntk" and R > 2:
        b = b * math.pow(s, R / (R - 2.0))
    m = 1.0 + 0.1 * math.log(s) if case["scaling"] == "yarn" else 1.0
    fs = []
    for i in range(R // 2):
        f = 1.0 / math.pow(b, 2.0 * i / R)
        if case["scaling"] == "linear":
            f /= s
        if case["scaling"] == "bands":
            turns = 8192.0 * f / (2.0 * math.pi)
            if turns < 1.0:
                f /= s
            elif turns <= 4.0:
                part = (turns - 1.0) / (4.0 - 1.0)
                f = part * f + (1.0 - part) * f / s
        if case["scaling"] == "yarn":
            low = math.floor(R * math.log(8192.0 / (32.0 * 2.0 * math.pi)) / (2.0 * math.log(b)))
            high = math.ceil(R * math.log(8192.0 / (1.0 * 2.0 * math.pi)) / (2.0 * math.log(b)))
            low, high = max(low, 0), min(high, R - 1)
            part = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
            f = (1.0 - part) * f + part * f / s
        fs.append(f)
    angle = torch.outer(pos.double(), torch.tensor(fs, dtype=torch.float64, device="cuda"))
    return torch.cos(angle) * m, torch.sin(angle) * m


def _turned(case, x, pos, w=None):
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    c, s = (t[:, None, :] for t in _angles(case, pos))
    h = case["R"] // 2
    y = x.clone()
    one = slice(0, 2 * h, 2) if case["inter"] else slice(0, h)
    two = slice(1, 2 * h, 2) if case["inter"] else slice(h, 2 * h)
    y[:, :, one] = x[:, :, one] * c - x[:, :, two] * s
    y[:, :, two] = x[:, :, one] * s + x[:, :, two] * c
    return y


def exact(case, seed):
    if case["op"] in ("rope", "qk", "kv"):
        i = _row_inputs(case, seed)
        if case["op"] == "rope":
            return _turned(case, i["X"], i["pos"])
        if case["op"] == "qk":
            return _turned(case, i["Q"], i["pos"], i["qw"]), _turned(case, i["K"], i["pos"], i["kw"])
        n = case["T"]                                   # the padded tokens stand at the end
        out = []
        for rows in (_turned(case, i["K"], i["pos"], i["kw"]), i["V"].double()):
            cache = torch.zeros((i["blocks"] * case["bs"], case["Hkv"], 128), dtype=torch.float64, device="cuda")
            cache[i["slots"][:n]] = rows[:n]
            out.append(cache.reshape(i["blocks"], case["bs"], case["Hkv"], 128))
        if case["Hq"]:
            out.append(_turned(case, i["Q"], i["pos"], i["qw"]))
        return tuple(out)
    Q, cu, K, V, table, lens = _attn_inputs(case, seed)
    qn, L = _lens(case)
    bs, Hkv, G = case["bs"], case["Hkv"], case["Hq"] // case["Hkv"]
    out = torch.empty(Q.shape, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        a0, a1, n = int(cu[b]), int(cu[b + 1]), L[b]
        new = torch.arange(n - (a1 - a0), n, device="cuda")[:, None]
        old = torch.arange(n, device="cuda")
        far = old <= n - (a1 - a0) - case["W"]          # out of every new token's window
        old = old[~far | (old < case["S"])]
        see = (old[None, :] <= new) & ((new - old[None, :] < case["W"]) | (old[None, :] < case["S"]))
        rows = table[b].long()[torch.div(old, bs, rounding_mode="floor")], old % bs
        for h in range(Hkv):
            k, v = K[rows[0], rows[1], h].double(), V[rows[0], rows[1], h].double()
            for i in range(h * G, (h + 1) * G):
                s = (Q[a0:a1, i].double() @ k.T) * (128 ** -0.5)
                s = torch.where(see, s, torch.full_like(s, -math.inf))
                out[a0:a1, i] = torch.softmax(s, dim=-1) @ v
    return out
