"""Runs seeded calls of the operators over heads and of windowed attention on the GPU and prints a digest of each
output and the final device status, one JSON line: run with the release and with the bounds-checked debug library
(BI_LIBRARY=debug), the digests have to agree. Not collected by pytest (helper script)."""
import hashlib
import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import invariant_deterministic_bi_gb300 as bi  # noqa: E402


def digest(*ts):
    return [hashlib.sha256(t.contiguous().view(torch.uint8).cpu().numpy().tobytes()).hexdigest()[:16] for t in ts]


def main():
    bi.load()
    out = {"debug_build": bi.debug_build()}
    g = torch.Generator(device="cuda").manual_seed(5)
    bf = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)
    for T in (1, 37, 3000):
        for D, R, inter in ((128, 128, False), (128, 64, True), (64, 32, False), (256, 96, True), (80, 80, False)):
            x, w, pos = bf(T, 9, D), bf(D), torch.arange(T, device="cuda") * 31
            fr = bi.rope_freqs(R, interleaved=inter)
            Kc, Vc = (torch.zeros((-(-T // 16) + 1, 16, 2, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            slots = torch.randperm(Kc.shape[0] * 16, device="cuda", generator=g)[:T]
            q = bi.kv_append(x[:, 5:7], x[:, 7:], slots, Kc, Vc, pos, fr, k_weight=w, Q=x[:, :5], q_weight=w)
            out[f"heads{T}_{D}"] = digest(bi.rope(x, pos, fr), *bi.qk_norm_rope(x[:, :5], x[:, 5:], w, w, 1e-6, pos, fr), Kc, Vc, q)
    for Hq, Hkv, bs in ((8, 2, 16), (8, 1, 24), (8, 1, 20), (4, 4, 128)):
        nb = -(-2600 // bs)
        K, V = bf(4 * nb, bs, Hkv, 128), bf(4 * nb, bs, Hkv, 128)
        table = torch.randperm(4 * nb, device="cuda", generator=g).to(torch.int32).view(4, nb)
        lens = torch.tensor([2600, 900, 130, 1], dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, 300, 303, 433, 434], dtype=torch.int32, device="cuda")
        Q, q = bf(434, Hq, 128), bf(4, Hq, 128)
        many = torch.arange(4, device="cuda").repeat(40)
        for W, S in ((100, 4), (1000, 0), (2500, 200)):
            small = torch.empty(16, dtype=torch.uint8, device="cuda")
            out[f"attention{bs}_{W}"] = digest(
                bi.attention_decode_window(q, K, V, table, lens, 2600, 0.09, W, S),
                bi.attention_decode_window(q[many], K, V, table[many].contiguous(), lens[many], 2600, 0.09, W, S),
                bi.attention_extend_window(Q, cu, K, V, table, lens, 2600, 300, 0.09, W, S),
                bi.attention_extend_window(Q, cu, K, V, table, lens, 2600, 300, 0.09, W, S, workspace=small))
    torch.cuda.synchronize()
    out["status"] = bi.status_string(bi.device_status())
    print(json.dumps(out), flush=True)


if __name__ == "__main__":
    main()
