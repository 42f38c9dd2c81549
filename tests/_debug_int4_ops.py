"""Runs one seeded call of every 4-bit operator on the GPU and prints a digest of each output and the final
device status, one JSON line: run with the release and with the bounds-checked debug library (BI_LIBRARY=debug),
the digests have to agree. Not collected by pytest (helper script)."""
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
    g = torch.Generator(device="cuda").manual_seed(4)
    bf = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)
    for bs in (16, 24):                                   # block copies, row copies
        Hq, Hkv, nb = 32, 8, 40
        lens = torch.tensor([300, 17, 8 * bs], dtype=torch.int32, device="cuda")
        c = bi.kv_int4_cache(3 * nb, bs, Hkv)
        for T in (5, 3 * nb * bs):                        # one head a warp, four
            slots = torch.randperm(3 * nb * bs, device="cuda", generator=g)[:T]
            bi.kv_int4_append(bf(T, Hkv, 128), bf(T, Hkv, 128), slots, c)
        out[f"cache{bs}"] = digest(*c)
        out[f"read{bs}"] = digest(*bi.kv_int4_read(c, torch.arange(50, device="cuda") - 1))
        table = torch.randperm(3 * nb, device="cuda", generator=g).to(torch.int32).view(3, nb)
        q = bf(3, Hq, 128)
        out[f"decode{bs}"] = digest(bi.attention_decode_int4(q, c, table, lens, nb * bs, 128 ** -0.5))
        cu = torch.tensor([0, 5, 6, 46], dtype=torch.int32, device="cuda")
        Q = bf(46, Hq, 128)
        for ws in (None, torch.empty(16, dtype=torch.uint8, device="cuda")):
            for most in (40, 16):                         # tiled; 16 refuses the third sequence
                O = torch.zeros_like(Q)
                bi.attention_extend_int4(Q, cu, c, table, lens, nb * bs, most, 128 ** -0.5, workspace=ws, O=O)
                out[f"extend{bs}_{ws is None}_{most}"] = digest(O)
                torch.cuda.synchronize()
                out[f"extend_status{bs}_{ws is None}_{most}"] = bi.status_string(bi.device_status())
    for M in (1, 3, 8, 16, 17, 40, 70):
        for K, grp in ((4096, 128), (1056, 32), (1088, 64), (768, 384)):
            N = 264
            W = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
            S = torch.rand((N, K // grp), device="cuda", generator=g).to(torch.bfloat16)
            Z = torch.randint(0, 16, (N, K // grp), dtype=torch.uint8, device="cuda", generator=g)
            X = bf(M, K)
            out[f"gemm{M}_{K}"] = digest(bi.gemm_int4(X, W, S), bi.gemm_int4(X, W, S, zeros=Z))
    torch.cuda.synchronize()
    out["status"] = bi.status_string(bi.device_status())
    print(json.dumps(out), flush=True)


if __name__ == "__main__":
    main()
