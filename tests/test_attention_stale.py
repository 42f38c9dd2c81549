"""What a cache block holds behind a sequence's end (rows never written, or left by an earlier sequence) does not
reach the results of attention, be it infinite or NaN."""
import numpy as np
import pytest

import bi_synth as syn
from util import bits_of, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu
D = 128


@pytest.mark.parametrize("bs", [8, 16, 24, 64, 128, 256])
@pytest.mark.parametrize("B,Hq,Hkv", [(5, 4, 4), (5, 16, 2), (120, 16, 4)])     # an item a CTA, and the ring
def test_rows_behind_a_sequence_do_not_reach_it(bi, B, Hq, Hkv, bs):
    import torch
    r = syn.rng(bs, B + Hq)
    lens = np.concatenate([[1, 17, 127, 129, 260], r.integers(1, 400, B)])[:B].astype(np.int32)
    nb = -(-400 // bs)
    blocks = B * nb
    table = r.permutation(blocks).astype(np.int32).reshape(B, nb)
    K, V = (syn.to_bf16_bits(syn.normal_rows(s, 0, blocks * bs, Hkv * D)).reshape(blocks, bs, Hkv, D) for s in (1, 2))
    stale_k, stale_v = K.copy(), V.copy()
    for b in range(B):
        for j in range(lens[b], nb * bs):
            stale_k[table[b, j // bs], j % bs] = 0x7FC0                          # NaN
            stale_v[table[b, j // bs], j % bs] = (0x7FC0, 0x7F80, 0xFF80)[j % 3] # NaN, infinities
    Q = to_dev_bf16(syn.to_bf16_bits(syn.normal_rows(3, 0, B * Hq, D)).reshape(B, Hq, D))
    td, ld = to_dev(table), to_dev(lens)
    want = bi.attention_decode(Q, to_dev_bf16(K), to_dev_bf16(V), td, ld, 400, D ** -0.5)
    Ks, Vs = to_dev_bf16(stale_k), to_dev_bf16(stale_v)
    got = bi.attention_decode(Q, Ks, Vs, td, ld, 400, D ** -0.5)
    assert np.array_equal(bits_of(got), bits_of(want)) and bool(torch.isfinite(got).all())
    cu = to_dev(np.arange(B + 1, dtype=np.int32))
    assert np.array_equal(bits_of(bi.attention_extend(Q, cu, Ks, Vs, td, ld, 400, 1, D ** -0.5)), bits_of(want))
    # over the 4-bit cache of the same rows
    outs = []
    for k, v in ((K, V), (stale_k, stale_v)):
        c = bi.kv_int4_cache(blocks, bs, Hkv)
        bi.kv_int4_append(to_dev_bf16(k).view(-1, Hkv, D), to_dev_bf16(v).view(-1, Hkv, D), torch.arange(blocks * bs, device="cuda"), c)
        outs += [bi.attention_decode_int4(Q, c, td, ld, 400, D ** -0.5)]
        outs += [bi.attention_extend_int4(Q, cu, c, td, ld, 400, 1, D ** -0.5, workspace=w)
                 for w in (None, torch.empty(16, dtype=torch.uint8, device="cuda"))]
    assert all(np.array_equal(bits_of(o), bits_of(outs[0])) for o in outs) and bool(torch.isfinite(outs[0]).all())
    assert bi.device_status() == bi.BI_OK
