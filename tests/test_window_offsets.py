"""A windowed extend call one of whose offsets is out of range: the sequences that begin or end there are left as they
were, every other one has the result that it has without that, split over the chunks or in tiles."""
import numpy as np
import pytest

import bi_synth as syn
from test_attention_window import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [5, 33, 100, 1100])
def test_an_offset_out_of_range_leaves_the_other_sequences(bi, n):
    import torch
    W, S = 90, 4
    r = syn.rng(n, 1)
    q = [int(x) for x in r.integers(1, 6, n)]
    for b in range(0, n, max(1, n // 5)):
        q[b] = int(r.integers(1, 90))
    c = Case([x + int(r.integers(0, 60)) for x in q], q, 8, 2, 16, seed=n)
    want = c.extend(bi, W, S)
    for k in sorted({0, 1, n // 2, n - 2, n - 1, n}):
        for value in (-1, -1000, -(1 << 31), len(want) + 1, 1 << 20, (1 << 31) - 1):
            cu = c.cu_np.copy()
            cu[k] = value
            keep = np.ones(n, bool)
            keep[max(0, k - 1):k + 1] = False
            keep = torch.from_numpy(np.repeat(keep, q)).cuda()
            for call in (c.extend, c.tiled):
                O = torch.full_like(want, 7.0)
                call(bi, W, S, O=O, cu=torch.from_numpy(cu).cuda())
                assert bi.device_status() == bi.BI_ERR_INVALID_ARG
                assert torch.equal(O[keep], want[keep]), (k, value)
                assert (O[~keep] == 7.0).all(), (k, value)
