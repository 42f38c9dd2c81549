"""bi_gemm_int4 with groups longer than the 128 k of a product block: K segments that begin inside a group, and stages
of 256 k that end in another group than they begin in, in the kernels for few rows and for many."""
import numpy as np
import pytest

import bi_synth as syn
from test_gemm_int4 import check, inputs, run
from util import bits_of

pytestmark = pytest.mark.gpu


def starts(K):
    """First 128-k block of each segment: units of 256 k, two a segment at least, eight segments at most."""
    units = -(-K // 256)
    n = 1 if units < 4 else min(8, units // 2)
    return [2 * (s * units // n) for s in range(n)]


# groups of 3, 4, 5, 6 and 9 blocks; 8, 8, 8, 4 and 4 segments
@pytest.mark.parametrize("g,K", [(384, 4608), (512, 4096), (640, 5120), (768, 2304), (1152, 2304)])
@pytest.mark.parametrize("zeros", [False, True])
def test_segments_that_begin_inside_a_group(bi, g, K, zeros):
    if g != 512:
        assert any(b % (g // 128) for b in starts(K))
    # scales that differ by group by far, so that a block with its neighbour's scale or zero shows
    X, W, S, Z = inputs(130, 136, K, g, zeros, seed=g)
    factor = 2.0 ** (syn.rng(g, 3).integers(-3, 4, (1, K // g)))
    S = syn.to_bf16_bits((syn.bf16_bits_to_f32(S) * factor).astype(np.float32))
    full = run(bi, X, W, S, Z)
    check(full, X, W, S, Z)                               # bounds what sums of K / 128 scaled blocks add: fewer than K / 16
    full = bits_of(full)
    for rows in (range(1), range(9), range(16), range(17), range(64), range(129, 130), range(100, 117)):
        rows = np.array(list(rows))
        assert np.array_equal(bits_of(run(bi, X[rows], W, S, Z)), full[rows]), rows
    assert bi.device_status() == bi.BI_OK
