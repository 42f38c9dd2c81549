"""bi_gemm_int4 on the GPU: the linear layer with 4-bit weights and group
scales against a plain 64-bit form, and its row's independence of the batch."""
import numpy as np
import pytest

import bi_synth as syn
import int4_ref as ref
from util import bits_of, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


def inputs(M, N, K, g, zeros, seed):
    r = syn.rng(seed, 7)
    X = syn.to_bf16_bits(syn.normal_rows(seed, 0, M, K))
    W = r.integers(0, 256, (N, K // 2)).astype(np.uint8)
    S = syn.to_bf16_bits((0.01 * (0.5 + r.random((N, K // g)))).astype(np.float32))
    Z = r.integers(0, 16, (N, K // g)).astype(np.uint8) if zeros else None
    return X, W, S, Z


def run(bi, X, W, S, Z, **kw):
    return bi.gemm_int4(to_dev_bf16(X), to_dev(W), to_dev_bf16(S), zeros=None if Z is None else to_dev(Z), **kw)


def check(got, X, W, S, Z):
    """One bf16 rounding (2^-8 of the value), and sums in fp32: each of the at most K / 16 + K / g + 8 additions
    of a chain is off by at most 2^-22 of the sum of magnitudes (the tensor cores may cut instead of round)."""
    x, s = syn.bf16_bits_to_f32(X).astype(np.float64), syn.bf16_bits_to_f32(S).astype(np.float64)
    want, mag = ref.gemm(x, W, s, Z)
    K = X.shape[1]
    tol = 2.0 ** -8 * np.abs(want) + (K / 16 + S.shape[1] + 8) * 2.0 ** -22 * mag
    err = np.abs(got.float().cpu().numpy() - want)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("g,K", [(32, 32), (32, 160), (32, 1056), (64, 64), (64, 1088), (128, 128), (128, 1152),
                                 (256, 768), (384, 384)])
@pytest.mark.parametrize("M,N,zeros", [(1, 8, False), (3, 24, True), (8, 40, True), (17, 136, False), (70, 16, True)])
def test_parity(bi, M, N, K, g, zeros):
    a = inputs(M, N, K, g, zeros, seed=M + N)
    check(run(bi, *a), *a)
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("K,g", [(4096, 128), (4096, 64), (4224, 32)])
def test_rows_do_not_depend_on_the_batch(bi, K, g):
    """Every row alone gives the bits it has among 1, 9, 16, 31, 33, 64, 65 and 200 rows, at any place."""
    X, W, S, Z = inputs(200, 264, K, g, True, seed=5)
    full = bits_of(run(bi, X, W, S, Z))
    check(run(bi, X[:40], W, S, Z), X[:40], W, S, Z)
    for rows in ([0], [199], range(9), range(100, 116), range(31), range(33, 66), range(64), range(65)):
        rows = np.array(list(rows))
        assert np.array_equal(bits_of(run(bi, X[rows], W, S, Z)), full[rows]), rows
    perm = syn.rng(6, 0).permutation(200)
    assert np.array_equal(bits_of(run(bi, X[perm], W, S, Z)), full[perm])


@pytest.mark.parametrize("M,N,K,g", [(2500, 2048, 1024, 128), (1290, 4104, 1056, 32)])
def test_many_tiles(bi, M, N, K, g):
    """More tiles than the GPU holds at once: the same bits as the rows alone, and parity on some of them."""
    a = X, W, S, Z = inputs(M, N, K, g, True, seed=11)
    full = run(bi, *a)
    for rows in (slice(0, 1), slice(M - 5, M), slice(60, 76), slice(100, 140)):
        part = run(bi, X[rows], W, S, Z)
        assert np.array_equal(bits_of(part), bits_of(full[rows])), rows
    check(full[-5:], X[-5:], W, S, Z)


def test_strided_rows(bi):
    """X and Y as column slices of wider buffers: nothing outside Y's slice is written."""
    import torch
    X, W, S, Z = inputs(5, 48, 256, 64, False, seed=8)
    want = run(bi, X, W, S, Z)
    wide = torch.full((5, 256 + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:264] = to_dev_bf16(X)
    out = torch.full((5, 80), 7.0, dtype=torch.bfloat16, device="cuda")
    bi.gemm_int4(wide[:, 8:264], to_dev(W), to_dev_bf16(S), Y=out[:, 16:64])
    assert torch.equal(out[:, 16:64], want) and bool((out[:, :16] == 7).all()) and bool((out[:, 64:] == 7).all())


def test_special_values(bi):
    """An infinity or NaN in a row of X stays in that row; zeros above 15 count their low four bits; scale 0 gives 0."""
    import torch
    X, W, S, Z = inputs(4, 16, 128, 32, True, seed=9)
    clean = run(bi, X, W, S, Z)
    bad = X.copy()
    bad[2, 5] = 0x7F80
    got = run(bi, bad, W, S, Z)
    assert torch.equal(got[[0, 1, 3]], clean[[0, 1, 3]]) and not bool(torch.isfinite(got[2]).any())
    assert torch.equal(run(bi, X, W, S, Z | 0xF0), clean)
    assert not run(bi, X, W, np.zeros_like(S), Z).any()


def test_refusals(bi):
    import torch
    X = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    W = torch.zeros((16, 64), dtype=torch.uint8, device="cuda")
    S = torch.zeros((16, 4), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        bi.gemm_int4(X, W.int(), S)
    with pytest.raises(TypeError):
        bi.gemm_int4(X, W, S.float())
    with pytest.raises(ValueError):
        bi.gemm_int4(X[:, :64], W, S)
    with pytest.raises(ValueError):
        bi.gemm_int4(X, W, S, zeros=torch.zeros((16, 2), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        bi.gemm_int4(X.t().contiguous().t(), W, S)
    for groups in (8, 16):                                # groups of 16 and 8
        with pytest.raises(bi.BiError) as e:
            bi.gemm_int4(X, W, torch.zeros((16, groups), dtype=torch.bfloat16, device="cuda"))
        assert e.value.status == bi.BI_ERR_UNSUPPORTED
    with pytest.raises(bi.BiError) as e:
        bi.gemm_int4(X, W[:4], S[:4])                     # N % 8
    assert e.value.status == bi.BI_ERR_UNSUPPORTED
    wide = torch.zeros((2, 132), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(bi.BiError) as e:
        bi.gemm_int4(wide[:, 4:], W, S)
    assert e.value.status == bi.BI_ERR_MISALIGNED
    assert bi.gemm_int4(X[:0], W, S).shape == (0, 16)
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("g,zeros", [(128, False), (64, True), (32, False)])
@pytest.mark.parametrize("M,N,K", [(17, 6144, 4096), (64, 6144, 4096), (96, 6144, 4096), (130, 6144, 4096), (200, 4096, 12288)])
def test_every_form_of_the_tiles_has_the_bits_of_single_rows(bi, M, N, K, g, zeros):
    """Tiles of 32 and 64 rows, with a segment a CTA or all of them (the sizes choose): the rows kernel's bits."""
    import torch
    X, W, S, Z = inputs(M, N, K, g, zeros, seed=M + g)
    Y = run(bi, X, W, S, Z)
    for m in sorted({0, 15, 16, 31, 32, 63, M // 2, M - 1} & set(range(M))):
        assert torch.equal(Y[m:m + 1], run(bi, X[m:m + 1], W, S, Z))
    check(Y[:, -24:], X, W[-24:], S[-24:], Z[-24:] if zeros else None)
    assert bi.device_status() == bi.BI_OK
