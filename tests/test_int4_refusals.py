"""The 4-bit calls refuse arguments of another kind with a TypeError that names them."""
import pytest

pytestmark = pytest.mark.gpu
D = 128


@pytest.mark.parametrize("other", [None, "cache", (1, 2, 3, 4)])
def test_a_cache_of_another_kind(bi, other):
    import torch
    K = torch.zeros((3, 2, D), dtype=torch.bfloat16, device="cuda")
    s = torch.arange(3, device="cuda")
    t, ln = torch.zeros((3, 1), dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    for call in (lambda: bi.kv_int4_append(K, K, s, other), lambda: bi.kv_int4_read(other, s),
                 lambda: bi.attention_decode_int4(K, other, t, ln, 16, 0.1),
                 lambda: bi.attention_extend_int4(K, cu, other, t, ln, 16, 1, 0.1)):
        with pytest.raises(TypeError, match="KVInt4Cache"):
            call()


def test_tensors_of_another_kind(bi):
    import torch
    c = bi.kv_int4_cache(4, 16, 2)
    K = torch.zeros((3, 2, D), dtype=torch.bfloat16, device="cuda")
    s = torch.arange(3, device="cuda")
    t, ln = torch.zeros((3, 1), dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    X = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    W = torch.zeros((16, 64), dtype=torch.uint8, device="cuda")
    S = torch.zeros((16, 4), dtype=torch.bfloat16, device="cuda")
    for name, call in (("K", lambda x: bi.kv_int4_append(x, K, s, c)), ("V", lambda x: bi.kv_int4_append(K, x, s, c)),
                       ("slots", lambda x: bi.kv_int4_append(K, K, x, c)), ("slots", lambda x: bi.kv_int4_read(c, x)),
                       ("V", lambda x: bi.kv_int4_read(c, s, V=x)), ("Q", lambda x: bi.attention_decode_int4(x, c, t, ln, 16, 0.1)),
                       ("seq_lens", lambda x: bi.attention_decode_int4(K, c, t, x, 16, 0.1)),
                       ("workspace", lambda x: bi.attention_decode_int4(K, c, t, ln, 16, 0.1, workspace=x)),
                       ("O", lambda x: bi.attention_decode_int4(K, c, t, ln, 16, 0.1, O=x)),
                       ("cu_q", lambda x: bi.attention_extend_int4(K, x, c, t, ln, 16, 1, 0.1)),
                       ("X", lambda x: bi.gemm_int4(x, W, S)), ("W", lambda x: bi.gemm_int4(X, x, S)),
                       ("scales", lambda x: bi.gemm_int4(X, W, x)), ("zeros", lambda x: bi.gemm_int4(X, W, S, zeros=x)),
                       ("Y", lambda x: bi.gemm_int4(X, W, S, Y=x))):
        for other in ([1, 2], torch.zeros(3, dtype=torch.float64, device="cuda")):
            with pytest.raises(TypeError, match=name):
                call(other)
    assert bi.device_status() == bi.BI_OK
