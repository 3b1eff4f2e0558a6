"""4-bit products of up to 8 rows, whose ring of 5 stages is walked more than once:
the scales of every stage are those of its own columns, in every run."""
import pytest
import torch

import test_gpu_fp4 as F
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    need_gpu()
    import post_weight_quantization_syrk_b200 as P
    P.load()
    return P


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("m,k,n", [(1, 4096, 11008), (8, 11008, 3000), (5, 8200, 2000), (8, 2048, 20000), (3, 28672, 500)])
def test_scales_of_a_long_ring(P, fmt, m, k, n):
    A, B = F._quant(P, F._data(m + k, m, k), fmt), F._quant(P, F._data(n + k, n, k, torch.bfloat16), fmt)
    info = P.new_info(B.device)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    Y = P.kq_fp4_gemm(A, B, dtype=torch.float32, info=info)
    F._check(Y, F._values(A, fmt), F._values(B, fmt), False)
    for i in range(60):
        if i % 3 == 0:
            flush.fill_(i)                     # weights from memory, where copies land late and out of order
        assert torch.equal(P.kq_fp4_gemm(A, B, dtype=torch.float32, info=info), Y)
    assert F._code(info) == (0, 0)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("t,d,f", [(1, 4096, 2000), (8, 11008, 1500)])
def test_scales_of_a_long_ring_gated(P, fmt, t, d, f):
    X = F._quant(P, F._data(t, t, d), fmt)
    Wg, Wu = (F._quant(P, F._data(s, f, d, torch.bfloat16) / d, fmt) for s in (2, 3))
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    H = P.kq_fp4_gated_ffn(X, Wg, Wu, P.KQ_ACT_SILU)
    assert bool(torch.isfinite(H).all())
    for i in range(30):
        if i % 3 == 0:
            flush.fill_(i)
        assert torch.equal(P.kq_fp4_gated_ffn(X, Wg, Wu, P.KQ_ACT_SILU), H)
