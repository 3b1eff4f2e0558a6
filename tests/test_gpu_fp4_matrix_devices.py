"""Fp4Matrix refuses codes, scales and a global scale that do not lie together."""
import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def test_parts_from_the_host_are_refused():
    need_gpu()
    import post_weight_quantization_syrk_b200 as P
    M = torch.ones((8, 64), device="cuda")
    with pytest.raises(ValueError, match="one device"):
        P.Fp4Matrix.empty(8, 64, P.KQ_FP4_NV, M, torch.ones(1))
    g = torch.ones(1, device="cuda")
    Q = P.kq_fp4_quantize(M, P.KQ_FP4_NV, g, out=P.Fp4Matrix.empty(8, 64, P.KQ_FP4_NV, M, g))
    for codes, scales, gscale in ((Q.codes, Q.scales.cpu(), g), (Q.codes, Q.scales, g.cpu()), (Q.codes, Q.scales.cpu(), g.cpu())):
        with pytest.raises(ValueError, match="one device"):
            P.Fp4Matrix(8, 64, P.KQ_FP4_NV, codes, scales, gscale)
    # 1 / 6 as E4M3 is 11 / 64, the codes 6: 64 (6 * 11 / 64)^2 = 68.06, 68 in bf16
    assert torch.equal(P.kq_fp4_gemm(Q, P.Fp4Matrix(8, 64, P.KQ_FP4_NV, Q.codes, Q.scales, g)),
                       torch.full((8, 8), 68.0, dtype=torch.bfloat16, device="cuda"))
