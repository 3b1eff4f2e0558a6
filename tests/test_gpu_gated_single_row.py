"""One token or one feature: tensors of one row may be views of any row distance,
since the distance to a next row is not used."""
import pytest
import torch

import test_gpu_gated as G
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def _wide(t, cols):
    """The one row of t as a view into rows `cols` elements apart."""
    w = torch.full((3, cols), 5.0, dtype=t.dtype, device=t.device)
    w[1:2, :t.shape[1]] = t
    return w[1:2, :t.shape[1]]


@pytest.mark.parametrize("t,d,f", [(1, 64, 40), (1, 100, 1), (20, 64, 1), (300, 72, 1)])
def test_rows_of_any_distance(t, d, f):
    need_gpu()
    import post_weight_quantization_syrk_b200 as P
    X, Wg, Wu, dH = G._block(t + d, t, d, f)
    H = P.kq_gated_ffn(X, Wg, Wu, P.KQ_ACT_SILU)
    want = P.kq_gated_ffn_backward(X, Wg, Wu, dH, P.KQ_ACT_SILU)
    outs = [w.clone() for w in want]
    if t == 1:
        X, dH = _wide(X, 512), _wide(dH, 72)
        outs[0], outs[1], outs[2] = _wide(outs[0], 80), _wide(outs[1], 512), _wide(outs[2], 123)
    if f == 1:
        Wg, Wu = _wide(Wg, 512), _wide(Wu, 256)
        outs[3], outs[4] = _wide(outs[3], 131), _wide(outs[4], 512)
    if f == 1 and t > 1:
        outs[0], outs[1] = None, None
    assert torch.equal(P.kq_gated_ffn(X, Wg, Wu, P.KQ_ACT_SILU), H)
    got = P.kq_gated_ffn_backward(X, Wg, Wu, dH, P.KQ_ACT_SILU, outs[0], outs[1], dX=outs[2], dW_gate=outs[3], dW_up=outs[4])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for o in outs:
        if o is not None and o.shape[0] == 1 and o._base is not None:
            assert bool((o._base[[0, 2]] == 5.0).all()) and bool((o._base[1, o.shape[1]:] == 5.0).all())
