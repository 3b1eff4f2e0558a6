"""An output given at the address of another tensor of the call is refused on the
host (the addresses are never read)."""
import pytest

import post_weight_quantization_syrk_b200 as P
from post_weight_quantization_syrk_b200 import _lib as K

AT = [0x100000 * (i + 1) for i in range(11)]
INPUTS, OUTPUTS = ("X", "W_gate", "W_up", "dH"), ("dG", "dU", "H", "dX", "dW_gate", "dW_up")


def backward(**same):
    at = dict(zip(INPUTS + OUTPUTS, AT), info=AT[-1])
    at.update({k: at[v] for k, v in same.items()})
    t, d, f = 32, 64, 128
    return K.load().kq_gated_ffn_backward(
        at["X"], t, d, d, at["W_gate"], at["W_up"], f, d, P.KQ_ACT_SILU, at["dH"], f, at["dG"], at["dU"], f, at["H"], f,
        at["dX"], d, at["dW_gate"], at["dW_up"], d, at["info"], None)


@pytest.mark.parametrize("out,other", [(o, x) for o in OUTPUTS for x in INPUTS + OUTPUTS if x != o])
def test_backward(out, other):
    assert backward(**{out: other}) == 1
    assert b"another tensor" in K.load().kq_last_error()


@pytest.mark.parametrize("other", [0, 1, 2])
def test_forward(other):
    L = K.load()
    assert L.kq_gated_ffn(AT[0], 8, 64, 64, AT[1], AT[2], 32, 64, P.KQ_ACT_GELU, AT[other], 64, AT[3], None) == 1
    assert b"another tensor" in L.kq_last_error()


def test_quantize():
    L = K.load()
    q = K.kq_fp4(16, 64, 32, P.KQ_FP4_MX, AT[0], AT[1], None)
    assert L.kq_fp4_quantize(AT[2], P.KQ_F32, 64, q, AT[2], 64, AT[3], None) == 1
    assert b"overlap" in L.kq_last_error()
