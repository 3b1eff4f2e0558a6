"""A 4-bit matrix takes its global scale from its own device only: the kernels
read it there."""
import pytest
import torch

import post_weight_quantization_syrk_b200 as P


class OnDevice:
    """Stands for a tensor on a CUDA device, on a machine without one."""

    def __init__(self, t, index=0):
        self.t, self.index = t, index

    def get_device(self):
        return self.index

    def new_empty(self, *shape, **kw):
        return self.t.new_empty(*shape, **kw)

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_empty_refuses_a_scale_from_elsewhere():
    like = OnDevice(torch.zeros(1))
    for g in (torch.ones(1), OnDevice(torch.ones(1), 1)):
        with pytest.raises(ValueError, match="one device"):
            P.Fp4Matrix.empty(4, 64, P.KQ_FP4_NV, like, g)
    q = P.Fp4Matrix.empty(4, 64, P.KQ_FP4_NV, like, OnDevice(torch.ones(1)))
    assert q.get_device() == 0 and q.codes.shape == (4, 32)
    with pytest.raises(TypeError):
        P.Fp4Matrix.empty(4, 64, P.KQ_FP4_NV, like, OnDevice(torch.ones(2)))
