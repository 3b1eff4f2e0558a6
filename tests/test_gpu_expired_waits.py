"""Kernels of the tile engine whose waits give up in the middle of a tile, at the
last load or at the end: either the wait limit was long enough and the result is
right, or the error is reported; the call returns soon, and the next is right."""
import time

import pytest
import torch

import test_gpu_fp4 as F
import test_gpu_gated as G
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

LIMITS = (0, 300, 1000, 3000, 10000, 30000)       # ns


@pytest.fixture(scope="module")
def P():
    need_gpu()
    import post_weight_quantization_syrk_b200 as P
    P.load()
    return P


def _under_limits(P, call, dev):
    want = [t.clone() for t in call(P.new_info(dev))]
    torch.cuda.synchronize()
    expired = 0
    for limit in LIMITS * 3:
        info = P.new_info(dev)
        torch.cuda.synchronize()
        t0 = time.monotonic()
        old = P.kq_set_wait_limit_ns(limit)
        try:
            got = call(info)
            torch.cuda.synchronize()
        finally:
            P.kq_set_wait_limit_ns(old)
        assert time.monotonic() - t0 < 2.0, limit        # no drain ran into its own bound (4 s)
        code = F._code(info)[0]
        assert code in (0, 8)
        expired += code == 8
        if code == 0:
            assert all(torch.equal(a, b) for a, b in zip(got, want)), limit
        info = P.new_info(dev)
        assert all(torch.equal(a, b) for a, b in zip(call(info), want)), limit
        assert F._code(info) == (0, 0)
    assert expired >= 3                                   # limit 0 at least


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("m,k,n", [(8, 8192, 3000), (300, 4096, 1000), (2304, 256, 2304), (2304, 4096, 2304), (4000, 1000, 4200)])
def test_4_bit_products(P, fmt, m, k, n):
    A, B = F._quant(P, F._data(1, m, k), fmt), F._quant(P, F._data(2, n, k), fmt)
    _under_limits(P, lambda info: [P.kq_fp4_gemm(A, B, info=info)], B.device)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_4_bit_gated(P, fmt):
    X, W = F._quant(P, F._data(1, 2304, 2048), fmt), F._quant(P, F._data(2, 1500, 2048) / 64, fmt)
    _under_limits(P, lambda info: [P.kq_fp4_gated_ffn(X, W, W, 0, info=info)], X.device)


@pytest.mark.parametrize("t,d,f", [(40, 2048, 1024), (2304, 2048, 1500)])
def test_gated_and_backward(P, t, d, f):
    X, Wg, Wu, dH = G._block(21, t, d, f)
    _under_limits(P, lambda info: [P.kq_gated_ffn(X, Wg, Wu, 0, info=info)], X.device)
    _under_limits(P, lambda info: P.kq_gated_ffn_backward(X, Wg, Wu, dH, 0, info=info), X.device)
