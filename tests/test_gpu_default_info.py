"""Device errors of calls without an `info` of their own are kept in the device's
default word, where check_info() finds them."""
import os
import subprocess
import sys

import pytest
import torch

import test_gpu_fp4 as F
import test_gpu_gated as G
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture()
def P():
    need_gpu()
    import post_weight_quantization_syrk_b200 as P
    P.load()
    P.default_info().zero_()
    torch.cuda.synchronize()
    yield P
    P.default_info().zero_()


def _raises(P, status):
    with pytest.raises(P.KronqError) as e:
        P.check_info(P.default_info(), "test")
    assert e.value.status == status
    P.default_info().zero_()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_bad_values(P, fmt):
    M = F._data(1, 40, 128)
    g = torch.tensor([0.01], device="cuda") if fmt == "nv" else None
    P.kq_fp4_quantize(M, F._fmt(P, fmt), g)
    P.check_info(P.default_info())
    M[17, 3] = float("nan")
    own = P.new_info(M.device)
    P.kq_fp4_quantize(M, F._fmt(P, fmt), g, info=own)          # an info of its own: recorded there
    P.check_info(P.default_info())
    assert F._code(own) == (7, 17)
    P.kq_fp4_quantize(M, F._fmt(P, fmt), g)
    M[17, 3] = 1.0
    P.kq_fp4_quantize(M, F._fmt(P, fmt), g)                    # the first error sticks
    _raises(P, 7)
    P.check_info(P.default_info())


def test_expired_waits(P):
    A, B = F._quant(P, F._data(1, 300, 4096), "mx"), F._quant(P, F._data(2, 1000, 4096), "mx")
    X, Wg, Wu, dH = G._block(21, 300, 2048, 1024)
    for call in (lambda: P.kq_fp4_gemm(A, B), lambda: P.kq_fp4_gated_ffn(A, B, B, 0), lambda: P.kq_gated_ffn(X, Wg, Wu, 0),
                 lambda: P.kq_gated_ffn_backward(X, Wg, Wu, dH, 0)):
        call()
        P.check_info(P.default_info())
        old = P.kq_set_wait_limit_ns(0)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            P.kq_set_wait_limit_ns(old)
        _raises(P, 8)


def test_other_streams_and_devices_words(P):
    M = F._data(1, 8, 64)
    M[2, 2] = float("inf")
    torch.cuda.synchronize()
    P.kq_fp4_quantize(M, P.KQ_FP4_MX, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    _raises(P, 7)
    assert P.default_info("cuda").data_ptr() == P.default_info(M.device).data_ptr() == P.default_info().data_ptr()


def test_first_call_is_captured():
    """The word needs no allocation: a process whose first call is captured records in it."""
    need_gpu()
    script = """
import torch
import post_weight_quantization_syrk_b200 as P
M = torch.ones((4, 64), device="cuda")
M[3, 5] = float("nan")
side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.stream(side):
    with torch.cuda.graph(graph, stream=side):
        Q = P.kq_fp4_quantize(M, P.KQ_FP4_MX)
P.check_info(P.default_info())
graph.replay()
torch.cuda.synchronize()
try:
    P.check_info(P.default_info())
except P.KronqError as e:
    assert e.status == 7
    print("recorded")
"""
    r = subprocess.run([sys.executable, "-c", script], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "recorded", r.stderr[-2000:]


def test_wrong_words_are_refused(P):
    A = F._quant(P, F._data(1, 8, 64), "mx")
    for info in (torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")):
        with pytest.raises(TypeError, match="info"):
            P.kq_fp4_gemm(A, A, info=info)
