"""The 4-bit and gated products where K is split over eight CTAs or is shorter
than the ring, on a stream that is not the current one, and with waits that give
up after every load has been issued."""
import pytest
import torch

import test_gpu_fp4 as F
import test_gpu_gated as G
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    need_gpu()
    import post_weight_quantization_syrk_b200 as P
    P.load()
    return P


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("m,k,n", [(1, 8192, 100), (16, 8200, 300), (64, 8448, 1000), (64, 1280, 128), (60, 2050, 700)])
def test_products_of_few_rows(P, fmt, m, k, n):
    """Few tiles and long K: over 8, 4, 2 CTAs and one, pieces of unequal length."""
    F.test_gemm(P, fmt, m, k, n)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("t,d,f", [(16, 8200, 130), (64, 8448, 500), (3, 2050, 70)])
def test_fp4_gated_of_few_rows(P, fmt, t, d, f):
    F.test_fp4_gated(P, fmt, "silu", t, d, f)


@pytest.mark.parametrize("t,d,f", [(1, 4096, 300), (16, 4100, 500), (64, 2200, 512), (100, 2048, 64)])
def test_gated_of_few_rows(P, t, d, f):
    G.test_forward(P, "silu", t, d, f)


def _busy_block(nbytes):
    """Frees a block of the current stream's whose last write is still queued
    behind some milliseconds of other work."""
    big = torch.zeros((4096, 4096), device="cuda")
    block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    for _ in range(40):
        torch.mm(big, big)
    block.fill_(0xA5)


def test_results_belong_to_the_stream_given(P):
    """Outputs that a call with a stream allocates are not memory that the current
    stream still writes to."""
    M, W = F._data(1, 256, 2048, torch.bfloat16), F._data(2, 512, 2048, torch.bfloat16)
    act = P.KQ_ACT_SILU
    dH = F._data(3, 256, 512, torch.bfloat16)

    def calls(**kw):
        A, B = P.kq_fp4_quantize(M, P.KQ_FP4_MX, **kw), P.kq_fp4_quantize(W, P.KQ_FP4_MX, **kw)
        return [A.codes, P.kq_fp4_gemm(A, B, **kw), P.kq_fp4_matvec(B, M[:3], **kw), P.kq_fp4_gated_ffn(A, B, B, act, **kw),
                P.kq_gated_ffn(M, W, W, act, **kw), *P.kq_gated_ffn_backward(M, W, W, dH, act, **kw)]

    want = [t.clone() for t in calls()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i, w in enumerate(want):
        # a freed block of each output's size, in turn
        nbytes = w.numel() * w.element_size() if i else w.numel() + 256 // 128 * 2048 // 128 * 512
        _busy_block(nbytes)
        got = calls(stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("m,k", [(40, 256), (40, 1024), (2304, 256), (2304, 1000)])
def test_expired_wait_after_the_last_load(P, fmt, m, k):
    """Wait limit 0 where the ring holds all of K: the producer never waits, the
    other warps give up; the error is reported and the next call is right."""
    A, B = F._quant(P, F._data(1, m, k), fmt), F._quant(P, F._data(2, 2304, k), fmt)
    want = P.kq_fp4_gemm(A, B)
    torch.cuda.synchronize()
    info = P.new_info(want.device)
    old = P.kq_set_wait_limit_ns(0)
    try:
        P.kq_fp4_gemm(A, B, info=info)
        torch.cuda.synchronize()
    finally:
        P.kq_set_wait_limit_ns(old)
    assert F._code(info)[0] == 8
    assert torch.equal(P.kq_fp4_gemm(A, B), want)
