"""Calls in a row that hand on the same buffers: each kernel may be scheduled while
the one before still runs, and reads what that one wrote, not what was there."""
import pytest
import torch

import test_gpu_fp4 as F
import test_gpu_gated as G
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("captured", [False, True])
def test_buffers_handed_on(fmt, dtype, captured):
    need_gpu()
    import post_weight_quantization_syrk_b200 as P
    d, f, n, steps = 512, 768, 640, 24
    Ws = F._quant(P, F._data(1, f, d), fmt)
    Wv = F._quant(P, F._data(2, n, f), fmt)
    Xs = [F._data(10 + i, 8, d, torch.bfloat16) for i in range(steps)]
    g = torch.tensor([0.5], device="cuda") if fmt == "nv" else None
    info = P.new_info("cuda")
    Q = F._quant(P, Xs[0], fmt, g=g)
    Y = torch.empty((8, f), dtype=F.DT[dtype], device="cuda")          # written and read in every step
    V = torch.empty((8, n), dtype=F.DT[dtype], device="cuda")

    def step(i, wait):
        for call in (lambda: P.kq_fp4_quantize(Xs[i], F._fmt(P, fmt), g, out=Q, info=info),
                     lambda: P.kq_fp4_gemm(Q, Ws, Y, info=info), lambda: P.kq_fp4_matvec(Wv, Y, V)):
            call()
            if wait:
                torch.cuda.synchronize()
        return V.clone()

    want = [step(i, True) for i in range(steps)]
    if captured:
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                got = [step(i, False) for i in range(steps)]
    for _ in range(5):
        if captured:
            graph.replay()
        else:
            got = [step(i, False) for i in range(steps)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    P.check_info(info)


def test_gradients_handed_on():
    """The block's gradients into the same buffers, step after step."""
    need_gpu()
    import post_weight_quantization_syrk_b200 as P
    blocks = [G._block(i, 70, 264, 328) for i in range(6)]
    want = [P.kq_gated_ffn_backward(*b, P.KQ_ACT_SILU) for b in blocks]
    outs = [torch.empty_strided(w.shape, w.stride(), dtype=w.dtype, device="cuda") for w in want[0]]
    H = torch.empty((70, 328), dtype=torch.bfloat16, device="cuda")
    for _ in range(4):
        got = []
        for X, Wg, Wu, dH in blocks:
            P.kq_gated_ffn_backward(X, Wg, Wu, dH, P.KQ_ACT_SILU, *outs[:2], H=H, dX=outs[2], dW_gate=outs[3], dW_up=outs[4])
            got.append([o.clone() for o in outs])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
