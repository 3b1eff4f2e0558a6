"""The gated feed-forward block in bf16 and its backward pass against the
float64 formulas, stage by stage, and the calibration path that uses them."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import cov_close, need_gpu, np64

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8          # half a step of bf16, relative


@pytest.fixture(scope="module")
def P():
    need_gpu()
    import post_weight_quantization_syrk_b200 as P
    P.load()
    return P


def _act(P, act):
    return P.KQ_ACT_SILU if act == "silu" else P.KQ_ACT_GELU


def _code(info):
    v = int(info.item()) & 0xFFFFFFFF
    return v >> 24, v & 0xFFFFFF


def _mat(rng, rows, cols, scale=1.0, extra=0):
    """bf16 view of rows a multiple of 8 elements apart; NaN between the rows."""
    ld = -(-cols // 8) * 8 + extra
    t = torch.full((rows, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
    t[:, :cols] = torch.from_numpy(scale * rng.standard_normal((rows, cols))).bfloat16()
    return t[:, :cols]


def _block(seed, t, d, f, extra=0):
    rng = np.random.default_rng(seed)
    return (_mat(rng, t, d, 1.0, extra), _mat(rng, f, d, d ** -0.5, extra), _mat(rng, f, d, d ** -0.5, extra),
            _mat(rng, t, f, 1.0, extra))


def _sum_bound(a, b):
    """What an fp32 sum of bf16 products may lose: a unit of 2^-23 of the running
    magnitude for every product added (the tensor core truncates as it aligns)."""
    return (a.shape[1] + 8) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)


def _product_close(got, a, b):
    ref = a @ b.T
    tol = _sum_bound(a, b)
    tol = tol + BF16 * (np.abs(ref) + tol) + 1e-38
    err = np.abs(np64(got) - ref)
    assert np.all(err <= tol), float((err / tol).max())
    assert np.linalg.norm(err) <= BF16 * np.linalg.norm(ref) + 1e-30


def _gate_close(got, ref, slope_tol):
    tol = slope_tol + BF16 * (np.abs(ref) + slope_tol) + 1e-30
    err = np.abs(np64(got) - ref)
    assert np.all(err <= tol), float((err / tol).max())


SIZES = [(1, 1, 1), (1, 64, 8), (3, 100, 65), (8, 1000, 333), (64, 512, 64), (128, 520, 1000), (129, 256, 130),
         (333, 1001, 2730), (2304, 264, 1024), (2050, 1032, 777)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("t,d,f", SIZES)
def test_forward(P, act, t, d, f):
    X, Wg, Wu, _ = _block(t + d, t, d, f, 8 if t % 2 else 0)
    H = torch.full((t + 1, f + 3), 5.0, dtype=torch.bfloat16, device="cuda")
    info = P.new_info(H.device)
    P.kq_gated_ffn(X, Wg, Wu, _act(P, act), H[:t, :f], info=info)
    x, wg, wu = np64(X), np64(Wg), np64(Wu)
    g, u = x @ wg.T, x @ wu.T
    dg, du = _sum_bound(x, wg), _sum_bound(x, wu)
    a = O.gate(g, act)
    # |act'| <= 1.13; the gate's arithmetic is good to a few fp32 ulp, its exponential to 2^-21 (1 + |g|)
    _gate_close(H[:t, :f], a * u, 1.13 * dg * (np.abs(u) + du) + np.abs(a) * du + 2.0 ** -20 * (1 + np.abs(g)) * np.abs(a * u))
    assert _code(info) == (0, 0)
    assert bool((H[t:] == 5.0).all()) and bool((H[:, f:] == 5.0).all())
    assert torch.equal(P.kq_gated_ffn(X, Wg, Wu, _act(P, act)), H[:t, :f])       # aligned rows: the same bits


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("t,d,f", SIZES)
def test_backward(P, act, t, d, f):
    X, Wg, Wu, dH = _block(t + f, t, d, f, 8 if t % 2 else 0)
    info = P.new_info(X.device)
    H = torch.empty((t, f), dtype=torch.bfloat16, device="cuda")
    dG, dU, dX, dWg, dWu = P.kq_gated_ffn_backward(X, Wg, Wu, dH, _act(P, act), H=H, info=info)
    torch.cuda.synchronize()
    assert _code(info) == (0, 0)
    x, wg, wu, dh = np64(X), np64(Wg), np64(Wu), np64(dH)
    g, u = x @ wg.T, x @ wu.T
    eg, eu = _sum_bound(x, wg), _sum_bound(x, wu)
    a, s = O.gate(g, act), O.gate_slope(g, act)
    fast = 2.0 ** -20 * (1 + np.abs(g))
    _gate_close(H, a * u, 1.13 * eg * (np.abs(u) + eu) + np.abs(a) * eu + fast * np.abs(a * u))
    _gate_close(dU, dh * a, np.abs(dh) * (1.13 * eg + fast * np.abs(a)))
    # |act''| <= 1.2 for both; the slope's terms are at most 1 + |g| times their ulp
    _gate_close(dG, dh * u * s, np.abs(dh) * (1.2 * eg * (np.abs(u) + eu) + np.abs(s) * eu + fast * (1 + np.abs(g)) * np.abs(u)))
    # the products, on the bf16 dG and dU that the kernel gave
    gg, gu = np64(dG), np64(dU)
    _product_close(dX, np.concatenate([gg, gu], 1), np.concatenate([wg, wu], 0).T)
    _product_close(dWg, gg.T, x.T)
    _product_close(dWu, gu.T, x.T)
    # the parts alone give the same bits; what is not asked for is not computed
    parts = P.kq_gated_ffn_backward(X, Wg, Wu, dH, _act(P, act), need_dX=False, need_dW=False)
    assert torch.equal(parts[0], dG) and torch.equal(parts[1], dU) and parts[2:] == (None, None, None)
    again = P.kq_gated_ffn_backward(X, Wg, Wu, dH, _act(P, act))
    assert all(torch.equal(p, q) for p, q in zip(again, (dG, dU, dX, dWg, dWu)))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward_matches_differences(P, act):
    """d(sum(H dH)) along random directions against the forward kernel's own
    function in float64 (the formulas), small enough that bf16 rounding is the
    only difference."""
    t, d, f = 40, 48, 72
    X, Wg, Wu, dH = _block(3, t, d, f)
    grads = P.kq_gated_ffn_backward(X, Wg, Wu, dH, _act(P, act))
    x, wg, wu, dh = np64(X), np64(Wg), np64(Wu), np64(dH)
    rng = np.random.default_rng(4)
    for k, grad in ((0, grads[2]), (1, grads[3]), (2, grads[4])):
        args = [x, wg, wu]
        v = rng.standard_normal(args[k].shape)
        eps = 1e-5
        val = []
        for sgn in (eps, -eps):
            b = list(args)
            b[k] = b[k] + sgn * v
            val.append((O.gated_ffn(*b, act) * dh).sum())
        num = (val[0] - val[1]) / (2 * eps)
        # each gradient element carries its own rounding (2^-8) and those of dG and dU in its sum
        gn = np64(grad)
        assert abs(num - (gn * v).sum()) <= 3 * BF16 * np.linalg.norm(gn) * np.linalg.norm(v) / np.sqrt(v.size) * 4


def test_large_gates_saturate(P):
    """Gates far on both sides: act(g) -> g and 0, the slopes 1 and 0, nothing NaN."""
    d, f = 64, 64
    X = torch.zeros((4, d), dtype=torch.bfloat16, device="cuda")
    X[:, 0] = torch.tensor([100.0, -100.0, 1e4, -1e4])
    W = torch.zeros((f, d), dtype=torch.bfloat16, device="cuda")
    W[:, 0] = 1.0
    dH = torch.ones((4, f), dtype=torch.bfloat16, device="cuda")
    for act in ("silu", "gelu"):
        H = P.kq_gated_ffn(X, W, W, _act(P, act))
        want = np.array([1e4, 0.0, 1e8, 0.0])[:, None] * np.ones((1, f))
        assert np.all(np.abs(np64(H) - want) <= BF16 * want + 1e-30)
        dG, dU, dX, dWg, dWu = P.kq_gated_ffn_backward(X, W, W, dH, _act(P, act))
        assert np.all(np.abs(np64(dG) - np.array([100, 0, 1e4, 0])[:, None]) <= BF16 * 1e4 * np.array([0.01, 0, 1, 0])[:, None] + 1e-30)
        assert all(bool(torch.isfinite(v).all()) for v in (dG, dU, dX, dWg, dWu))
    # gates whose square overflows fp32 (an up projection of 0 keeps the product finite)
    X[:, 0] = torch.tensor([1e25, -1e25, 3e38, -3e38])
    Wu = torch.zeros_like(W)
    for act in ("silu", "gelu"):
        assert bool((P.kq_gated_ffn(X, W, Wu, _act(P, act)) == 0).all())
        dG, dU, _, _, _ = P.kq_gated_ffn_backward(X, W, Wu, dH, _act(P, act), need_dX=False, need_dW=False)
        assert bool((dG == 0).all()) and bool(torch.isfinite(dU).all()) and bool((dU[[1, 3]] == 0).all())


def test_nonfinite_tokens_stay_in_their_rows(P):
    X, Wg, Wu, dH = _block(8, 140, 256, 200)
    want = P.kq_gated_ffn(X, Wg, Wu, P.KQ_ACT_SILU)
    X[5, 3], X[131, 7] = float("nan"), float("inf")
    got = P.kq_gated_ffn(X, Wg, Wu, P.KQ_ACT_SILU)
    keep = torch.ones(140, dtype=torch.bool)
    keep[[5, 131]] = False
    assert torch.equal(got[keep], want[keep])
    assert bool(torch.isnan(got[5]).all())


def test_no_tokens(P):
    X, Wg, Wu, dH = _block(8, 4, 64, 72)
    assert P.kq_gated_ffn(X[:0], Wg, Wu, P.KQ_ACT_SILU).shape == (0, 72)
    dW = [torch.full((72, 72), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dG, dU, dX, dWg, dWu = P.kq_gated_ffn_backward(X[:0], Wg, Wu, dH[:0], P.KQ_ACT_SILU, dW_gate=dW[0][:, :64],
                                                   dW_up=dW[1][:, :64])
    assert dG.shape == (0, 72) and dX.shape == (0, 64)
    for w in dW:
        assert bool((w[:, :64] == 0).all()) and bool((w[:, 64:] == 5.0).all())


def test_outputs_in_wider_tensors(P):
    """Every output as a view: what lies beside and behind stays as it was."""
    t, d, f = 200, 96, 136
    X, Wg, Wu, dH = _block(12, t, d, f)
    want = P.kq_gated_ffn_backward(X, Wg, Wu, dH, P.KQ_ACT_GELU)
    outs = [torch.full((r + 1, c + p), 5.0, dtype=torch.bfloat16, device="cuda")
            for r, c, p in ((t, f, 8), (t, f, 8), (t, d, 3), (f, d, 5), (f, d, 5))]
    views = [o[:w.shape[0], :w.shape[1]] for o, w in zip(outs, want)]
    P.kq_gated_ffn_backward(X, Wg, Wu, dH, P.KQ_ACT_GELU, *views[:2], dX=views[2], dW_gate=views[3], dW_up=views[4])
    for o, v, w in zip(outs, views, want):
        assert torch.equal(v, w)
        assert bool((o[w.shape[0]:] == 5.0).all()) and bool((o[:, w.shape[1]:] == 5.0).all())


def test_streams_and_graph(P):
    X, Wg, Wu, dH = _block(20, 150, 264, 320)
    want = (P.kq_gated_ffn(X, Wg, Wu, 0),) + P.kq_gated_ffn_backward(X, Wg, Wu, dH, 0)
    torch.cuda.synchronize()
    got = []
    for st in [torch.cuda.Stream() for _ in range(2)] * 3:
        with torch.cuda.stream(st):
            got.append((P.kq_gated_ffn(X, Wg, Wu, 0),) + P.kq_gated_ffn_backward(X, Wg, Wu, dH, 0))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    info = P.new_info(X.device)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = (P.kq_gated_ffn(X, Wg, Wu, 0, info=info),) + P.kq_gated_ffn_backward(X, Wg, Wu, dH, 0, info=info)
    for _ in range(2):
        for o in out:
            o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.slow
def test_offsets_past_32_bits(P):
    """40000 tokens x 60000 features: H, dG and dU past 2^31 elements; the last rows as on their own."""
    t, d, f, tail = 40000, 64, 60000, 130
    rng = np.random.default_rng(1)
    X, Wg, Wu = _mat(rng, t, d), _mat(rng, f, d, 0.1), _mat(rng, f, d, 0.1)
    dH = torch.ones((t, f), dtype=torch.bfloat16, device="cuda")
    H = P.kq_gated_ffn(X, Wg, Wu, 0)
    assert torch.equal(H[-tail:], P.kq_gated_ffn(X[-tail:], Wg, Wu, 0))
    dG, dU, dX, _, _ = P.kq_gated_ffn_backward(X, Wg, Wu, dH, 0, H=H, need_dW=False)
    want = P.kq_gated_ffn_backward(X[-tail:], Wg, Wu, dH[-tail:], 0, need_dW=False)
    assert torch.equal(dG[-tail:], want[0]) and torch.equal(dU[-tail:], want[1])
    # dX: one chain over K or several
    a, b = dX[-tail:].float(), want[2].float()
    assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-3 * float(b.abs().max())).all())


@pytest.mark.parametrize("t", [40, 2304])
def test_expired_wait_is_reported(P, t):
    X, Wg, Wu, _ = _block(21, t, 2048, 1024)
    want = P.kq_gated_ffn(X, Wg, Wu, 0)
    torch.cuda.synchronize()
    info = P.new_info(X.device)
    old = P.kq_set_wait_limit_ns(0)
    try:
        P.kq_gated_ffn(X, Wg, Wu, 0, info=info)
        torch.cuda.synchronize()
    finally:
        P.kq_set_wait_limit_ns(old)
    assert _code(info)[0] == 8
    assert torch.equal(P.kq_gated_ffn(X, Wg, Wu, 0), want)


def test_refusals(P):
    X, Wg, Wu, dH = _block(22, 16, 64, 72)
    with pytest.raises(P.KronqError):
        P.kq_gated_ffn(X, Wg, Wu, 5)
    with pytest.raises(ValueError):
        P.kq_gated_ffn(X, Wg, Wu[:64], 0)
    with pytest.raises(ValueError):
        P.kq_gated_ffn_backward(X, Wg, Wu, dH[:8], 0)
    with pytest.raises(TypeError):
        P.kq_gated_ffn(X.float(), Wg, Wu, 0)
    odd = torch.zeros((16, 67), dtype=torch.bfloat16, device="cuda")[:, :64]
    with pytest.raises(P.KronqError) as e:
        P.kq_gated_ffn(odd, Wg, Wu, 0)
    assert e.value.status == 3


def test_calibration_of_a_gated_mlp(P):
    """Two token batches through the block's backward pass into the four
    covariances, which then quantize the gate projection."""
    from post_weight_quantization_syrk_b200.pipeline import GatedCalibration, LayerQuantizer
    d, f, n = 256, 512, 700
    X, Wg, Wu, dH = _block(30, n, d, f)
    cal = GatedCalibration(d, f)
    for a, b in ((0, 300), (300, n)):
        dX = cal.add(X[a:b], Wg, Wu, dH[a:b], n)
        assert dX.shape == (b - a, d)
    cal.check()
    x, wg, wu, dh = np64(X), np64(Wg), np64(Wu), np64(dH)
    dG, dU, _, _, _ = O.gated_ffn_backward(x, wg, wu, dh, "silu")
    h = O.gated_ffn(x, wg, wu, "silu")
    for C, A in ((cal.H_X, x), (cal.H_X_down, h), (cal.H_G_gate, dG), (cal.H_G_up, dU)):
        fro, ent = cov_close(np64(C), O.covariance(A))
        # X is exact; H, dG and dU carry their rounding to bf16: 2 * 2^-8 in a product of two at most
        assert fro <= (1e-4 if A is x else 2 * BF16) and ent <= (1e-4 if A is x else 2 * BF16), (fro, ent)
    lq = LayerQuantizer(f, d)
    lq.H_X.copy_(cal.H_X)
    lq.H_G.copy_(cal.H_G_gate)
    lq.Wp.copy_(Wg.float())
    lq.factor()
    res = lq.alloc_results([(4, 0)])
    lq.quantize_all(res)
    lq.loss_all(res)
    lq.check()
    assert np.isfinite(res[0].loss.item()) and res[0].loss.item() > 0
