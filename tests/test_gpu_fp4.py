"""Microscaled 4-bit floating point on the GPU against the float64 oracle:
codes and scale bytes bit for bit, products within the bound of their sums."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import need_gpu, np64

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8          # half a step of bf16, relative
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def P():
    need_gpu()
    import post_weight_quantization_syrk_b200 as P
    P.load()
    return P


def _fmt(P, fmt):
    return {"mx": P.KQ_FP4_MX, "nv": P.KQ_FP4_NV}[fmt]


def _code(info):
    v = int(info.item()) & 0xFFFFFFFF
    return v >> 24, v & 0xFFFFFF


def _data(seed, rows, cols, dtype=torch.float32, pad=0):
    """Values over several octaves, a view of rows `pad` elements further apart; NaN between the rows."""
    rng = np.random.default_rng(seed)
    m = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1))) * np.exp(rng.standard_normal(cols))
    t = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    t[:, :cols] = torch.from_numpy(m).to(dtype)
    return t[:, :cols]


def _g(M):
    return (M.float().abs().amax() / 2688.0).reshape(1)


def _quant(P, M, fmt, info=None, g=None):
    if fmt == "nv" and g is None:
        g = _g(M)
    return P.kq_fp4_quantize(M, _fmt(P, fmt), g if fmt == "nv" else None, info=info)


def _values(Q, fmt):
    """The float64 matrix that a quantized matrix stands for, by the oracle from its bytes."""
    c = Q.codes.cpu().numpy()
    codes = np.empty((Q.rows, 2 * c.shape[1]), np.uint8)
    codes[:, 0::2], codes[:, 1::2] = c & 15, c >> 4
    nb = O.fp4_blocks(Q.cols, fmt)
    t = Q.scales.cpu().numpy().reshape(-1, -(-nb // 4), 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(-1, -(-nb // 4) * 4)
    return O.fp4_dequantize(codes[:, :Q.cols], t[:Q.rows, :nb], fmt, None if fmt == "mx" else Q.gscale.item())


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 4096, 0), (3, 31, 1), (129, 257, 0), (64, 512, 8), (200, 1000, 3)])
def test_quantize_bit_for_bit(P, fmt, dtype, rows, cols, pad):
    M = _data(rows + cols, rows, cols, DT[dtype], pad)
    g = _g(M) if fmt == "nv" else None
    info = P.new_info(M.device)
    hat = torch.full((rows, cols + 4), 7.0, device="cuda")[:, :cols]
    # every byte written, padding included: start from garbage
    out = P.Fp4Matrix(rows, cols, _fmt(P, fmt), torch.full((rows, -(-cols // 32) * 16 + 16), 0xAA, dtype=torch.uint8, device="cuda"),
                      torch.full((P.kq_fp4_scale_bytes(rows, cols, _fmt(P, fmt)),), 0xAA, dtype=torch.uint8, device="cuda"), g)
    P.kq_fp4_quantize(M, _fmt(P, fmt), g, M_hat=hat, out=out, info=info)
    torch.cuda.synchronize()
    assert _code(info) == (0, 0)
    codes, byte = O.fp4_quantize(np64(M), fmt, None if g is None else g.item())
    got = out.codes.cpu().numpy()
    packed = O.fp4_pack(codes)
    assert np.array_equal(got[:, :packed.shape[1]], packed)
    assert np.all(got[:, packed.shape[1]:] == 0xAA)        # beyond the padded row: left as it was
    assert np.array_equal(out.scales.cpu().numpy(), O.fp4_tile_scales(byte))
    want = O.fp4_dequantize(codes, byte, fmt, None if g is None else g.item())
    # the kernel's value is code * fl(s g): one rounding of s g and one of the product
    assert np.all(np.abs(np64(hat) - want) <= 2 * 2.0 ** -24 * np.abs(want))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantize_quotients_at_ties(P, fmt):
    """Values that lie on and next to the ties of their grid: the code goes by
    the fp32 quotient, exactly."""
    rng = np.random.default_rng(11)
    rows, bs = 400, 32 if fmt == "mx" else 16
    M = np.zeros((rows, bs), np.float32)
    g = np.float32(0.7310586)
    for r in range(rows):
        amax = np.float32(np.exp(rng.uniform(-20, 20)))
        M[r, 0] = amax
        _, byte = O.fp4_quantize(M[r:r + 1].astype(np.float64), fmt, g)
        if fmt == "mx":
            d = np.float32(2.0 ** (int(byte[0, 0]) - 127))
        else:
            d = np.float32(O.e4m3_table()[byte[0, 0]] * float(g))
        t = np.float32(rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], bs - 1)) * d
        for i in range(bs - 1):
            for _ in range(rng.integers(0, 3)):
                t[i] = np.nextafter(t[i], np.float32(rng.choice([-1e30, 1e30])))
        M[r, 1:] = np.minimum(t, amax) * rng.choice([-1, 1], bs - 1)
    T = torch.from_numpy(M).cuda()
    Q = P.kq_fp4_quantize(T, _fmt(P, fmt), torch.tensor([g], device="cuda") if fmt == "nv" else None)
    codes, byte = O.fp4_quantize(M.astype(np.float64), fmt, g)
    assert np.array_equal(Q.codes.cpu().numpy(), O.fp4_pack(codes))
    assert np.array_equal(Q.scales.cpu().numpy(), O.fp4_tile_scales(byte))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantize_extremes(P, fmt):
    """Zeros, subnormals, the largest finite values, blocks far apart in size."""
    M = np.zeros((6, 64), np.float32)
    M[1] = np.float32(1e-45)
    M[2, ::3] = np.finfo(np.float32).max
    M[3] = np.linspace(-1, 1, 64)
    M[4, :16], M[4, 16:32], M[4, 32:] = 1e-30, 1e30, -1e-38
    M[5, 0] = np.finfo(np.float32).tiny
    for g in ((None,) if fmt == "mx" else (1.0, 1e-30, 1e30)):
        T = torch.from_numpy(M).cuda()
        info = P.new_info(T.device)
        G = None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda")
        Q = P.kq_fp4_quantize(T, _fmt(P, fmt), G, info=info)
        codes, byte = O.fp4_quantize(M.astype(np.float64), fmt, None if g is None else G.item())
        assert np.array_equal(Q.codes.cpu().numpy(), O.fp4_pack(codes)), g
        assert np.array_equal(Q.scales.cpu().numpy(), O.fp4_tile_scales(byte)), g
        assert _code(info) == (0, 0)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantize_reports_nonfinite_blocks(P, fmt):
    M = _data(5, 8, 128)
    M[3, 40] = float("nan")
    M[6, 100] = float("-inf")
    g = torch.tensor([0.01], device="cuda")
    info = P.new_info(M.device)
    hat = torch.empty((8, 128), device="cuda")
    Q = P.kq_fp4_quantize(M, _fmt(P, fmt), g if fmt == "nv" else None, M_hat=hat, info=info)
    code, row = _code(info)
    assert code == 7 and row in (3, 6)
    bs = 32 if fmt == "mx" else 16
    bad = torch.zeros((8, 128), dtype=torch.bool)
    bad[3, 40 // bs * bs:40 // bs * bs + bs] = True
    bad[6, 100 // bs * bs:100 // bs * bs + bs] = True
    assert torch.equal(torch.isnan(hat).cpu(), bad)
    assert int((Q.scales == (0xFF if fmt == "mx" else 0x7F)).sum()) == 2
    # and the product carries the NaN to those rows only
    Y = P.kq_fp4_gemm(Q, _quant(P, _data(6, 40, 128), fmt), dtype=torch.float32)
    assert torch.equal(torch.isnan(Y).all(1).cpu(), bad.any(1)) and torch.equal(torch.isnan(Y).any(1).cpu(), bad.any(1))


def test_quantize_reports_a_bad_global_scale(P):
    M = _data(5, 4, 64)
    for g in (0.0, -1.0, float("inf"), float("nan")):
        info = P.new_info(M.device)
        Q = P.kq_fp4_quantize(M, P.KQ_FP4_NV, torch.tensor([g], device="cuda"), info=info)
        assert _code(info)[0] == 1
        assert int(Q.codes.sum()) == 0


# ------------------------------------------------------------ products

def _product_bound(A, B):
    """Σ|a||b| per output times what the sums may lose.  The tensor core adds the
    products of an MMA step (64 codes) to the accumulator with at least 24 bits
    kept below the largest term: at most one unit of 2^-23 of the running
    magnitude per product added."""
    return (A.shape[1] + 8) * 2.0 ** -23 * (np.abs(A) @ np.abs(B).T)


def _check(Y, A, B, bf16):
    ref = A @ B.T
    tol = _product_bound(A, B) + 2.0 ** -22 * np.abs(ref)      # the global scales' product and its application
    if bf16:
        tol = tol + BF16 * (np.abs(ref) + tol)
    err = np.abs(np64(Y) - ref)
    assert np.all(err <= tol + 1e-38), float((err / (tol + 1e-38)).max())
    # and in the norm, where the sums' losses average: far below the bound
    assert np.linalg.norm(err) <= (2.0 ** -8 if bf16 else 1e-5) * np.linalg.norm(ref) + 1e-30


SIZES = [(1, 1, 1), (1, 64, 300), (5, 33, 70), (8, 4096, 129), (16, 200, 1000), (128, 520, 64), (129, 512, 200),
         (200, 1000, 333), (256, 256, 256), (1000, 264, 4200), (2100, 1032, 2050)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("m,k,n", SIZES)
def test_gemm(P, fmt, m, k, n):
    A, B = _quant(P, _data(m + k, m, k), fmt), _quant(P, _data(n + k, n, k, torch.bfloat16), fmt)
    a, b = _values(A, fmt), _values(B, fmt)
    for dtype in (torch.bfloat16, torch.float32):
        # a padded, misaligned output: rows behind and beside the result stay as they were
        Y = torch.full((m + 2, n + 3), 5.0, dtype=dtype, device="cuda")
        info = P.new_info(Y.device)
        P.kq_fp4_gemm(A, B, Y[:m, 1:n + 1], info=info)
        _check(Y[:m, 1:n + 1], a, b, dtype == torch.bfloat16)
        assert _code(info) == (0, 0)
        assert bool((Y[m:] == 5.0).all()) and bool((Y[:, 0] == 5.0).all()) and bool((Y[:, n + 1:] == 5.0).all())
        Z = P.kq_fp4_gemm(A, B, dtype=dtype)
        torch.cuda.synchronize()
        assert torch.equal(Z, Y[:m, 1:n + 1])          # aligned rows: the same bits


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_gemm_codes_and_scales_cover_the_formats(P, fmt):
    """All codes and many scale exponents, hand-made: every product is exact in
    fp32, so the sums of few terms are too."""
    rng = np.random.default_rng(2)
    m, k, n = 130, 64, 96
    nb = O.fp4_blocks(k, fmt)

    def mat(rows):
        codes = rng.integers(0, 16, (rows, k)).astype(np.uint8)
        codes[:, rng.permutation(k)[8:]] = 0                     # eight columns in use
        byte = (rng.integers(120, 134, (rows, nb)) if fmt == "mx" else 8 * rng.integers(3, 12, (rows, nb))).astype(np.uint8)
        g = None if fmt == "mx" else torch.ones(1, device="cuda")
        Q = P.Fp4Matrix(rows, k, _fmt(P, fmt), torch.from_numpy(O.fp4_pack(codes)).cuda(),
                        torch.from_numpy(O.fp4_tile_scales(byte)).cuda(), g)
        return Q, O.fp4_dequantize(codes, byte, fmt, 1.0)

    A, a = mat(m)
    B, b = mat(n)
    Y = P.kq_fp4_gemm(A, B, dtype=torch.float32)
    # exponents of one row's terms span under 24 bits: exact up to the accumulator's alignment
    _check(Y, a, b, False)


def test_empty_products(P):
    A0 = P.kq_fp4_quantize(torch.empty((0, 64), device="cuda"), P.KQ_FP4_MX)
    B = _quant(P, _data(1, 32, 64), "mx")
    assert P.kq_fp4_gemm(A0, B).shape == (0, 32)
    assert P.kq_fp4_gemm(B, A0).shape == (32, 0)
    assert P.kq_fp4_gated_ffn(A0, B, B, P.KQ_ACT_SILU).shape == (0, 32)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,k,n,pad", [(1, 1, 1, 0), (1, 128, 16, 0), (2, 33, 17, 1), (3, 1000, 100, 0), (8, 4096, 530, 8), (7, 2050, 40, 0)])
def test_matvec(P, fmt, dtype, batch, k, n, pad):
    W = _quant(P, _data(n + k, n, k), fmt)
    X = _data(batch, batch, k, DT[dtype], pad)
    Y = torch.full((batch + 1, n + 2), 5.0, dtype=DT[dtype], device="cuda")
    P.kq_fp4_matvec(W, X, Y[:batch, :n])
    x, w = np64(X), _values(W, fmt)
    ref = x @ w.T
    # mma.sync: 16 products per step, fp32 chains of 128 columns; fp32 vectors in three bf16 parts (exact)
    tol = (3 * 24 + k / 128 + 8) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    if dtype == "bf16":
        tol = tol + BF16 * (np.abs(ref) + tol)
    assert np.all(np.abs(np64(Y[:batch, :n]) - ref) <= tol)
    assert bool((Y[batch:] == 5.0).all()) and bool((Y[:, n:] == 5.0).all())


def test_matvec_nonfinite_vectors(P):
    """An infinity or NaN in one vector stays in that vector."""
    W = _quant(P, _data(3, 64, 256) + 10.0, "mx")            # no zero codes where it matters
    X = _data(4, 3, 256)
    X[1, 7] = float("inf")
    X[2, 9] = float("nan")
    Y = P.kq_fp4_matvec(W, X)
    ref = np64(X[:1]) @ _values(W, "mx").T
    assert np.allclose(np64(Y[:1]), ref, rtol=1e-4)
    assert bool(torch.isinf(Y[1]).all()) and bool(torch.isnan(Y[2]).all())


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("t,d,f", [(1, 64, 8), (7, 100, 65), (16, 512, 1000), (128, 256, 130), (300, 1000, 260), (2100, 520, 700), (2304, 256, 1030)])
def test_fp4_gated(P, fmt, act, t, d, f):
    rng = np.random.default_rng(t + d)
    X = _quant(P, torch.from_numpy(rng.standard_normal((t, d)).astype(np.float32)).cuda(), fmt)
    Wg = _quant(P, torch.from_numpy((rng.standard_normal((f, d)) / np.sqrt(d)).astype(np.float32)).cuda(), fmt)
    Wu = _quant(P, torch.from_numpy((rng.standard_normal((f, d)) / np.sqrt(d)).astype(np.float32)).cuda(), fmt)
    H = torch.full((t + 1, f + 1), 5.0, dtype=torch.bfloat16, device="cuda")
    info = P.new_info(H.device)
    A = P.KQ_ACT_SILU if act == "silu" else P.KQ_ACT_GELU
    P.kq_fp4_gated_ffn(X, Wg, Wu, A, H[:t, :f], info=info)
    x, wg, wu = _values(X, fmt), _values(Wg, fmt), _values(Wu, fmt)
    g, u = x @ wg.T, x @ wu.T
    dg, du = _product_bound(x, wg), _product_bound(x, wu)
    ref = O.gate(g, act) * u
    # |act'| <= 1.13 for both; the gate's own arithmetic a few fp32 ulp (2^-20 with its exponential)
    tol = 1.13 * dg * (np.abs(u) + du) + np.abs(O.gate(g, act)) * du + 2.0 ** -20 * (1 + np.abs(g)) * np.abs(ref)
    tol = tol + BF16 * (np.abs(ref) + tol) + 1e-30
    assert np.all(np.abs(np64(H[:t, :f]) - ref) <= tol)
    assert _code(info) == (0, 0)
    assert bool((H[t:] == 5.0).all()) and bool((H[:, f:] == 5.0).all())
    assert torch.equal(P.kq_fp4_gated_ffn(X, Wg, Wu, A), H[:t, :f])


# ------------------------------------------------------------ streams, graphs, errors

def test_products_on_side_streams_and_in_graphs(P):
    """Two streams at once and a replayed graph give the bits of the eager call."""
    X, W = _data(1, 40, 512, torch.bfloat16), _quant(P, _data(2, 300, 512), "mx")
    want = P.kq_fp4_gemm(P.kq_fp4_quantize(X, P.KQ_FP4_MX), W)
    v = P.kq_fp4_matvec(W, X[:3])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for st in streams * 4:
        with torch.cuda.stream(st):
            got.append((P.kq_fp4_gemm(P.kq_fp4_quantize(X, P.KQ_FP4_MX), W), P.kq_fp4_matvec(W, X[:3])))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, v) for a, b in got)
    info = P.new_info(X.device)
    Xs = X.clone()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            Y = P.kq_fp4_gemm(P.kq_fp4_quantize(Xs, P.KQ_FP4_MX, info=info), W, info=info)
    for shift in (0, 5):
        Xs.copy_(X.roll(shift, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want.roll(shift, 0))


@pytest.mark.parametrize("m", [40, 2304])
def test_expired_wait_is_reported(P, m):
    """Wait limit 0: the first incomplete wait gives up, the kernel reports it
    and returns; the next call is right again."""
    A, B = _quant(P, _data(1, m, 4096), "mx"), _quant(P, _data(2, 2304, 4096), "mx")
    want = P.kq_fp4_gemm(A, B)
    torch.cuda.synchronize()
    info = P.new_info(want.device)
    old = P.kq_set_wait_limit_ns(0)
    try:
        P.kq_fp4_gemm(A, B, info=info)
        torch.cuda.synchronize()
    finally:
        P.kq_set_wait_limit_ns(old)
    assert _code(info)[0] == 8
    assert torch.equal(P.kq_fp4_gemm(A, B), want)


def test_wrong_shapes_are_refused(P):
    A, B = _quant(P, _data(1, 8, 64), "mx"), _quant(P, _data(2, 8, 96), "mx")
    with pytest.raises(P.KronqError):
        P.kq_fp4_gemm(A, B)
    with pytest.raises(ValueError):
        P.kq_fp4_matvec(A, _data(1, 2, 96))
    with pytest.raises(P.KronqError):
        P.kq_fp4_matvec(A, _data(1, 9, 64))
    with pytest.raises(ValueError):
        P.kq_fp4_gemm(A, A, Y=torch.empty((8, 9), device="cuda"))
    with pytest.raises(P.KronqError):
        P.kq_fp4_quantize(_data(1, 8, 64), P.KQ_FP4_NV)              # no global scale
    with pytest.raises(ValueError):
        P.Fp4Matrix(8, 64, P.KQ_FP4_MX, A.codes, A.scales[:256])


@pytest.mark.slow
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_offsets_past_32_bits(P, fmt):
    """70016 x 65536: codes past 2^31 bytes, M past 2^32: the last rows as on their own."""
    rows, cols, tail = 70016, 65536, 128
    M = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    M[-tail:] = _data(5, tail, cols, torch.bfloat16)
    g = _g(M[-tail:]) if fmt == "nv" else None
    Q = P.kq_fp4_quantize(M, _fmt(P, fmt), g)
    last = P.kq_fp4_quantize(M[-tail:], _fmt(P, fmt), g)
    del M
    assert torch.equal(Q.codes[-tail:], last.codes) and torch.equal(Q.scales[-last.scales.numel():], last.scales)
    assert int(Q.codes[:tail].sum()) == 0
    X = _data(6, 3, cols, torch.bfloat16)
    assert torch.equal(P.kq_fp4_matvec(Q, X)[:, -tail:], P.kq_fp4_matvec(last, X))
    B = _quant(P, _data(7, 64, cols), fmt)
    Y, Z = P.kq_fp4_gemm(Q, B), P.kq_fp4_gemm(last, B)
    # one chain over K or several: within the sums' bound
    tol = 2.0 ** -7 * Z.float().abs() + 2.0 ** -23 * cols * float(Z.float().abs().max()) / 100
    assert bool(((Y[-tail:].float() - Z.float()).abs() <= tol).all()) and int((Y[:-tail] != 0).sum()) == 0


@pytest.mark.slow
def test_long_products_keep_their_sums(P):
    """131072 columns of one sign, where truncation adds up: within its bound."""
    k = 131072
    A = P.kq_fp4_quantize(torch.rand((40, k), device="cuda") + 0.5, P.KQ_FP4_MX)
    B = P.kq_fp4_quantize(torch.rand((200, k), device="cuda") + 0.5, P.KQ_FP4_MX)
    ref = _values(A, "mx") @ _values(B, "mx").T
    Y = np64(P.kq_fp4_gemm(A, B, dtype=torch.float32))
    # k / 64 MMAs, each up to 2^-24 of the sum so far (twice for the alignment of its terms)
    assert np.abs(Y / ref - 1).max() <= 2 * k / 64 * 2.0 ** -24


# ------------------------------------------------------------ together

@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_mlp_served_in_4_bits(P, fmt):
    """The whole block over 4-bit operands, stage by stage on the kernels' own bytes."""
    from post_weight_quantization_syrk_b200.pipeline import Fp4MLP
    rng = np.random.default_rng(9)
    d, f = 264, 700
    Wg, Wu = (torch.from_numpy((rng.standard_normal((f, d)) / 16).astype(np.float32)).cuda() for _ in range(2))
    Wd = torch.from_numpy((rng.standard_normal((d, f)) / 26).astype(np.float32)).cuda()
    mlp = Fp4MLP(Wg, Wu, Wd, _fmt(P, fmt))
    X = torch.from_numpy(rng.standard_normal((150, d)).astype(np.float32)).cuda().bfloat16()
    if fmt == "nv":
        with pytest.raises(RuntimeError):
            mlp(X)
    mlp.calibrate(X)
    for t in (1, 8, 150):
        Y = mlp(X[:t])
        H = mlp._hidden(X[:t], None)
        Hq = P.kq_fp4_quantize(H, _fmt(P, fmt), mlp.g_h)
        _check(Y, _values(Hq, fmt), _values(mlp.down, fmt), True)
        # and near the block in float64
        x = np64(X[:t])
        ref = O.gated_ffn(x, np64(Wg), np64(Wu), "silu") @ np64(Wd).T
        assert np.linalg.norm(np64(Y) - ref) < 0.4 * np.linalg.norm(ref)
    v = mlp.decode("gate", X[:2])
    assert np.allclose(np64(v), np64(X[:2]) @ _values(mlp.gate, fmt).T, atol=0.05)
    mlp.check()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_layer_quantizer_fp4(P, fmt):
    """Rotate, quantize to 4-bit floating point, loss: beside the integer settings of the same layer."""
    import synth
    from gpu_util import device_rht
    from post_weight_quantization_syrk_b200.pipeline import LayerQuantizer
    spec = synth.scaled(synth.WORKLOADS["attn4096"], d_out=256, d_in=384, n_tokens=1000)
    W, X, G, Ti, To = synth.layer(spec, 77)
    lq = LayerQuantizer(spec.d_out, spec.d_in)
    res = lq.run(W.cuda(), X.cuda(), G.cuda(), device_rht(Ti), device_rht(To), [(4, 0)])
    r = lq.quantize_fp4(_fmt(P, fmt))
    lq.check()
    assert np.allclose(np64(r.W_hat), _values(r.matrix, fmt), rtol=2.0 ** -22, atol=0)
    ref = O.kron_loss(np64(lq.Wp), np64(r.W_hat), np64(lq.H_X), np64(lq.H_G))
    assert abs(r.loss.item() - ref) <= 1e-3 * ref
    assert 0 < r.loss.item() and res[0].loss.item() > 0
