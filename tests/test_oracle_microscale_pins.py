"""Pins of the microscale and gated-block oracle: hand-worked blocks, brute
force over the code tables, gradients against central differences."""
import numpy as np
import pytest

import oracle as O


def test_e2m1_rounding_ties_go_to_the_even_code():
    # a block whose amax is 6 has MX scale 2^0: the codes are the rounded values themselves
    x = np.zeros((1, 32))
    x[0, :16] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, -0.25, -0.75, 0.26, 2.49, -5.0, -5.5, 0.2]
    codes, byte = O.fp4_quantize(x, "mx")
    assert byte[0, 0] == 127
    want = [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 0.0, -1.0, 0.5, 2.0, -4.0, -6.0, 0.0]
    assert np.array_equal(O.fp4_dequantize(codes, byte, "mx")[0, :16], want)


def test_mx_scale_exponents():
    for amax, k in ((1.0, -2), (3.999, -1), (4.0, 0), (7.9, 0), (2.0 ** -130, -127), (0.0, -127), (2.0 ** 127, 125)):
        x = np.zeros((1, 32))
        x[0, 3] = -amax
        _, byte = O.fp4_quantize(x, "mx")
        assert int(byte[0, 0]) - 127 == k, amax
    # 7.9 is above the largest code: saturates at 6
    x[0, 3] = 7.9
    codes, byte = O.fp4_quantize(x, "mx")
    assert O.fp4_dequantize(codes, byte, "mx")[0, 3] == 6.0


def test_e4m3_table_and_scale():
    t = O.e4m3_table()
    assert len(t) == 127 and t[-1] == 448.0 and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and np.all(np.diff(t) > 0)
    x = np.zeros((1, 16))
    x[0, 0] = 6.0 * 448.0 * 10            # above what s can hold at g = 1: s = 448, code 6
    codes, byte = O.fp4_quantize(x, "nv", 1.0)
    assert byte[0, 0] == 126 and O.fp4_dequantize(codes, byte, "nv", 1.0)[0, 0] == 2688.0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_codes_are_the_nearest(fmt):
    rng = np.random.default_rng(3)
    M = rng.standard_normal((7, 50)).astype(np.float32).astype(np.float64)
    g = None if fmt == "mx" else np.float64(np.float32(np.abs(M).max() / 2688))
    codes, byte = O.fp4_quantize(M, fmt, g)
    W = O.fp4_dequantize(codes, byte, fmt, g)
    bs = 32 if fmt == "mx" else 16
    s = np.repeat(O.fp4_dequantize(np.full((7, byte.shape[1] * bs), 2, np.uint8), byte, fmt, g)[:, ::bs], bs, axis=1)[:, :50]
    grid = np.concatenate([O.E2M1, -O.E2M1])
    best = np.min(np.abs(M[..., None] - s[..., None] * grid), axis=-1)
    assert np.all(np.abs(M - W) <= best + 1e-7 * s)


def test_packing_and_tiling_by_hand():
    codes = np.arange(35, dtype=np.uint8).reshape(1, 35) % 16
    p = O.fp4_pack(codes)
    assert p.shape == (1, 32) and p[0, 0] == 0x10 and p[0, 17] == (34 % 16) and p[0, 18] == 0
    byte = np.arange(200 * 5, dtype=np.int64).reshape(200, 5) % 251
    t = O.fp4_tile_scales(byte.astype(np.uint8)).reshape(2, 2, 32, 4, 4)
    for r, b in ((0, 0), (33, 2), (127, 4), (128, 3), (199, 4)):
        assert t[r // 128, b // 4, r % 32, r % 128 // 32, b % 4] == byte[r, b]
    assert t[1, 1, 31, 3, 3] == 0


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_gradients_match_differences(act):
    rng = np.random.default_rng(5)
    X, Wg, Wu = rng.standard_normal((4, 6)), rng.standard_normal((5, 6)), rng.standard_normal((5, 6))
    dH = rng.standard_normal((4, 5))
    dG, dU, dX, dWg, dWu = O.gated_ffn_backward(X, Wg, Wu, dH, act)

    def loss(X, Wg, Wu):
        return float((O.gated_ffn(X, Wg, Wu, act) * dH).sum())

    eps = 1e-6
    for k, grad in ((0, dX), (1, dWg), (2, dWu)):
        args = [X, Wg, Wu]
        for idx in np.ndindex(grad.shape):
            d = []
            for s in (eps, -eps):
                a = [v.copy() for v in args]
                a[k][idx] += s
                d.append(loss(*a))
            assert abs((d[0] - d[1]) / (2 * eps) - grad[idx]) < 1e-7
    # dG, dU are the gradients at the projections
    G, U = X @ Wg.T, X @ Wu.T
    e = np.zeros_like(G)
    e[1, 2] = eps
    num = ((O.gate(G + e, act) - O.gate(G - e, act)) * U * dH).sum() / (2 * eps)
    assert abs(num - dG[1, 2]) < 1e-7 and np.allclose(dU, dH * O.gate(G, act))
