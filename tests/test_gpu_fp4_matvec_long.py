"""kq_fp4_matvec with rows so long that a CTA forms the parts of fp32 vectors in
several pieces of 12 steps of 128 columns (above 8 * 12 * 128 = 12288 columns),
the last piece short, full or of one step."""
import numpy as np
import pytest

import test_gpu_fp4 as F
from gpu_util import need_gpu, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    need_gpu()
    import post_weight_quantization_syrk_b200 as P
    P.load()
    return P


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,k", [(1, 12288), (1, 12289), (8, 13824), (1, 14336), (8, 14336), (3, 16384), (2, 24576), (1, 28672),
                                     (8, 28672), (5, 50001)])
def test_long_rows(P, fmt, dtype, batch, k):
    n = 150                                        # a full block of 128 rows and a ragged one
    W = F._quant(P, F._data(n + k, n, k), fmt)
    X = F._data(batch, batch, k, F.DT[dtype])
    x, w = np64(X), F._values(W, fmt)
    ref = x @ w.T
    # mma.sync: 16 products per step, fp32 chains of 128 columns (three with fp32 vectors, whose
    # parts are exact), then the chains' sums in fp32, at most k / 128 + 8 of them
    tol = (3 * 24 + k / 128 + 8) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    if dtype == "bf16":
        tol = tol + F.BF16 * (np.abs(ref) + tol)
    Y = P.kq_fp4_matvec(W, X)
    err = np.abs(np64(Y) - ref)
    assert np.all(err <= tol), float((err / tol).max())
