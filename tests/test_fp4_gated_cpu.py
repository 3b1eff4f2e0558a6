"""Host-side refusals of the 4-bit floating-point and gated feed-forward entry
points: every check fails before a CUDA call (the pointers are never read)."""
import ctypes

import pytest
import torch

import post_weight_quantization_syrk_b200 as P
from post_weight_quantization_syrk_b200 import _lib as K

A = 0x10000        # an aligned address that is never dereferenced


def lib():
    return K.load()


def mat(rows=16, cols=64, ld=None, fmt=P.KQ_FP4_MX, codes=A, scales=A, g=None):
    return K.kq_fp4(rows, cols, -(-cols // 32) * 16 if ld is None else ld, fmt, codes, scales, g)


def test_scale_bytes():
    assert P.kq_fp4_scale_bytes(1, 1, P.KQ_FP4_MX) == 512
    assert P.kq_fp4_scale_bytes(129, 129, P.KQ_FP4_MX) == 2 * 2 * 512
    assert P.kq_fp4_scale_bytes(4096, 11008, P.KQ_FP4_NV) == 32 * 172 * 512
    assert P.kq_fp4_scale_bytes(0, 64, P.KQ_FP4_NV) == 0
    assert P.kq_fp4_scale_bytes(4, 0, P.KQ_FP4_MX) == 0
    assert P.kq_fp4_scale_bytes(4, 64, 7) == 0


BAD_MATRICES = [
    (dict(fmt=2), 1), (dict(rows=-1), 1), (dict(cols=0), 1), (dict(codes=None), 1), (dict(scales=None), 1),
    (dict(ld=16), 1), (dict(ld=40), 3), (dict(codes=A + 8), 3), (dict(scales=A + 4), 3), (dict(g=A), 1),
    (dict(rows=(1 << 30) + 1), 2), (dict(cols=(1 << 24) + 1), 2),
]


@pytest.mark.parametrize("kw,status", BAD_MATRICES)
def test_matrix_descriptions_are_refused_everywhere(kw, status):
    bad, ok = mat(**kw), mat()
    L = lib()
    assert L.kq_fp4_quantize(A, P.KQ_BF16, 1 << 25, bad, None, 0, A, None) == status
    assert L.kq_fp4_gemm(bad, ok, A, P.KQ_BF16, 64, A, None) == status
    assert L.kq_fp4_gemm(ok, bad, A, P.KQ_BF16, 64, A, None) == status
    assert L.kq_fp4_matvec(bad, A, P.KQ_BF16, 1 << 25, 1, A, 64, None) == status
    assert L.kq_fp4_gated_ffn(ok, bad, ok, 0, A, 64, A, None) == status
    assert L.kq_fp4_gated_ffn(ok, ok, bad, 0, A, 64, A, None) == status
    assert L.kq_fp4_gemm(None, ok, A, P.KQ_BF16, 64, A, None) == 1


def test_quantize_refusals():
    L = lib()

    def call(M=A, dtype=P.KQ_F32, ldm=64, q=None, hat=None, ldh=0, info=A):
        return L.kq_fp4_quantize(M, dtype, ldm, q or mat(), hat, ldh, info, None)

    assert call(M=None) == 1
    assert call(dtype=2) == 1 and b"dtype" in L.kq_last_error()
    assert call(ldm=63) == 1
    assert call(hat=A, ldh=63) == 1
    assert call(info=None) == 1
    assert call(M=A + 2) == 3
    assert call(M=A + 1, dtype=P.KQ_BF16) == 3
    assert call(hat=A + 2, ldh=64) == 3
    assert call(q=mat(fmt=P.KQ_FP4_NV)) == 1 and b"gscale" in L.kq_last_error()
    assert call(q=mat(rows=0), M=None) == 0          # nothing to do


def test_product_refusals():
    L = lib()
    a = mat()
    assert L.kq_fp4_gemm(a, mat(cols=96), A, P.KQ_F32, 16, A, None) == 1
    assert L.kq_fp4_gemm(a, mat(fmt=P.KQ_FP4_NV), A, P.KQ_F32, 16, A, None) == 1
    assert L.kq_fp4_gemm(a, a, A, 5, 16, A, None) == 1
    assert L.kq_fp4_gemm(a, a, None, P.KQ_F32, 16, A, None) == 1
    assert L.kq_fp4_gemm(a, a, A, P.KQ_F32, 15, A, None) == 1
    assert L.kq_fp4_gemm(a, a, A, P.KQ_F32, 16, None, None) == 1
    assert L.kq_fp4_gemm(a, a, A + 2, P.KQ_F32, 16, A, None) == 3
    assert L.kq_fp4_gemm(mat(cols=(1 << 20) + 1), mat(cols=(1 << 20) + 1), A, P.KQ_F32, 16, A, None) == 2
    w = mat(cols=(1 << 20) + 1)
    assert L.kq_fp4_gated_ffn(w, w, w, 0, A, 16, A, None) == 2
    assert L.kq_fp4_matvec(mat(rows=1 << 30, cols=1 << 24), A, P.KQ_F32, 1 << 24, 1, A, 1 << 30, None) == 2   # scale tiles
    huge = mat(rows=1 << 22)
    assert L.kq_fp4_gemm(huge, huge, A, P.KQ_F32, 1 << 22, A, None) == 2
    assert L.kq_fp4_gemm(mat(rows=0), a, None, P.KQ_F32, 16, A, None) == 0
    assert L.kq_fp4_gemm(a, mat(rows=0), None, P.KQ_F32, 16, A, None) == 0
    for batch, status in ((0, 2), (9, 2)):
        assert L.kq_fp4_matvec(a, A, P.KQ_F32, 64, batch, A, 16, None) == status
    assert L.kq_fp4_matvec(a, A, 3, 64, 1, A, 16, None) == 1
    assert L.kq_fp4_matvec(a, None, P.KQ_F32, 64, 1, A, 16, None) == 1
    assert L.kq_fp4_matvec(a, A, P.KQ_F32, 63, 1, A, 16, None) == 1
    assert L.kq_fp4_matvec(a, A, P.KQ_F32, 64, 1, A, 15, None) == 1
    assert L.kq_fp4_matvec(a, A + 1, P.KQ_BF16, 64, 1, A, 16, None) == 3


def test_fp4_gated_refusals():
    L = lib()
    x, w = mat(), mat(rows=32)
    assert L.kq_fp4_gated_ffn(x, w, mat(rows=33), 0, A, 40, A, None) == 1
    assert L.kq_fp4_gated_ffn(x, w, mat(rows=32, cols=96), 0, A, 40, A, None) == 1
    assert L.kq_fp4_gated_ffn(mat(fmt=P.KQ_FP4_NV), w, w, 0, A, 40, A, None) == 1
    assert L.kq_fp4_gated_ffn(x, w, w, 2, A, 40, A, None) == 1 and b"activation" in L.kq_last_error()
    assert L.kq_fp4_gated_ffn(x, w, w, 0, A, 31, A, None) == 1
    assert L.kq_fp4_gated_ffn(x, w, w, 0, None, 32, A, None) == 1
    assert L.kq_fp4_gated_ffn(x, w, w, 0, A, 32, None, None) == 1
    assert L.kq_fp4_gated_ffn(x, w, w, 0, A + 1, 32, A, None) == 3
    assert L.kq_fp4_gated_ffn(mat(rows=0), w, w, 0, None, 32, A, None) == 0


def gated(X=A, T=16, d=64, ldx=64, wg=A, wu=A, f=32, ldw=64, act=0, H=A, ldh=32, info=A):
    return lib().kq_gated_ffn(X, T, d, ldx, wg, wu, f, ldw, act, H, ldh, info, None)


def backward(X=A, T=16, d=64, ldx=64, wg=A, wu=A, f=32, ldw=64, act=0, dH=A, lddh=32, dG=A, dU=A, ldg=32, H=None,
             ldh=0, dX=None, lddx=0, dWg=None, dWu=None, lddw=0, info=A):
    return lib().kq_gated_ffn_backward(X, T, d, ldx, wg, wu, f, ldw, act, dH, lddh, dG, dU, ldg, H, ldh, dX, lddx, dWg,
                                       dWu, lddw, info, None)


@pytest.mark.parametrize("fn", [gated, backward])
@pytest.mark.parametrize("kw,status", [
    (dict(X=None), 1), (dict(wg=None), 1), (dict(wu=None), 1), (dict(info=None), 1), (dict(T=-1), 1), (dict(d=0), 1),
    (dict(f=0), 1), (dict(ldx=63), 1), (dict(ldw=63), 1), (dict(act=-1), 1), (dict(act=2), 1), (dict(ldx=68), 3),
    (dict(ldw=68), 3), (dict(X=A + 8), 3), (dict(wg=A + 2), 3), (dict(wu=A + 4), 3), (dict(T=(1 << 24) + 1), 2),
    (dict(d=(1 << 17) + 1, ldx=1 << 21, ldw=1 << 21), 2), (dict(f=(1 << 17) + 1, ldh=1 << 21), 2),
    (dict(T=1 << 24, f=1 << 17, ldh=1 << 17), 2)])
def test_gated_refusals(fn, kw, status):
    if fn is backward:
        kw = {k: v for k, v in kw.items() if k != "ldh"}
    assert fn(**kw) == status


def test_gated_output_refusals():
    assert gated(H=None) == 1
    assert gated(ldh=31) == 1
    assert gated(H=A + 1) == 3
    assert gated(T=0, X=None, H=None) == 0
    assert backward(dH=None) == 1
    assert backward(dG=None) == 1
    assert backward(dU=None) == 1
    assert backward(lddh=31) == 1
    assert backward(ldg=31) == 1
    assert backward(ldg=36) == 3
    assert backward(dG=A + 2) == 3
    assert backward(H=A, ldh=31) == 1
    assert backward(dX=A, lddx=63) == 1
    assert backward(dWg=A, dWu=A, lddw=63) == 1
    assert backward(dWg=A, lddw=64) == 1 and b"go together" in lib().kq_last_error()
    assert backward(dX=A + 1, lddx=64) == 3
    assert backward(T=(1 << 18) + 1, dWg=A, dWu=A, lddw=64) == 2 and b"2^18" in lib().kq_last_error()
    assert backward(T=0, X=None, dH=None, dG=None, dU=None) == 0      # no weights' gradients asked: nothing to do


def test_python_wrappers_check_their_tensors():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (lambda: P.kq_fp4_quantize(x, P.KQ_FP4_MX), lambda: P.kq_gated_ffn(x, x, x, P.KQ_ACT_SILU),
                 lambda: P.kq_gated_ffn_backward(x, x, x, x, P.KQ_ACT_SILU)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError):
        P.kq_fp4_quantize(x.half(), P.KQ_FP4_MX)
    with pytest.raises(ValueError, match="current CUDA device"):
        K._device(x)
    with pytest.raises(TypeError, match="CUDA tensor"):
        P.Fp4Matrix(4, 64, P.KQ_FP4_MX, torch.zeros((4, 32), dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8))
    with pytest.raises(ValueError, match="format"):
        P.Fp4Matrix(4, 64, 3, None, None)
