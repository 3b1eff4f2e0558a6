"""Float64 oracle of the microscaled 4-bit formats and of the gated
feed-forward block.  TEST INFRASTRUCTURE, NOT PRODUCT CODE (see kronq.py); it
imports nothing from the package.

Formats: blocks of 32 columns under a power-of-two scale (OCP Microscaling
Formats specification, MXFP4: scale exponent floor(log2 amax) - emax, emax = 2
of e2m1), or blocks of 16 under an E4M3 scale times one number g per matrix.
The places where a quotient is rounded to fp32 before a decision are part of
the definition: the scale's amax / fl(6 g), and a code's v / fl(s g).
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["E2M1", "MX_BLOCK", "NV_BLOCK", "e4m3_table", "fp4_blocks", "fp4_quantize", "fp4_dequantize", "fp4_pack",
           "fp4_tile_scales", "gate", "gate_slope", "gated_ffn", "gated_ffn_backward"]

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MX_BLOCK, NV_BLOCK = 32, 16


def _f32(x):
    return np.asarray(x, dtype=np.float64).astype(np.float32).astype(np.float64)


def e4m3_table():
    """The 127 non-negative finite E4M3 values, by byte."""
    out = []
    for b in range(127):
        e, m = b >> 3, b & 7
        out.append(math.ldexp(m / 8, -6) if e == 0 else math.ldexp(1 + m / 8, e - 7))
    return np.array(out)


def _nearest_even(x, table):
    """Index of the table entry nearest to x >= 0, ties to the even index, the last entry above it."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = x - table[lo], table[hi] - x
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(x >= table[-1], len(table) - 1, np.where(up, hi, lo))


def fp4_blocks(cols, fmt):
    return -(-cols // (MX_BLOCK if fmt == "mx" else NV_BLOCK))


def fp4_quantize(M, fmt, g=None):
    """(codes uint8 [rows, cols], scale bytes uint8 [rows, blocks]) of a finite matrix of fp32 values."""
    M = np.asarray(M, dtype=np.float64)
    rows, cols = M.shape
    bs, nb = (MX_BLOCK if fmt == "mx" else NV_BLOCK), fp4_blocks(cols, fmt)
    codes = np.zeros((rows, cols), np.uint8)
    byte = np.zeros((rows, nb), np.uint8)
    e4m3 = e4m3_table()
    for b in range(nb):
        x = M[:, b * bs:(b + 1) * bs]
        amax = np.abs(x).max(axis=1)
        if fmt == "mx":
            k = np.array([math.frexp(a)[1] - 3 if a else -127 for a in amax])
            k = np.clip(k, -127, 127)
            byte[:, b] = k + 127
            d = np.exp2(k.astype(np.float64))
        else:
            t = np.minimum(_f32(amax / _f32(6.0 * float(g))), 448.0)
            byte[:, b] = _nearest_even(t, e4m3)
            d = _f32(e4m3[byte[:, b]] * float(g))
        q = np.where(d[:, None] > 0, _f32(x / np.where(d > 0, d, 1.0)[:, None]), 0.0)
        codes[:, b * bs:(b + 1) * bs] = _nearest_even(np.abs(q), E2M1) | np.where(np.signbit(q), 8, 0)
    return codes, byte


def fp4_dequantize(codes, byte, fmt, g=None):
    """The matrix that codes and scale bytes stand for (g None: 1)."""
    cols = codes.shape[1]
    v = np.concatenate([E2M1, -E2M1])[codes]
    if fmt == "mx":
        s, bs = np.exp2(byte.astype(np.float64) - 127), MX_BLOCK
    else:
        s, bs = e4m3_table()[byte] * (1.0 if g is None else float(g)), NV_BLOCK
    return v * np.repeat(s, bs, axis=1)[:, :cols]


def fp4_pack(codes):
    """Two codes a byte, the even column low, rows padded with zero codes to 32 columns."""
    rows, cols = codes.shape
    p = np.zeros((rows, -(-cols // 32) * 32), np.uint8)
    p[:, :cols] = codes
    return p[:, 0::2] | (p[:, 1::2] << 4)


def fp4_tile_scales(byte):
    """Scale bytes [rows, blocks] in tiles of 128 rows x 4 blocks, zeros in the places of the rest."""
    rows, nb = byte.shape
    kat = -(-nb // 4)
    out = np.zeros(-(-rows // 128) * kat * 512, np.uint8)
    for r in range(rows):
        for b in range(nb):
            out[((r // 128) * kat + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = byte[r, b]
    return out


# ------------------------------------------------------------ gated block

def gate(g, act):
    """silu: g sigmoid(g); gelu: g/2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3)))."""
    g = np.asarray(g, dtype=np.float64)
    if act == "silu":
        return g / (1.0 + np.exp(-g))
    return 0.5 * g * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))


def gate_slope(g, act):
    g = np.asarray(g, dtype=np.float64)
    if act == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return s + g * s * (1.0 - s)
    c = math.sqrt(2.0 / math.pi)
    t = np.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def gated_ffn(X, Wg, Wu, act):
    return gate(X @ Wg.T, act) * (X @ Wu.T)


def gated_ffn_backward(X, Wg, Wu, dH, act):
    """dG, dU, dX, dWg, dWu."""
    G, U = X @ Wg.T, X @ Wu.T
    dU, dG = dH * gate(G, act), dH * U * gate_slope(G, act)
    return dG, dU, dG @ Wg + dU @ Wu, dG.T @ X, dU.T @ X
