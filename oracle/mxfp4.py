"""Oracle of the MXFP4 operators and of residual_norm: plain float64 NumPy.

TEST INFRASTRUCTURE ONLY (see the package docstring).

  quantize    float values -> E2M1 codes and E8M0 scale codes of blocks of 32
  dequantize  their values
  gemm        sum_k A[i, k] B[g, n, k] with g = m_indices[i], and the sums of
              the products' magnitudes, of which the tolerances are made
  gated       silu(gate) * up of such sums
  norm        h = residual + scale gate u, y = weight h / rms(h)

The format is the OCP microscaling one: code e of a block stands for
2^(e - 127), 255 for NaN; of a block whose largest magnitude lies in
[2^p, 2^(p + 1)) it is max(p - 2, -127) + 127, 2 being the exponent of E2M1's
largest value.  A block with an infinity or NaN gets 255 and codes of zero.

Parity unpinned: no source of this repository quotes outputs of these
operators; the tests pin the functions by cases with known results.
"""
from __future__ import annotations

import numpy as np

from .formats import decode_e2m1, unpack_e2m1

VALUES = decode_e2m1(np.arange(8, dtype=np.uint8))


def e2m1(a) -> np.ndarray:
    """Codes of the magnitudes a (float64): nearest, ties to even, 6 at most."""
    a = np.asarray(a, np.float64)
    middle = (VALUES[1:] + VALUES[:-1]) / 2
    # a tie goes down from an even code, up from an odd one
    code = np.zeros(a.shape, np.uint8)
    for i, m in enumerate(middle):
        code += (a > m) if i % 2 == 0 else (a >= m)
    return code


def scales(x) -> np.ndarray:
    """E8M0 codes of the blocks of x [M, K]."""
    top = np.abs(np.asarray(x, np.float64)).reshape(x.shape[0], -1, 32).max(-1)
    finite = np.where(np.isfinite(top) & (top > 0), top, 1.0)
    p = np.frexp(finite)[1] - 1
    return np.where(np.isfinite(top), np.where(top > 0, np.maximum(p - 2, -127) + 127, 0), 255).astype(np.uint8)


def quantize(x, code=None):
    """x [M, K] -> (packed codes uint8 [M, K/2], scale codes uint8 [M, K/32]);
    with scale codes given, the codes for those."""
    x = np.asarray(x, np.float64)
    s = scales(x) if code is None else code
    nan = s == 255
    step = np.ldexp(1.0, np.where(nan, 127, s).astype(np.int64) - 127)
    b = np.where(nan[..., None], 0.0, x.reshape(*s.shape, 32))
    c = (e2m1(np.abs(b) / step[..., None]) | (np.signbit(b) * 8).astype(np.uint8)).reshape(x.shape)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8), s


def dequantize(q, s) -> np.ndarray:
    """float64 values of codes [..., K/2] and scales [..., K/32]."""
    step = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    v = decode_e2m1(unpack_e2m1(q))
    return (v.reshape(*s.shape, 32) * step[..., None]).reshape(v.shape)


def gemm(A, B, sA, sB, ids=None):
    """(C, magnitudes) float64 [M, N]; B [G, N, K/2] (without ids: [N, K/2])."""
    a = dequantize(A, sA)
    if ids is None:
        B, sB, ids = B[None], sB[None], np.zeros(len(a), np.int64)
    C = np.zeros((len(a), B.shape[1]))
    S = np.zeros_like(C)
    for g in range(len(B)):
        rows = np.nonzero(ids == g)[0]
        if len(rows):
            b = dequantize(B[g], sB[g])
            C[rows] = a[rows] @ b.T
            S[rows] = np.abs(a[rows]) @ np.abs(b).T
    return C, S


def silu(x):
    return x / (1 + np.exp(-x))


def gated(A, B, sA, sB, ids=None):
    """(values, sums, magnitudes) of the gated product, each half [M, F]."""
    C, S = gemm(A, B, sA, sB, ids)
    f = C.shape[1] // 2
    with np.errstate(over="ignore"):
        return silu(C[:, :f]) * C[:, f:], (C[:, :f], C[:, f:]), (S[:, :f], S[:, f:])


def rms_normed(x, weight, eps):
    return weight * x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def norm(x, residual, weight, post_weight=None, gate=None, scale=1.0, eps=1e-6):
    """(y, h) float64."""
    u = x if post_weight is None else rms_normed(x, post_weight, eps)
    h = scale * u * (1.0 if gate is None else gate) + (0.0 if residual is None else residual)
    return rms_normed(h, weight, eps), h
