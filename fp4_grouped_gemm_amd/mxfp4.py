"""MXFP4 entry points of the binding: quantisation of activations, dense and
grouped products, the gated feed-forward product, and the norm at a block's
border (C ABI: quantize_mxfp4, mxfp4_gemm, mxfp4_gated_gemm, residual_norm and
their variants in include/fgg.h).

MXFP4 is E2M1 codes two a byte (value 2j in the low nibble of byte j) with one
E8M0 code, a power of two, for each 32 values of a row.  Codes are uint8 (or
float4_e2m1fn_x2) [..., K / 2], scales uint8 (or float8_e8m0fnu) [..., K / 32].

As the attention operators' these functions check, derive sizes and pass
pointers on in the compiled module; nothing is read back to the host, so calls
can be captured in a HIP graph and replayed after their operands' contents
(the routing among them) change.

A call gives the same bits every time.  A row of a product may have other last
bits in another batch, where its sums are added in another order.
"""
from __future__ import annotations

from . import compiled


def quantize_mxfp4(X, *, rows=None, stream=None):
    """BF16 X [M, K] -> (codes uint8 [M, K / 2], scales uint8 [M, K / 32]): the
    A operand of the MXFP4 products, or weights laid out once.

    rows (int32 [R], optional): the MoE row expansion fused in -- output row r
    quantises X[rows[r]], zeros where rows[r] is outside [0, M)."""
    if stream is not None:
        with compiled.on(stream, X):
            return (compiled.C or compiled.load()).quantize_mxfp4(X, rows)
    return (compiled.C or compiled.load()).quantize_mxfp4(X, rows)


def dequantize_mxfp4(Q, S, *, stream=None):
    """The values of codes Q [M, K / 2] and scales S [M, K / 32], BF16 [M, K]."""
    if stream is not None:
        with compiled.on(stream, Q):
            return (compiled.C or compiled.load()).dequantize_mxfp4(Q, S)
    return (compiled.C or compiled.load()).dequantize_mxfp4(Q, S)


def _product(A, B, a_scale, b_scale, m_indices, out, gated, quantize, stream):
    if stream is not None:
        with compiled.on(stream, A):
            return (compiled.C or compiled.load()).mxfp4_product(A, B, a_scale, b_scale, m_indices, out, gated, quantize)
    return (compiled.C or compiled.load()).mxfp4_product(A, B, a_scale, b_scale, m_indices, out, gated, quantize)


def _routed(m_indices):
    if m_indices is None:
        raise ValueError("m_indices must be an int32 tensor of shape (M,)")
    return m_indices


def mxfp4_gemm(A, B, a_scale, b_scale, out=None, *, stream=None):
    """C[M, N] (bfloat16) of the dense MXFP4 product A B^T: A [M, K / 2] and
    B [N, K / 2] codes, a_scale [M, K / 32] and b_scale [N, K / 32]."""
    return _product(A, B, a_scale, b_scale, None, out, False, False, stream)


def grouped_mxfp4_gemm(A, B, a_scale, b_scale, m_indices, out=None, *, stream=None):
    """C[M, N] (bfloat16) of the grouped MXFP4 product: B [G, N, K / 2], b_scale
    [G, N, K / 32]; m_indices int32 [M] gives each row's expert, in any order
    (outside [0, G): padding, zeros in C)."""
    return _product(A, B, a_scale, b_scale, _routed(m_indices), out, False, False, stream)


def mxfp4_gated_gemm(A, B, a_scale, b_scale, out=None, *, quantize=False, stream=None):
    """silu(A Bg^T) * (A Bu^T), the first half of a gated feed-forward block: B
    [2 F, K / 2] holds F gate rows Bg, then F up rows Bu.  Returns bfloat16
    [M, F], or with quantize (codes [M, F / 2], scales [M, F / 32]): the A
    operand of the second product."""
    return _product(A, B, a_scale, b_scale, None, out, True, quantize, stream)


def grouped_mxfp4_gated_gemm(A, B, a_scale, b_scale, m_indices, out=None, *, quantize=False, stream=None):
    """mxfp4_gated_gemm with the rows' experts' weights, B [G, 2 F, K / 2]; rows
    as for grouped_mxfp4_gemm (of padding: zeros)."""
    return _product(A, B, a_scale, b_scale, _routed(m_indices), out, True, quantize, stream)


def residual_norm(x, residual, weight, *, post_weight=None, gate=None, scale=1.0, eps=1e-6, quantize=False,
                  stream=None):
    """The border between two blocks of a layer:

        h = residual + scale * gate * u,  u = x or post_weight * x / rms(x)
        y = weight * h / rms(h),  rms(v) = sqrt(mean(v ** 2) + eps) over a row

    x [T, H]: bfloat16, rows any multiple of 8 values apart; residual likewise, or
    None (0); weight and post_weight bfloat16 [H]; gate bfloat16 [H] or [T, H],
    or None (1).  Returns (y, h): bfloat16 [T, H] both, or with quantize
    ((codes, scales) of y in MXFP4, h)."""
    if stream is not None:
        with compiled.on(stream, x):
            return (compiled.C or compiled.load()).residual_norm(x, residual, weight, post_weight, gate, scale, eps, quantize)
    return (compiled.C or compiled.load()).residual_norm(x, residual, weight, post_weight, gate, scale, eps, quantize)
