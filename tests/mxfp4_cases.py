"""Inputs and bounds shared by the MXFP4 tests."""
import numpy as np

from oracle import mxfp4 as om
from oracle.formats import bf16_bits_to_float, bf16_rne_bits

STEP = 2.0 ** -23  # what one FP32 sum may lose of its terms' magnitudes, cut off rather than rounded


def bf16(x):
    """float64 values rounded to BF16."""
    return bf16_bits_to_float(bf16_rne_bits(x))


def coded(shape, rng, spread):
    """Random codes [..., K/2] of shape [..., K] and scale codes [..., K/32] within `spread` of 127."""
    q = rng.integers(0, 256, shape[:-1] + (shape[-1] // 2,), dtype=np.uint8)
    s = (127 + rng.integers(-spread, spread + 1, shape[:-1] + (shape[-1] // 32,))).astype(np.uint8)
    return q, s


def exact_spread(K):
    """Largest spread of the scales at which every partial sum of K products is an FP32 number: products are
    multiples of 2^(-2 - 2 spread) up to 36 * 2^(2 spread), sums at most K of them; 24 bits hold them."""
    return max(0, int((24 - 2 - np.log2(36.0 * K)) // 4))


def sum_bound(S, K):
    """An FP32 sum of K products in K / 128 sums of 128 (eight levels each), joined from eight waves."""
    return (K / 128 + 8 + 8) * STEP * S


def gated_bound(z, halves, S, K):
    """silu' lies in (-0.1, 1.1); the exponential, sum, quotient and product lose a few 2^-23 of z, and
    the exponential the rounding of its argument too."""
    (g, u), (sg, su) = halves, S
    dg, du = sum_bound(sg, K), sum_bound(su, K)
    return 1.1 * dg * (np.abs(u) + du) + np.abs(om.silu(g)) * du + (8 + np.abs(g)) * STEP * np.abs(z)


def check_bf16(got, want, off, what=""):
    """got: BF16 values; within `off` before the rounding, of half a step (2^-8) of the value."""
    bad = ~(np.abs(got - want) <= off + 2.0 ** -8 * (np.abs(want) + off) + 2.0 ** -134)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


def check_mxfp4(q, s, want, off, what=""):
    """Codes and scales of values within `off` of `want` [M, K]: the scale of some such block, and codes
    between those of the ends of the values' ranges."""
    off = np.broadcast_to(off, want.shape)
    blocks = np.abs(want).reshape(len(want), -1, 32)
    room = off.reshape(blocks.shape)
    low = om.scales(np.maximum(blocks - room, 0).reshape(want.shape))
    high = om.scales((blocks + room).reshape(want.shape))
    assert ((low <= s) & (s <= high)).all(), (what, np.argwhere(~((low <= s) & (s <= high)))[:5])
    got = om.dequantize(q, s)
    ends = [om.dequantize(*om.quantize(want + sign * off, s)) for sign in (-1, 1)]
    bad = ~((ends[0] <= got) & (got <= ends[1]))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


def routed(M, G, rng, kind):
    """m_indices: unsorted, in runs, in runs padded to 16 rows, one expert's only, or of nobody."""
    if kind == "one":
        return np.full(M, G - 1, np.int32)
    if kind == "none":
        return np.full(M, -1, np.int32)
    ids = rng.integers(-1, G + 1, M).astype(np.int32)  # -1 and G: padding
    if kind == "runs":
        ids = np.sort(ids)
    if kind == "padded":
        ids = np.sort(rng.integers(0, G, M)).astype(np.int32)
        ids[rng.random(M) < 0.1] = -1
    return ids
