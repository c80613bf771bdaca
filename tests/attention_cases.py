"""Inputs of the attention operators on which a single wrong token or a weight of
too few bits is visible, and how far results may be off.  Host code (NumPy):
test_attention_cases.py plants mistakes in the oracle and sees that they are
found, test_gpu_attention_cases.py runs the kernels.

counted   all scores equal, so every weight is exactly 1; the values of a token
          are zeros but a one in the dimension of its class.  A result is the share
          of a class among the tokens that are seen: with at most kMost tokens of a
          class that share moves by 1 / kMost or more with each lost or repeated
          one, and is off by its rounding to BF16 alone, 2^-8 of it, and by
          2^-15 where weights are the sum of two BF16 values.

opposed   two kinds of tokens whose weights are 1 and 1 - a few 2^-10, with values
          +x and -x: the result is as small as the weights' difference, of which
          weights rounded to BF16 (2^-8) leave nothing.

decode_bound   |result - oracle| at most, for weights of 16 bits:
  2^-8 |o|     the output's rounding to BF16 (8 bits of significand)
  2^-15 A      A = sum p_t |v_t|: a weight is its upper half, cut, plus what is
               left (below 2^-7 of it) rounded to 8 bits
  2 delta A    delta = (D + 8) 2^-23 S + 2^-22: scores summed in FP32 over D terms
               whose sizes add up to S, scaled and exponentiated; a weight is off
               by its own score's error and by that of what it is divided by
  (n / 8 + 64) 2^-24 A   the sums over n tokens in FP32
"""
import numpy as np

MOST = 32  # tokens of a class


def counted(n, d, part=0, classes=None):
    """Values [n, d] of part `part` of the tokens: an odd number of classes, so that
    tokens a tile or a page apart are of different ones.  Parts: parts_of(n, d)."""
    classes = classes or d - 1
    t = np.arange(n)
    v = np.zeros((n, d))
    mine = t // (MOST * classes) == part
    v[t[mine], t[mine] % classes] = 1.0
    return v


def parts_of(n, d, classes=None):
    return max(1, -(-n // (MOST * (classes or d - 1))))


def counted_bound(want):
    return (2.0 ** -8 + 2.0 ** -15) * np.abs(want) + 2.0 ** -30


def opposed(n, hq, hk, d):
    """q [hq, d], k and v [n, hk, d]; scale 1.  Scores 0 and -w of a head's own w,
    from 0.1 to 3 times 2^-8, values +-1, all of them in BF16 and E4M3."""
    q, k, v = np.zeros((hq, d)), np.zeros((n, hk, d)), np.zeros((n, hk, d))
    w = np.linspace(0.1, 3.0, hq) * 2.0 ** -8
    q[:, 5] = (w.astype(np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32)  # BF16
    k[1::2, :, 5] = -1.0
    v[0::2], v[1::2] = 1.0, -1.0
    v[:, :, 1::2] *= -1.0
    return q, k, v


def decode_bound(want, mag, size, n, d):
    """want, mag (sums of p |v|) [..., D]; size: largest sum of |q k| scale, [...]."""
    delta = (d + 8) * 2.0 ** -23 * np.asarray(size)[..., None] + 2.0 ** -22
    return 2.0 ** -8 * np.abs(want) + mag * (2.0 ** -15 + 2 * delta + (n / 8 + 64) * 2.0 ** -24) + 2.0 ** -30


def prompt_bound(want, mag, size, n, d):
    """The same where weights are rounded to BF16, in the product with V and in the
    sum that divides it alike: each by 2^-8 at most."""
    return decode_bound(want, mag, size, n, d) + 2.0 ** -7 * (1 + 2.0 ** -7) * mag


def beyond(got, want, bound):
    """Elements that are further off than they may be (NaN counts)."""
    return int((~(np.abs(np.asarray(got, np.float64) - want) <= bound)).sum())
