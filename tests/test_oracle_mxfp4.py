"""The MXFP4 oracle on cases with known results."""
import numpy as np
import pytest

from oracle import mxfp4 as om


def test_codes_of_ties_and_their_neighbours():
    down, up = np.nextafter, np.nextafter
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    for t, code in ties.items():
        assert om.e2m1(t) == code
        assert om.e2m1(down(t, 0)) == {0.25: 0, 0.75: 1, 1.25: 2, 1.75: 3, 2.5: 4, 3.5: 5, 5.0: 6}[t]
        assert om.e2m1(up(t, 9)) == om.e2m1(down(t, 0)) + 1
    assert om.e2m1([6, 7.99, 0, 0.5, 1, 1.5, 2, 3, 4]).tolist() == [7, 7, 0, 1, 2, 3, 4, 5, 6]


@pytest.mark.parametrize("top,code", [(4.0, 127), (7.9, 127), (8.0, 128), (3.99, 126), (1.0, 125), (0.0, 0),
                                      (2.0 ** -125, 0), (2.0 ** -124, 1), (2.0 ** -130, 0), (3.3e38, 252),
                                      (np.inf, 255), (np.nan, 255)])
def test_scales(top, code):
    x = np.zeros((1, 64))
    x[0, 40] = -top
    assert om.scales(x).tolist() == [[0, code]]


def test_values_come_back():
    rng = np.random.default_rng(0)
    q = rng.integers(0, 256, (5, 64), dtype=np.uint8)
    q[:, ::16] = (q[:, ::16] & 0xF0) | 7  # a 6 in each block, so that the block's scale is found again
    s = rng.integers(0, 254, (5, 4), dtype=np.uint8)
    x = om.dequantize(q, s)
    q2, s2 = om.quantize(x)
    assert np.array_equal(s, s2)
    same = (q == q2) | (x.reshape(5, 64, 2) == 0).any(-1)
    assert same.all() and np.array_equal(np.signbit(om.dequantize(q2, s2)), np.signbit(x))


def test_products_by_hand():
    A = np.zeros((2, 64), np.uint8)
    B = np.zeros((1, 64), np.uint8)
    A[0, 0], B[0, 0] = 0x72, 0x95  # values 1, 6 and 3, -0.5
    sA, sB = np.full((2, 4), 127, np.uint8), np.full((1, 4), 128, np.uint8)
    C, S = om.gemm(A, B, sA, sB)
    assert C.tolist() == [[2 * (3 - 3.0)], [0.0]] and S.tolist() == [[12.0], [0.0]]
    sA[0, 0] = 255
    assert np.isnan(om.gemm(A, B, sA, sB)[0][0, 0])
    C, _ = om.gemm(A, B[None], np.full((2, 4), 127, np.uint8), sB[None], np.array([-1, 0]))
    assert C.tolist() == [[0.0], [0.0]]


def test_norm_by_hand():
    x, r = np.array([[3.0, 4.0]]), np.array([[1.0, -1.0]])
    y, h = om.norm(x, None, np.ones(2), eps=0.0)
    assert np.allclose(y, x / np.sqrt(12.5)) and np.array_equal(h, x)
    y, h = om.norm(x, r, np.array([2.0, 1.0]), post_weight=np.array([1.0, 0.5]), gate=np.array([1.0, 2.0]), scale=0.5, eps=0.0)
    u = np.array([[3.0, 4.0]]) / np.sqrt(12.5)
    assert np.allclose(h, r + 0.5 * u)
    assert np.allclose(y, np.array([2.0, 1.0]) * h / np.sqrt((h * h).mean()))
