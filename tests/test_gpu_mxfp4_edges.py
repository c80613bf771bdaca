"""What include/fgg.h says of values at the edges of FP32's range, and of a row's bits in other batches."""
import numpy as np
import pytest

import fp4_grouped_gemm_amd as fgg
from oracle import mxfp4 as om
from oracle.formats import bf16_bits_to_float
from tests.gpu_util import c_bits, c_to_f64, log
from tests.mxfp4_cases import bf16, check_bf16, coded, exact_spread, sum_bound
from tests.test_gpu_mxfp4 import dev

pytestmark = pytest.mark.gpu


def test_values_of_the_largest_scale():
    """Codes 0, 0.5, 1, 1.5 of scale 2^127 are BF16 numbers; 2, 3, 4 and 6 are infinities, of either sign."""
    q = np.tile(np.array([0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE], np.uint8), 8)[None]
    log("dequantize_mxfp4 largest scale")
    x = c_to_f64(fgg.dequantize_mxfp4(dev(q), dev(np.full((1, 4), 254, np.uint8))))
    v = om.VALUES * 2.0 ** 127
    v[4:] = np.inf
    assert np.array_equal(x[0, :8], v) and np.array_equal(x[0, 8:16], -v)


def test_rows_whose_squares_leave_fp32():
    """y of rows of one magnitude, which is one in exact arithmetic.  Sums of 256 squares: of 2^64 and of 2^60 they are 2^136
    and 256 * 2^120 = 2^128, past FP32's largest number, so y is 0; of 2^-60 2^-112, and y is 1; squares of 2^-80 are
    2^-160, below FP32's smallest, 2^-149, so that with eps = 0 y is infinite."""
    import torch
    x = torch.full((4, 256), 1.0, dtype=torch.bfloat16, device="cuda")
    x[0] *= 2.0 ** 64
    x[1] *= 2.0 ** 60
    x[2] *= 2.0 ** -60
    x[3] *= 2.0 ** -80
    log("residual_norm past FP32")
    y, h = fgg.residual_norm(x, None, torch.ones(256, dtype=torch.bfloat16, device="cuda"), eps=0.0)
    assert torch.equal(h, x) and not y[:2].any() and (y[2] == 1).all() and torch.isinf(y[3]).all()


@pytest.mark.parametrize("M", [2, 300])
def test_silu_below_the_exponential(M):
    """A gate of -2^7: its exponential is past FP32, silu is -0 and the result a zero."""
    A, sA = np.full((M, 64), 0x22, np.uint8), np.full((M, 4), 127, np.uint8)  # ones
    B, sB = np.full((64, 64), 0x22, np.uint8), np.full((64, 4), 127, np.uint8)
    B[:16] = 0xAA  # -1: gates of -128, and of 128 in columns 16 to 31
    log(f"gated {M} below the exponential")
    C = c_to_f64(fgg.mxfp4_gated_gemm(dev(A), dev(B), dev(sA), dev(sB)))
    assert not C[:, :16].any() and (C[:, 16:] == 128.0 * 128.0).all()


def test_a_row_alone_and_in_batches():
    """Exact sums have the same bits in every batch; others stay within their bound."""
    rng = np.random.default_rng(4)
    G, N, K = 4, 96, 4096
    B, sB = coded((G, N, K), rng, exact_spread(K))
    A, sA = coded((400, K), rng, exact_spread(K))
    wide = (127 + rng.integers(-20, 21, sA.shape)).astype(np.uint8)
    ids = rng.integers(0, G, 400).astype(np.int32)
    for s in (sA, wide):
        want, S = om.gemm(A, B, s, sB, ids)
        for M in (1, 2, 40, 250, 400):
            log(f"a row in a batch of {M}")
            C = fgg.grouped_mxfp4_gemm(dev(A[-M:]), dev(B), dev(s[-M:]), dev(sB), dev(ids[-M:]))
            if s is sA:
                assert np.array_equal(bf16_bits_to_float(c_bits(C))[-1], bf16(want[-1]))
            else:
                check_bf16(c_to_f64(C)[-1], want[-1], sum_bound(S[-1], K))
