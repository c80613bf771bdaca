"""residual_norm of rows that are too long for registers: the sum of squares loses no more than its bound where a
row's first values are so large that later squares are less than half of a sum's last place."""
import numpy as np
import pytest

import fp4_grouped_gemm_amd as fgg
from oracle import mxfp4 as om
from tests.gpu_util import c_to_f64, log
from tests.mxfp4_cases import bf16
from tests.test_gpu_norm import dev16

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of FP32


def rms_bound(H):
    """Roundings that 1 / sqrt(sum / H + eps) carries: of the sum of positive terms the H / 2048 that follow each other in a
    lane, 3 + 6 + 3 where the sums of a lane, of a wave's lanes and of the waves are joined, and the quotient's and
    the sum's with eps, all halved by the root; the root's and the reciprocal's."""
    return ((-(-H // 2048) + 3 + 6 + 3 + 2) / 2 + 2) * U


def check(got, want, rel, what):
    """A value within `rel` of `want`, rounded to BF16."""
    a, b = bf16(want * (1 - rel)), bf16(want * (1 + rel))
    bad = (got < np.minimum(a, b)) | (got > np.maximum(a, b))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


@pytest.mark.parametrize("H", [1 << 19, (1 << 20) - 1032, 1 << 20])
def test_large_values_first(H):
    rng = np.random.default_rng(H)
    x = bf16(rng.uniform(0.9375, 1, (2, H)) * rng.choice([-1, 1], (2, H)))
    x[0, 0:2048:8] = 4096  # a lane's first value; the second row's first eight of each
    x[1, :2048] = 4096
    w, p = (bf16(1 + 0.3 * rng.random(H)) for _ in range(2))
    log(f"residual_norm large values first {H}")
    y, h = fgg.residual_norm(dev16(x), None, dev16(w))
    wy, wh = om.norm(x, None, w)
    assert np.array_equal(c_to_f64(h), wh)
    check(c_to_f64(y), wy, rms_bound(H) + 2 * U, "y")
    y, h = fgg.residual_norm(dev16(x), None, dev16(w), post_weight=dev16(p))
    wy, wh = om.norm(x, None, w, p)
    check(c_to_f64(h), wh, rms_bound(H) + 2 * U, "h")
    # the first norm's factor is one for the whole row, so that of y only its values' own two roundings are left
    check(c_to_f64(y), wy, rms_bound(H) + 5 * U, "y of a normed x")
