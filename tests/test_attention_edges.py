"""Host tests of the attention operators' definitions at the edges."""
import numpy as np

from oracle import attention as oa


def test_a_start_before_an_earlier_one_counts_as_that_one():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((9, 2, 4)), rng.standard_normal((9, 1, 4)), rng.standard_normal((9, 1, 4))
    for starts, same in (([0, 9, 0, 9], [0, 9]), ([3, 7, 5, 8], [3, 7, 7, 8]), ([-4, 6, 2, 100, 1], [0, 6, 6, 9])):
        for got, want in zip(oa.prompt_attention(q, k, v, starts, 0.5), oa.prompt_attention(q, k, v, same, 0.5)):
            assert np.array_equal(got, want)
    out, _ = oa.prompt_attention(q, k, v, [3, 7, 5, 8], 0.5)
    assert not out[:3].any() and not out[8:].any() and out[3:8].all()
