"""What the cases of attention_cases.py find: the oracle, computed as the kernels
round, passes; with a mistake planted in it, it does not."""
import numpy as np
import pytest

from oracle import attention as oa
from tests.attention_cases import MOST, beyond, counted, counted_bound, decode_bound, opposed, parts_of, prompt_bound


def _bf16(x):
    """To BF16 and back, to nearest even."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def _sixteen_bits(p):
    hi = (np.asarray(p, np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32).astype(np.float64)
    return hi + _bf16(np.float32(p) * (1 + 2.0 ** -23) - hi)


def _attend(q, k, v, scale, weight, keep=None):
    """One head's output with weights rounded by `weight`, of the tokens `keep`."""
    if keep is not None:
        k, v = k[keep], v[keep]
    s = scale * (k @ q)
    p = np.exp(s - s.max())
    return _bf16((weight(p) @ v) / p.sum())


@pytest.mark.parametrize("n,d", [(5000, 128), (9001, 128), (9001, 64), (33, 64), (1, 64)])
def test_a_lost_or_repeated_token_is_seen(n, d):
    rng = np.random.default_rng(n)
    q, k = np.zeros(d), rng.standard_normal((n, d))
    for t in {0, n - 1, n // 2, 127 % n, 128 % n, int(rng.integers(n))}:
        lost, twice = np.delete(np.arange(n), t), np.append(np.arange(n), t)
        seen = [0, 0]
        for part in range(parts_of(n, d)):
            v = counted(n, d, part)
            assert v.sum(0).max() <= MOST
            want, _ = oa._attend(q, k, v, 1.0)
            bound = counted_bound(want)
            assert beyond(_attend(q, k, v, 1.0, _sixteen_bits), want, bound) == 0
            assert beyond(_attend(q, k, v, 1.0, _bf16), want, bound) == 0
            if n > 1:
                for i, keep in enumerate((lost, twice)):
                    seen[i] += beyond(_attend(q, k, v, 1.0, _sixteen_bits, keep), want, bound)
        assert n == 1 or min(seen) > 0, (t, seen)


@pytest.mark.parametrize("n", [2, 31, 300, 2600, 9001])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_rounded_to_bf16_are_seen(n, d):
    hq, hk = 16, 2
    q, k, v = opposed(n, hq, hk, d)
    assert np.array_equal(_bf16(q), q)
    right = wrong = 0
    for h in range(hq):
        kv = h // (hq // hk)
        want, mag = oa._attend(q[h], k[:, kv], v[:, kv], 1.0)
        size = np.abs(k[:, kv] * q[h]).sum(1).max()
        bound = decode_bound(want, mag, size, n, d)
        right += beyond(_attend(q[h], k[:, kv], v[:, kv], 1.0, _sixteen_bits), want, bound)
        wrong += beyond(_attend(q[h], k[:, kv], v[:, kv], 1.0, _bf16), want, bound)
        assert beyond(_attend(q[h], k[:, kv], v[:, kv], 1.0, _bf16), want, prompt_bound(want, mag, size, n, d)) == 0
    assert right == 0 and wrong >= hq * d // 2


def test_the_bound_holds_what_random_rows_are_off_by():
    rng = np.random.default_rng(0)
    for n, d in ((3, 64), (500, 128), (5000, 128)):
        q, k, v = (_bf16(rng.standard_normal(s)) for s in ((d,), (n, d), (n, d)))
        want, mag = oa._attend(q, k, v, d ** -0.5)
        size = d ** -0.5 * np.abs(k * q).sum(1).max()
        assert beyond(_attend(q, k, v, d ** -0.5, _sixteen_bits), want, decode_bound(want, mag, size, n, d)) == 0
