"""The attention oracle pinned by cases with known results."""
import numpy as np

from oracle import attention as oa


def test_rotation_keeps_lengths_and_turns_by_the_angle():
    x = np.arange(1.0, 9.0)
    c, s = np.cos([0.3, 1.1]), np.sin([0.3, 1.1])
    y = oa.rotate(x, c, s, False)
    for i in (0, 1):  # pairs (i, i + 2)
        z = complex(x[i], x[i + 2]) * complex(c[i], s[i])
        assert np.allclose([y[i], y[i + 2]], [z.real, z.imag])
    y = oa.rotate(x, c, s, True)
    for i in (0, 1):  # pairs (2 i, 2 i + 1)
        z = complex(x[2 * i], x[2 * i + 1]) * complex(c[i], s[i])
        assert np.allclose(y[2 * i:2 * i + 2], [z.real, z.imag])
    assert np.array_equal(y[4:], x[4:])


def test_append_places_tokens_and_leaves_the_rest():
    turns = np.array([[1.0, 0.0]] * 4)  # no rotation
    q, k, v = np.ones((3, 2, 2)), np.full((3, 1, 2), 2.0), np.full((3, 1, 2), 3.0)
    table = np.array([[1, 0], [7, 2]])  # 7: no page
    kc = vc = np.zeros((3, 1, 2, 2))
    qr, kr, k2, v2, written = oa.rope_kv_append(q, k, v, turns, [3, 0, -1], table, kc, vc,
                                                seq_ids=[0, 1, 0])
    assert np.array_equal(qr[:2], q[:2]) and not qr[2].any() and not kr[2].any()
    assert written.sum() == 1 and written[0, 1]  # position 3 of sequence 0: page 0, slot 1
    assert np.array_equal(k2[0, 0, 1], [2, 2]) and k2.sum() == 4 and v2.sum() == 6


def test_equal_scores_average_the_values():
    rng = np.random.default_rng(0)
    v = rng.standard_normal((5, 1, 4))
    out, mag = oa.prompt_attention(np.zeros((5, 2, 4)), rng.standard_normal((5, 1, 4)), v, [0, 2, 5],
                                   0.5)
    for t, lo in ((0, 0), (1, 0), (2, 2), (4, 2)):
        assert np.allclose(out[t, 1], v[lo:t + 1, 0].mean(0))
        assert np.allclose(mag[t, 0], np.abs(v[lo:t + 1, 0]).mean(0))


def test_decode_is_the_last_row_of_the_prompt():
    rng = np.random.default_rng(1)
    n, hk, d, size = 11, 2, 8, 4
    q, k, v = (rng.standard_normal((n, h, d)) for h in (4, hk, hk))
    want, _ = oa.prompt_attention(q, k, v, [0, n], 0.3)
    table = np.array([[2, 0, 1], [1, 1, 1]])
    kc, vc = np.full((3, hk, size, d), np.nan), np.full((3, hk, size, d), np.nan)
    for t in range(n):
        kc[table[0, t // size], :, t % size] = k[t]
        vc[table[0, t // size], :, t % size] = v[t]
    got, _ = oa.paged_decode_attention(q[[n - 1, 0]], kc, vc, table, [n, 0], 0.3)
    assert np.allclose(got[0], want[n - 1]) and not got[1].any()
    half, _ = oa.paged_decode_attention(q[[n - 1]], kc / 2, vc / 4, table[:1], [n], 0.3,
                                        k_scale=[2.0] * hk, v_scale=[4.0] * hk)
    assert np.allclose(half[0], want[n - 1])
