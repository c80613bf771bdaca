"""Oracle of the attention operators: plain float64 NumPy, one token (or
sequence) at a time.

  rope_kv_append          position rotation and append to a paged cache
  paged_decode_attention  one new token a sequence over its cached tokens
  prompt_attention        causal attention over packed prompts

Inputs are float64 arrays of the values the stored formats hold (for an E4M3
cache the decoded codes; the scale of each KV head is applied here).  The two
attention functions also return, beside the outputs, the same weighted sums
of |v|: rounding the weights p_t to BF16 (unit roundoff 2^-8) moves an output
by at most 2^-8 of that sum, so it is what their tolerances are made of.

Parity unpinned: no source of this repository quotes outputs of these
operators; the tests pin the functions by cases with known results.
"""
from __future__ import annotations

import numpy as np


def rotate(x, cos, sin, interleaved: bool):
    """x [..., D]: the first 2 len(cos) values rotated pair by pair."""
    n = len(cos)
    y = np.array(x, dtype=np.float64)
    first = np.arange(n) * 2 if interleaved else np.arange(n)
    second = first + 1 if interleaved else first + n
    a, b = y[..., first].copy(), y[..., second].copy()
    y[..., first] = a * cos - b * sin
    y[..., second] = b * cos + a * sin
    return y


def rope_kv_append(q, k, v, turns, positions, table, k_cache, v_cache, seq_ids=None,
                   interleaved=False, k_scale=None, v_scale=None):
    """Returns (rotated q, rotated k, k_cache, v_cache, written): the caches
    [pages, heads, page_size, D] as copies with the new values -- before they
    are rounded, divided by the head's scale and clamped to +-448 where scales
    are given -- and the mask of the (page, slot) places that were written."""
    T = len(positions)
    half = turns.shape[1] // 2
    qr, kr = np.zeros(q.shape), np.zeros(k.shape)
    kc, vc = np.array(k_cache, dtype=np.float64), np.array(v_cache, dtype=np.float64)
    pages, _, size, _ = kc.shape
    written = np.zeros((pages, size), bool)

    def stored(x, scale):
        if scale is None:
            return x
        y = x / np.asarray(scale, np.float64)[:, None]
        return np.clip(y, -448.0, 448.0)

    for t in range(T):
        p = int(positions[t])
        b = t if seq_ids is None else int(seq_ids[t])
        if p < 0 or p >= len(turns) or p >= table.shape[1] * size or not 0 <= b < len(table):
            continue
        cos, sin = np.asarray(turns[p, :half], np.float64), np.asarray(turns[p, half:], np.float64)
        qr[t] = rotate(q[t], cos, sin, interleaved)
        kr[t] = rotate(k[t], cos, sin, interleaved)
        page = int(table[b, p // size])
        if not 0 <= page < pages:
            continue
        kc[page, :, p % size] = stored(kr[t], k_scale)
        vc[page, :, p % size] = stored(v[t], v_scale)
        written[page, p % size] = True
    return qr, kr, kc, vc, written


def _attend(q, k, v, scale):
    """q [D], k and v [n, D] -> (output, weighted sum of |v|); zeros for n = 0."""
    if len(k) == 0:
        return np.zeros(v.shape[1]), np.zeros(v.shape[1])
    s = scale * (k @ q)
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ v, p @ np.abs(v)


def paged_decode_attention(q, k_cache, v_cache, table, lengths, scale, k_scale=None, v_scale=None):
    """q [B, Hq, D]; caches [pages, Hkv, page_size, D] -> (out, sums of |v|)."""
    B, hq, d = q.shape
    pages, hk, size, _ = k_cache.shape
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * size)
        at = [(int(table[b, t // size]), t % size) for t in range(n)]
        at = [x for x in at if 0 <= x[0] < pages]
        pg, sl = [x[0] for x in at], [x[1] for x in at]
        for h in range(hk):
            k, v = np.asarray(k_cache[pg, h, sl], np.float64), np.asarray(v_cache[pg, h, sl], np.float64)
            if k_scale is not None:
                k = k * np.asarray(k_scale[h], np.float64)
            if v_scale is not None:
                v = v * np.asarray(v_scale[h], np.float64)
            for i in range(h * (hq // hk), (h + 1) * (hq // hk)):
                out[b, i], mag[b, i] = _attend(np.asarray(q[b, i], np.float64), k, v, scale)
    return out, mag


def prompt_attention(q, k, v, starts, scale):
    """q [T, Hq, D], k and v [T, Hkv, D] -> (out, sums of |v|).  A start that lies
    before an earlier one counts as the largest of those."""
    T, hq, d = q.shape
    hk = k.shape[1]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    starts = np.maximum.accumulate(np.clip(np.asarray(starts, np.int64), 0, T))
    for i in range(len(starts) - 1):
        lo, hi = int(starts[i]), int(starts[i + 1])
        for t in range(lo, hi):
            for h in range(hq):
                kvh = h // (hq // hk)
                out[t, h], mag[t, h] = _attend(np.asarray(q[t, h], np.float64), np.asarray(k[lo:t + 1, kvh], np.float64),
                                               np.asarray(v[lo:t + 1, kvh], np.float64), scale)
    return out, mag
