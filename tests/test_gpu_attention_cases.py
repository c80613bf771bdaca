"""The attention operators on inputs on which one wrong token, or weights of too
few bits, are visible (attention_cases.py), in every form in which they are
launched; and batches of more prompts than a lane of the tile search holds one
of, with prompts of many tiles among them."""
import numpy as np
import pytest

import fp4_grouped_gemm_amd as fgg
from oracle import attention as oa
from tests.attention_cases import beyond, counted, counted_bound, decode_bound, opposed, parts_of, prompt_bound
from tests.gpu_util import log
from tests.test_gpu_attention import EDGES, _bf16, _f64, _int, _tables

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _put(x, table, pages, size, fp8, rng):
    """x: [n, heads, d] of each sequence -> a pool with them in their pages, noise
    elsewhere."""
    torch = _torch()
    hk, d = x[0].shape[1:]
    pool = rng.standard_normal((pages, hk, size, d)).astype(np.float32)
    for b, y in enumerate(x):
        t = np.arange(len(y))
        pool[table[b, t // size], :, t % size] = y
    pool = torch.from_numpy(pool).cuda()
    return pool.to(torch.float8_e4m3fn if fp8 else torch.bfloat16)


def _on_gpu(x):
    return _torch().from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(_torch().bfloat16)


# ------------------------------------------------------------------- decode
LENGTHS = {
    "one long": [9001],
    "one of two steps": [600],
    "long and short": [1, 5000, 0, 130, 4097, 31],
    "forty": [700] * 40,
    "edges": EDGES,
    "edges beside a long one": EDGES + [2600],
    "half a card": [700, 385] + [31, 64, 500] * 21,
    "a card": [1500, 1, 769] + [130, 1025, 33, 384] * 34,
    "many": [3000] + [40, 129, 300, 7] * 210,
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", LENGTHS)
def test_decode_counts_every_token_once(which, d, fp8):
    torch = _torch()
    lens = LENGTHS[which]
    hq, hk, size = (18, 1, 64) if which == "long and short" else (4, 2, 16)
    rng = np.random.default_rng(len(lens) + d)
    table, pages = _tables(rng, lens, size)
    k = _put([rng.standard_normal((n, hk, d)) for n in lens], table, pages, size, fp8, rng)
    q = torch.zeros((len(lens), hq, d), dtype=torch.bfloat16, device="cuda")
    scales = {n: torch.full((hk,), 2.0, device="cuda") if fp8 else None for n in ("k_scale", "v_scale")}
    for part in range(max(parts_of(n, d) for n in lens)):
        rows = [counted(n, d, part) for n in lens]
        v = _put([np.repeat(r[:, None], hk, 1) for r in rows], table, pages, size, fp8, rng)
        log(f"decode counted: {which} d={d} fp8={fp8} part {part}")
        got = _f64(fgg.paged_decode_attention(q, k, v, _int(table), _int(lens), **scales))
        for b, r in enumerate(rows):
            want = r.sum(0) / max(len(r), 1) * (2.0 if fp8 else 1.0)
            bad = beyond(got[b], want, counted_bound(want))
            assert bad == 0, f"{which}: sequence {b} of {lens[b]} tokens, part {part}: {bad} off"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[2], [31, 300], [2600], [9001], [700] * 40, [1500, 1400, 3] + [200] * 130])
def test_decode_weights_have_16_bits(lens, d, fp8):
    hq, hk, size = 16, 2, 32
    rng = np.random.default_rng(d)
    table, pages = _tables(rng, lens, size)
    cases = [opposed(n, hq, hk, d) for n in lens]
    k, v = (_put([c[i] for c in cases], table, pages, size, fp8, rng) for i in (1, 2))
    q = _on_gpu(np.stack([c[0] for c in cases]))
    log(f"decode opposed: {lens[:4]} d={d} fp8={fp8}")
    got = _f64(fgg.paged_decode_attention(q, k, v, _int(table), _int(lens), scale=1.0))
    done = {}
    for b, n in enumerate(lens):
        if n not in done:
            qh, kh, vh = cases[b]
            done[n] = [oa._attend(qh[h], kh[:, h // 8], vh[:, h // 8], 1.0) for h in range(hq)]
        for h, (want, mag) in enumerate(done[n]):
            size_ = np.abs(cases[b][1][:, h // 8] * cases[b][0][h]).sum(1).max()
            bad = beyond(got[b, h], want, decode_bound(want, mag, size_, n, d))
            assert bad == 0, f"sequence {b} of {n} tokens, head {h}: {bad} off"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", [[9001, 5000], EDGES, EDGES + [2600], [700] * 5])
def test_decode_random_rows_within_the_bound_of_16_bit_weights(lens, fp8):
    hq, hk, d, size = 4, 2, 128, 64
    rng = np.random.default_rng(7)
    table, pages = _tables(rng, lens, size)
    k, v = (_put([rng.standard_normal((n, hk, d)) for n in lens], table, pages, size, fp8, rng) for _ in range(2))
    q = _bf16(rng, len(lens), hq, d)
    log(f"decode random: {lens[:4]} fp8={fp8}")
    got = _f64(fgg.paged_decode_attention(q, k, v, _int(table), _int(lens)))
    want, mag = oa.paged_decode_attention(_f64(q), _f64(k), _f64(v), table, lens, d ** -0.5)
    kf, qf = np.abs(_f64(k)), np.abs(_f64(q))
    for b, n in enumerate(lens):
        t = np.arange(n)
        for h in range(hq):
            s = d ** -0.5 * (kf[table[b, t // size], h // 2, t % size] @ qf[b, h]).max() if n else 0.0
            bad = beyond(got[b, h], want[b, h], decode_bound(want[b, h], mag[b, h], s, n, d))
            assert bad == 0, f"sequence {b} of {n} tokens, head {h}: {bad} off"


# ------------------------------------------------------------------- prompt
PROMPTS = {
    "one on few heads": ([4001], 8, 1),  # keys split
    "a group of four": ([1500, 700, 33, 0, 64, 1], 32, 8),
    "pairs": ([1500, 127, 128, 129, 700], 16, 8),
    "each on its own": ([1025, 600, 95], 16, 16),
    "groups of seven": ([513, 300, 31], 14, 2),
    "many": ([int(x) for x in np.random.default_rng(1).integers(0, 200, 90)] + [900], 8, 2),
    "many on pairs": ([700] + [5, 65, 0, 33] * 20 + [513, 64, 190], 4, 2),
    "many on their own": ([130, 3, 257] * 30, 2, 2),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", PROMPTS)
def test_prompt_counts_every_token_once(which, d):
    torch = _torch()
    lens, hq, hk = PROMPTS[which]
    rng = np.random.default_rng(d)
    T = sum(lens)
    q = torch.zeros((T, hq, d), dtype=torch.bfloat16, device="cuda")
    k = _bf16(rng, T, hk, d)
    starts = np.concatenate([[0], np.cumsum(lens)])
    for part in range(max(parts_of(n, d) for n in lens)):
        rows = [counted(n, d, part) for n in lens]
        v = _on_gpu(np.repeat(np.concatenate(rows)[:, None], hk, 1))
        log(f"prompt counted: {which} d={d} part {part}")
        got = _f64(fgg.prompt_attention(q, k, v, _int(starts)))
        want = np.concatenate([np.cumsum(r, 0) / np.arange(1, len(r) + 1)[:, None] for r in rows if len(r)])[:, None]
        bad = beyond(got, want, np.broadcast_to(counted_bound(want), got.shape))
        assert bad == 0, f"{which} part {part}: {bad} off"


@pytest.mark.parametrize("hq,hk,d", [(4, 1, 64), (4, 2, 128), (2, 2, 64)])
def test_prompt_many_prompts_of_many_tiles(hq, hk, d):
    """Of more prompts than a lane of the search holds one of, some have several
    tiles, the last one the most."""
    rng = np.random.default_rng(hq)
    lens = [int(x) for x in rng.integers(0, 30, 130)]
    for i in range(0, 130, 9):
        lens[i] = int(rng.integers(60, 200))
    lens[-1] = 777
    T = sum(lens)
    q, k, v = _bf16(rng, T, hq, d), _bf16(rng, T, hk, d), _bf16(rng, T, hk, d)
    starts = np.concatenate([[0], np.cumsum(lens)])
    log(f"prompt: {len(lens)} prompts, {T} tokens, hq={hq} hk={hk} d={d}")
    got = _f64(fgg.prompt_attention(q, k, v, _int(starts)))
    qf, kf, vf = _f64(q), _f64(k), _f64(v)
    want, mag = oa.prompt_attention(qf, kf, vf, starts, d ** -0.5)
    for lo, hi in zip(starts[:-1], starts[1:]):
        for h in range(hq if hi > lo else 0):
            s = d ** -0.5 * np.tril(np.abs(qf[lo:hi, h]) @ np.abs(kf[lo:hi, h // (hq // hk)]).T).max(1)
            bad = beyond(got[lo:hi, h], want[lo:hi, h], prompt_bound(want[lo:hi, h], mag[lo:hi, h], s, hi - lo, d))
            assert bad == 0, f"prompt at {lo} of {hi - lo} tokens, head {h}: {bad} off"
