"""GPU tests of the attention operators where inputs are at the edge of what the
entry points define: bounds in any order, tables and batches of the largest
sizes, strides of dimensions that hold one entry.  Tolerances as in
test_gpu_attention.py."""
import numpy as np
import pytest

import fp4_grouped_gemm_amd as fgg
from tests.gpu_util import log
from tests.test_gpu_attention import _bf16, _check_decode, _check_prompt, _int, _prompt

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


# --------------------------------------------------- prompts: bounds in any order
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(4, 1), (8, 4), (2, 2), (64, 8)])
@pytest.mark.parametrize("starts", [[0, 200, 0, 200], [0, 200, 0, 200, 0, 200, 3], [150, 20, 160, 90, 140, 190],
                                    [-7, 120, 119, 1 << 30, 5], [200, 0], [60, 61, 60, 200, 100]])
def test_prompt_starts_that_decrease(starts, hq, hk, d):
    """Prompts never overlap and every row is written, whatever the bounds hold."""
    torch = _torch()
    rng = np.random.default_rng(len(starts) + d)
    q, k, v = _bf16(rng, 200, hq, d), _bf16(rng, 200, hk, d), _bf16(rng, 200, hk, d)
    out = torch.full_like(q, float("nan"))
    log(f"prompt starts={starts} hq={hq} hk={hk} d={d}")
    fgg.prompt_attention(q, k, v, _int(starts), out=out)
    if hq <= 8:
        _check_prompt(dict(q=q, k=k, v=v, starts=_int(starts), scale=None), out, str(starts))
    sorted_ = np.maximum.accumulate(np.clip(starts, 0, 200))
    assert torch.equal(out, fgg.prompt_attention(q, k, v, _int(sorted_)))


@pytest.mark.parametrize("batch", [61, 62, 63, 64, 200, 700])
@pytest.mark.parametrize("hq,hk", [(8, 2), (4, 2), (2, 2)])
def test_prompt_starts_in_no_order(batch, hq, hk):
    """Of many prompts, on both sides of the number up to which a lane of the
    search holds one of them."""
    torch = _torch()
    rng = np.random.default_rng(batch)
    T = 1000
    q, k, v = _bf16(rng, T, hq, 64), _bf16(rng, T, hk, 64), _bf16(rng, T, hk, 64)
    for which in range(3):
        starts = np.sort(rng.integers(-50, T + 50, batch + 1))
        if which == 1:  # a few out of order
            at = rng.integers(0, batch + 1, 5)
            starts[at] = rng.integers(0, T, 5)
        if which == 2:
            starts = rng.permutation(starts) // 2
        out = torch.full_like(q, float("nan"))
        log(f"prompt {batch} starts in order {which} hq={hq}")
        fgg.prompt_attention(q, k, v, _int(starts), out=out)
        _check_prompt(dict(q=q, k=k, v=v, starts=_int(starts), scale=None), out, f"order {which}")


def test_prompt_replay_with_starts_that_decrease():
    """A captured call whose bounds turn bad, and good again."""
    torch = _torch()
    a, _ = _prompt([200, 56], 4, 2, 128, seed=6)
    out = torch.empty_like(a["q"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fgg.prompt_attention(**a, out=out)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    log("prompt graph, bounds that decrease")
    with torch.cuda.graph(g):
        fgg.prompt_attention(**a, out=out)
    for starts in ([256, 0, 256], [0, 256, 0], [0, 200, 256]):
        a["starts"].copy_(_int(starts))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _check_prompt(a, out, f"replay {starts}")


# ------------------------------------------------------------ decode: largest sizes
@pytest.mark.parametrize("length", [(1 << 31) - 1, (1 << 31) - 64, (1 << 31) - 127, (1 << 31) - 128, (1 << 31) - 200])
def test_decode_table_of_2_31_tokens(length):
    """Lengths up to the end of a table of 2^31 - 64 tokens that has pages only at
    its start, across its middle and at its end."""
    torch = _torch()
    rng = np.random.default_rng(1)
    page, width, d = 64, (1 << 25) - 1, 64
    pages = {0: 3, (1 << 24) - 1: 1, 1 << 24: 0, width - 3: 5, width - 2: 2, width - 1: 4}
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    for col, p in pages.items():
        table[0, col] = p
    k, v = _bf16(rng, 6, 1, page, d), _bf16(rng, 6, 1, page, d)
    q = _bf16(rng, 1, 2, d)
    log(f"decode, a table of 2^31 - 64 tokens, length {length}")
    out = fgg.paged_decode_attention(q, k, v, table, _int([length]))
    # the same tokens under a short table
    n = min(length, page * width)
    tokens = sum(max(0, min(page, n - col * page)) for col in pages)
    short = dict(q=q, k_cache=k, v_cache=v, page_table=_int([list(pages.values())]), lengths=_int([tokens]), scale=None,
                 k_scale=None, v_scale=None)
    _check_decode(short, out)


def test_decode_more_rows_than_one_launch_takes():
    """A million short sequences of eight KV heads: a workgroup of 768 threads for
    each row would pass the 2^32 threads of a launch."""
    torch = _torch()
    batch, heads, d, pages = 1 << 20, 8, 64, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    k, v = (torch.randn((pages, heads, 1, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((batch, heads, d), generator=g, device="cuda", dtype=torch.bfloat16)
    table = torch.randint(0, pages, (batch, 1), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.randint(0, 2, (batch,), generator=g, device="cuda", dtype=torch.int32)
    log("decode, 2^20 sequences x 8 heads")
    out = fgg.paged_decode_attention(q, k, v, table, lens)
    # one token's weight is 1: its value as it is
    want = torch.where(lens[:, None, None] > 0, v[table[:, 0].long(), :, 0], torch.zeros((), dtype=v.dtype, device="cuda"))
    assert torch.equal(out, want)


# ------------------------------------------------------------------------ strides
def test_prompt_heads_first_of_a_long_prompt():
    """Keys and values of 33000 tokens stored head by head: heads lie further apart
    than tokens may."""
    torch = _torch()
    rng = np.random.default_rng(3)
    T, hq, hk, d = 33000, 4, 2, 128
    q, k, v = _bf16(rng, T, hq, d), _bf16(rng, T, hk, d), _bf16(rng, T, hk, d)
    starts = _int([0, 300, 32000, T])
    kt, vt = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (k, v))
    assert kt.stride(1) > 1 << 22
    log("prompt, heads first, 33000 tokens")
    assert torch.equal(fgg.prompt_attention(q, kt, vt, starts), fgg.prompt_attention(q, k, v, starts))


def _loose(x):
    """x with an odd stride in each dimension but the last that holds one entry."""
    return x.as_strided(x.shape, [7 if n == 1 else s for n, s in zip(x.shape[:-1], x.stride()[:-1])] + [1])


def test_strides_of_single_entries_do_not_matter():
    """One token, one head, one page: the stride of such a dimension is never used."""
    torch = _torch()
    rng = np.random.default_rng(4)
    q, k, v = _bf16(rng, 1, 1, 64), _bf16(rng, 1, 1, 64), _bf16(rng, 1, 1, 64)
    log("strides of single entries")
    assert torch.equal(fgg.prompt_attention(_loose(q), _loose(k), _loose(v), _int([0, 1])), v)
    turns = torch.tensor([[1.0] * 8 + [0.0] * 8], device="cuda")
    kc, vc = (torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = _int([[0]])
    got = fgg.rope_kv_append(_loose(q), _loose(k), _loose(v), turns, _int([0]), _loose(table), _loose(kc), _loose(vc))
    assert torch.equal(got, q) and torch.equal(kc[0, :, 0], k[0]) and torch.equal(vc[0, :, 0], v[0])
    assert torch.equal(fgg.paged_decode_attention(_loose(q), _loose(kc), _loose(vc), _loose(table), _int([1])), v)
    # one KV head among many tokens, its dimension moved into place
    k, v, q = _bf16(rng, 50, 64), _bf16(rng, 50, 64), _bf16(rng, 50, 4, 64)
    moved = [x[:, :, None].transpose(1, 2) for x in (k, v)]
    assert moved[0].stride(1) == 1
    assert torch.equal(fgg.prompt_attention(q, *moved, _int([0, 20, 50])),
                       fgg.prompt_attention(q, k.view(50, 1, 64), v.view(50, 1, 64), _int([0, 20, 50])))
