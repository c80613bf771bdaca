"""GPU parity of the attention operators against the float64 oracle, through
the binding and the C ABI.

Tolerances, per element, from the formulas' roundings (BF16 has 8 bits of
significand: unit roundoff 2^-8):

  attention   the output's rounding, 2^-8 |o|, and the rounding of the weights
              p_t to BF16, which moves o by at most 2^-8 A, A = sum p_t |v_t|
              (the sum they are divided by is not rounded); FP32 scores
              of magnitude below 64 are off by less than 64 * 2^-17 =
              2^-11 after their 128-term sums, which moves the weights, and o by
              2 * 2^-11 A at most
  append      BF16: 2^-8 |x|, and 2^-22 (|a| + |b|) for the FP32 sums of
              the pair; E4M3 (4 bits of significand, spacing 2^-9 below
              2^-6): 2^-4 |y| + 2^-10 of the quotient y, and the FP32 sums' error
              over the scale
"""
import numpy as np
import pytest

import fp4_grouped_gemm_amd as fgg
from oracle import attention as oa
from tests.gpu_util import log

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _bf16(rng, *shape, scale=1.0):
    torch = _torch()
    x = torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * np.float32(scale))
    return x.to(torch.bfloat16).cuda()


def _f64(t):
    return t.detach().cpu().double().numpy()


def _int(x):
    return _torch().tensor(np.asarray(x), dtype=_torch().int32, device="cuda")


def _close(got, want, mag, what):
    err = np.abs(_f64(got) - want)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -10) * mag + 1e-30
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(err / tol)}, first {np.argwhere(bad)[0]}"


# ------------------------------------------------------------------- caches
def _pool(rng, pages, hk, size, d, fp8, layout):
    """(k_cache, v_cache) of random values in one of the layouts."""
    torch = _torch()
    if layout == "heads":  # [pages, heads, tokens, D]
        k, v = (_bf16(rng, pages, hk, size, d) for _ in range(2))
    elif layout == "tokens":  # [pages, tokens, heads, D]
        k, v = (_bf16(rng, pages, size, hk, d) for _ in range(2))
    else:  # K and V side by side in a page
        both = _bf16(rng, pages, 2, hk, size, d)
        k, v = both[:, 0], both[:, 1]
    if fp8:
        if layout == "shared":
            both = (both * 30).to(torch.float8_e4m3fn)
            k, v = both[:, 0], both[:, 1]
        else:
            k, v = (k * 30).to(torch.float8_e4m3fn), (v * 30).to(torch.float8_e4m3fn)
    if layout == "tokens":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    return k, v


def _tables(rng, lens, size, spare=3):
    """A page table that gives every sequence pages of its own in shuffled
    order (unused entries -1), and the number of pages."""
    need = [-(-n // size) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(lens), max(max(need), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


# ------------------------------------------------------------------- decode
def _decode(lens, hq, hk, d, size, fp8=False, layout="heads", seed=0, scale=None, qscale=1.0, check=True):
    torch = _torch()
    rng = np.random.default_rng(seed)
    table, pages = _tables(rng, lens, size)
    k, v = _pool(rng, pages, hk, size, d, fp8, layout)
    q = _bf16(rng, len(lens), hq, d, scale=qscale)
    ks = torch.tensor(rng.uniform(0.02, 0.05, hk), dtype=torch.float32, device="cuda") if fp8 else None
    vs = torch.tensor(rng.uniform(0.02, 0.05, hk), dtype=torch.float32, device="cuda") if fp8 else None
    a = dict(q=q, k_cache=k, v_cache=v, page_table=_int(table), lengths=_int(lens), scale=scale,
             k_scale=ks, v_scale=vs)
    log(f"decode lens={lens[:8]} hq={hq} hk={hk} d={d} page={size} fp8={fp8} {layout}")
    out = fgg.paged_decode_attention(**a)
    if check:
        _check_decode(a, out)
    return a, out


def _check_decode(a, out, what="decode", rows=None):
    rows = slice(None) if rows is None else rows
    s = a["scale"] if a["scale"] is not None else a["q"].shape[2] ** -0.5
    want, mag = oa.paged_decode_attention(
        _f64(a["q"])[rows], _f64(a["k_cache"]), _f64(a["v_cache"]), a["page_table"].cpu().numpy()[rows],
        a["lengths"].cpu().numpy()[rows], s,
        None if a["k_scale"] is None else _f64(a["k_scale"]),
        None if a["v_scale"] is None else _f64(a["v_scale"]))
    _close(out[rows], want, mag, what)


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 0]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1, 2, 16, 64, 256])
def test_decode_lengths_and_pages(d, size, fp8):
    _decode(EDGES, 4, 2, d, size, fp8, seed=size + d)


@pytest.mark.parametrize("hq,hk", [(1, 1), (7, 1), (8, 8), (16, 1), (17, 1), (14, 2), (48, 3), (33, 1)])
def test_decode_head_groups(hq, hk):
    _decode([1, 40, 500], hq, hk, 128, 16, seed=hq)
    _decode([130, 7], hq, hk, 64, 32, True, seed=hq)


@pytest.mark.parametrize("layout", ["heads", "tokens", "shared"])
@pytest.mark.parametrize("fp8", [False, True])
def test_decode_layouts(layout, fp8):
    _decode([200, 3, 64], 8, 4, 128, 16, fp8, layout, seed=5)


@pytest.mark.parametrize("lens", [[9001], [1, 5000, 0, 130, 4097], [700] * 40])
def test_decode_split_rows_are_joined(lens):
    """Few long rows: each is shared by many workgroups."""
    _decode(lens, 4, 2, 128, 64, seed=len(lens))
    _decode(lens, 4, 1, 64, 16, True, seed=len(lens))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_edges_beside_a_long_row(d, fp8):
    """A long sequence in the batch: the lengths' edges where workgroups share
    the rows instead of taking one each."""
    _decode(EDGES + [2600], 6, 2, d, 16, fp8, seed=d)


@pytest.mark.parametrize("tokens", [384, 385, 767, 768, 769, 1536, 1537])
def test_decode_table_widths(tokens):
    """Around the widths up to which a workgroup takes a whole row, for few rows
    and for as many as there are compute units."""
    _decode([tokens, 1, 300], 4, 2, 64, 1, seed=tokens)
    lens = [tokens] + [int(x) for x in np.random.default_rng(tokens).integers(0, 90, 139)]
    a, out = _decode(lens, 2, 2, 64, 1, seed=tokens, check=False)
    _check_decode(a, out, rows=[0, 1, 2, 70, 138, 139])


@pytest.mark.parametrize("tokens", [384, 385, 768, 769])
def test_decode_table_widths_at_half_a_card_of_rows(tokens):
    _decode([tokens, 700, 0] + [31] * 60, 2, 2, 64, 1, seed=tokens)  # 126 rows
    _decode([tokens, 700, 0] + [31] * 61, 2, 2, 64, 1, seed=tokens)  # 128


def test_decode_more_rows_than_slices():
    """Rows of many more sequences than there are workgroups, some of them shared."""
    lens = [int(x) for x in np.random.default_rng(5).integers(0, 300, 420)]
    lens[3], lens[200], lens[419] = 3000, 2000, 2500
    a, out = _decode(lens, 4, 2, 64, 32, seed=6, check=False)
    _check_decode(a, out, rows=[0, 1, 2, 3, 4, 199, 200, 201, 300, 418, 419])
    a, out = _decode(lens, 2, 2, 128, 16, True, seed=7, check=False)
    _check_decode(a, out, rows=[0, 3, 200, 419])


def test_decode_many_sequences():
    """More sequences than a workgroup has threads: several lengths a thread."""
    rng = np.random.default_rng(3)
    a, out = _decode([int(x) for x in rng.integers(0, 200, 700)], 2, 1, 64, 16, seed=4, check=False)
    _check_decode(a, out, rows=[0, 1, 2, 255, 256, 257, 511, 512, 513, 698, 699])


def test_decode_sharp_and_reversed_scores():
    _decode([400, 33], 4, 2, 128, 16, seed=6, qscale=4.0)  # scores up to 64: one weight near 1
    _decode([400, 33], 4, 2, 128, 16, seed=7, scale=-0.1)
    _decode([400, 33], 4, 2, 128, 16, seed=8, scale=0.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_what_is_masked_never_arrives(fp8):
    """NaN in every slot that no sequence owns: past the lengths (inside the
    last page too) and in the spare pages; and pages that are none in the
    middle of a sequence are left out."""
    torch = _torch()
    a, _ = _decode([5, 16, 130, 0, 77, 300], 8, 2, 128, 16, fp8, seed=9, check=False)
    table, lens = a["page_table"].cpu().numpy(), a["lengths"].cpu().numpy()
    own = np.zeros((a["k_cache"].shape[0], 16), bool)
    for b, n in enumerate(lens):
        for t in range(n):
            own[table[b, t // 16], t % 16] = True
    for name in ("k_cache", "v_cache"):
        c = a[name].view(torch.uint8) if fp8 else a[name]
        gone = torch.from_numpy(~own).cuda()[:, None, :, None].expand(c.shape)
        c[gone] = 0x7F if fp8 else float("nan")
    log("decode masked places")
    out = fgg.paged_decode_attention(**a)
    assert torch.isfinite(out).all()

    def clean(x):  # the oracle reads owned places only, whatever the others hold
        return x
    _check_decode({k: clean(v) for k, v in a.items()}, out)
    assert not out[3].any()
    t2 = a["page_table"].clone()
    t2[2, 3], t2[5, 0], t2[4, :] = -1, a["k_cache"].shape[0], 1 << 30
    a["page_table"] = t2
    out = fgg.paged_decode_attention(**a)
    _check_decode(a, out, "decode with missing pages")
    assert not out[4].any()


def test_decode_infinite_values_stay_in_their_row():
    torch = _torch()
    a, base = _decode([50, 60, 70], 4, 2, 64, 16, seed=10)
    page = int(a["page_table"][1, 2])
    a["v_cache"][page, 1, 3, 7] = float("inf")
    out = fgg.paged_decode_attention(**a)
    want = base.clone()
    want[1, 2:, 7] = float("inf")
    assert torch.equal(out, want)


def test_decode_lengths_are_clamped_to_the_table():
    torch = _torch()
    a, _ = _decode([32, 20], 2, 1, 64, 16, seed=11)
    a["page_table"] = torch.where(a["page_table"] < 0, 0, a["page_table"])
    full = fgg.paged_decode_attention(**dict(a, lengths=_int([32, 32])))
    assert torch.equal(fgg.paged_decode_attention(**dict(a, lengths=_int([1 << 30, 33]))), full)
    none = fgg.paged_decode_attention(**dict(a, lengths=_int([-5, -(1 << 31)])))
    assert not none.any()


def test_decode_strided_operands_and_out():
    torch = _torch()
    a, base = _decode([100, 9, 47], 6, 2, 128, 16, seed=12)
    wide = torch.full((3, 8, 136), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = wide[:, 1:7, :128]
    q.copy_(a["q"])
    table = torch.full((3, a["page_table"].shape[1] + 5), 77777, dtype=torch.int32, device="cuda")
    t = table[:, 2:2 + a["page_table"].shape[1]]
    t.copy_(a["page_table"])
    out = torch.full((3, 6, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = fgg.paged_decode_attention(**dict(a, q=q, page_table=t), out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, base)


def test_decode_repeats_bitwise_and_on_another_stream():
    torch = _torch()
    a, base = _decode([5000, 300, 1, 2222], 8, 2, 128, 64, seed=13, check=False)
    for _ in range(3):
        assert torch.equal(fgg.paged_decode_attention(**a), base)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fgg.paged_decode_attention(**a, stream=s)
    s.synchronize()
    assert torch.equal(got, base)


def test_decode_cache_past_32_bit_offsets():
    """Pages 3 GiB apart: byte offsets past 2^32, value offsets past 2^31."""
    torch = _torch()
    rng = np.random.default_rng(14)
    step = 3 << 29  # values of 2 bytes
    pool = torch.empty(2 * step + 2 * 2 * 16 * 64, dtype=torch.bfloat16, device="cuda")
    k = pool.as_strided((3, 2, 16, 64), (step, 16 * 64, 64, 1))
    v = pool.as_strided((3, 2, 16, 64), (step, 16 * 64, 64, 1), 2 * 16 * 64)
    k.copy_(_bf16(rng, 3, 2, 16, 64))
    v.copy_(_bf16(rng, 3, 2, 16, 64))
    a = dict(q=_bf16(rng, 2, 4, 64), k_cache=k, v_cache=v, page_table=_int([[2, 0], [1, 2]]),
             lengths=_int([30, 17]), scale=None, k_scale=None, v_scale=None)
    log("decode past 32-bit offsets")
    _check_decode(a, fgg.paged_decode_attention(**a))
    turns = torch.tensor([[1.0] * 8 + [0.0] * 8] * 32, device="cuda")
    x = _bf16(rng, 1, 2, 64)
    fgg.rope_kv_append(x, x, -x, turns, _int([3]), a["page_table"], k, v, seq_ids=_int([0]))
    assert torch.equal(k[2, :, 3], x[0]) and torch.equal(v[2, :, 3], -x[0])


def test_decode_graph_replays_reread_lengths_and_tables():
    torch = _torch()
    a, _ = _decode([900, 10, 333], 8, 2, 128, 16, seed=15, check=False)
    out = torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fgg.paged_decode_attention(**a, out=out)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    log("decode graph")
    with torch.cuda.graph(g):
        fgg.paged_decode_attention(**a, out=out)
    table = a["page_table"].clone()
    for lens, order in (([900, 10, 333], [0, 1, 2]), ([1, 0, 17], [0, 1, 2]), ([333, 900, 10], [2, 0, 1])):
        a["lengths"].copy_(_int(lens))
        a["page_table"].copy_(table[order])
        torch.cuda.synchronize()
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, fgg.paged_decode_attention(**a))
        torch.cuda.synchronize()
        _check_decode(a, out, f"replay {lens}")


# ------------------------------------------------------------------- append
def _append(T, hq, hk, d, rot, size, fp8=False, layout="heads", interleaved=False, seed=0, positions=None,
            seqs=1, seq_ids=None, width=None, joint=True):
    torch = _torch()
    rng = np.random.default_rng(seed)
    width = width or -(-max(max(positions), 0) // size) + 1
    table, pages = _tables(rng, [width * size] * seqs, size)
    k_cache, v_cache = _pool(rng, pages, hk, size, d, fp8, layout)
    if joint:  # views of a joint projection's rows
        qkv = _bf16(rng, T, hq + 2 * hk, d, scale=3.0)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    else:
        q, k, v = (_bf16(rng, T, h, d, scale=3.0) for h in (hq, hk, hk))
    angle = rng.uniform(-3, 3, (max(max(positions), 0) + 1, rot // 2))
    turns = torch.tensor(np.concatenate([np.cos(angle), np.sin(angle)], 1), dtype=torch.float32, device="cuda")
    ks = torch.tensor(rng.uniform(0.005, 0.05, hk), dtype=torch.float32, device="cuda") if fp8 else None
    vs = torch.tensor(rng.uniform(0.005, 0.05, hk), dtype=torch.float32, device="cuda") if fp8 else None
    return dict(q=q, k=k, v=v, cos_sin=turns, positions=_int(positions), page_table=_int(table),
                k_cache=k_cache, v_cache=v_cache, seq_ids=None if seq_ids is None else _int(seq_ids),
                interleaved=interleaved, k_scale=ks, v_scale=vs)


def _check_append(a, what):
    torch = _torch()
    fp8 = a["k_cache"].dtype != torch.bfloat16
    old = {n: a[n].clone() for n in ("k_cache", "v_cache")}
    log(f"append {what}")
    q2, k2 = fgg.rope_kv_append(**a, return_k=True)
    opt = {n: None if a[n] is None else _f64(a[n]) for n in ("k_scale", "v_scale")}
    qr, kr, kc, vc, written = oa.rope_kv_append(
        _f64(a["q"]), _f64(a["k"]), _f64(a["v"]), _f64(a["cos_sin"]), a["positions"].cpu().numpy(),
        a["page_table"].cpu().numpy(), _f64(old["k_cache"]), _f64(old["v_cache"]),
        None if a["seq_ids"] is None else a["seq_ids"].cpu().numpy(), a["interleaved"], **opt)
    for got, want, src in ((q2, qr, a["q"]), (k2, kr, a["k"])):
        pair = 2 * np.abs(_f64(src)).max(-1, keepdims=True)  # |a| + |b| at most
        err = np.abs(_f64(got) - want)
        assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * pair).all(), f"{what}: {err.max()}"
        assert not got[a["positions"] < 0].any()
    bits = torch.uint8 if fp8 else torch.int16
    for name, want in (("k_cache", kc), ("v_cache", vc)):
        new = _f64(a[name])
        w = np.broadcast_to(written[:, None, :, None], new.shape)
        # (pairs below 40, scales from 0.005)
        rel, tiny = (2.0 ** -4, 2.0 ** -10 + 2.0 ** -22 * 40 / 0.005) if fp8 else (2.0 ** -8, 2.0 ** -22 * 40)
        err = np.abs(new - want)[w]
        assert (err <= rel * np.abs(want)[w] + tiny).all(), f"{what} {name}: {err.max()}"
        same = (a[name].view(bits) == old[name].view(bits)).cpu().numpy()
        assert same[~w].all(), f"{what}: {name} changed outside the new tokens' places"
    return q2


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48)])
def test_append_rotations(d, rot, interleaved, fp8):
    pos = list(range(37))
    a = _append(37, 6, 2, d, rot, 16, fp8, interleaved=interleaved, positions=pos, seq_ids=[0] * 37, seed=rot)
    _check_append(a, f"d={d} rot={rot} interleaved={interleaved} fp8={fp8}")


@pytest.mark.parametrize("layout", ["heads", "tokens", "shared"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("size", [1, 8, 64])
def test_append_layouts_pages_and_padding(layout, fp8, size):
    """Tokens of several sequences in any order, padding between them; a
    position past the table, a sequence that is none."""
    rng = np.random.default_rng(size)
    ids = rng.integers(0, 3, 50)
    places = {b: list(rng.permutation(90)) for b in range(3)}
    pos = [int(places[b].pop()) for b in ids]
    pos[7], pos[49] = -1, -(1 << 31)
    ids[11], ids[12] = 3, -1
    a = _append(50, 5, 1, 64, 32, size, fp8, layout, positions=pos, seqs=3, seq_ids=ids, seed=size)
    width = a["page_table"].shape[1]
    a["positions"][20] = width * size
    a["positions"][21] = (1 << 31) - 1
    a["page_table"][1, 0], a["page_table"][2, 0] = -1, a["k_cache"].shape[0]
    q2 = _check_append(a, f"{layout} fp8={fp8} page={size}")
    assert not q2[[7, 49, 11, 12, 20, 21]].any()


def test_append_one_token_a_sequence_without_ids():
    a = _append(9, 8, 8, 128, 128, 32, positions=[0, 31, 32, 5, 63, 64, -1, 1, 95], seqs=9, seed=2, joint=False)
    q2 = _check_append(a, "decode")
    assert _torch().equal(fgg.rope_kv_append(**a), q2)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_odd_values(fp8):
    """NaN and infinities stay with their pair; E4M3 saturates at 448 scales."""
    torch = _torch()
    a = _append(4, 1, 1, 64, 32, 16, fp8, positions=[0, 1, 2, 3], seqs=1, seq_ids=[0] * 4, seed=3)
    a["k"][1, 0, 2], a["v"][2, 0, 40], a["v"][3, 0, 0] = float("nan"), float("inf"), -3e38
    log("append odd values")
    fgg.rope_kv_append(**a)
    page = int(a["page_table"][0, 0])
    k, v = a["k_cache"][page, 0, :4].float(), a["v_cache"][page, 0, :4].float()
    nan = torch.zeros((4, 64), dtype=torch.bool, device="cuda")
    nan[1, 2] = nan[1, 18] = True
    assert torch.equal(torch.isnan(k), nan)
    if fp8:
        assert v[2, 40] == 448 and v[3, 0] == -448 and not torch.isnan(v).any()
    else:
        assert v[2, 40] == float("inf") and v[3, 0] < -2.9e38


# ------------------------------------------------------------------- prompt
def _prompt(lens, hq, hk, d, seed=0, scale=None, qscale=1.0, before=0, after=0):
    rng = np.random.default_rng(seed)
    T = before + sum(lens) + after
    q, k, v = _bf16(rng, T, hq, d, scale=qscale), _bf16(rng, T, hk, d), _bf16(rng, T, hk, d)
    starts = before + np.concatenate([[0], np.cumsum(lens)])
    a = dict(q=q, k=k, v=v, starts=_int(starts), scale=scale)
    log(f"prompt lens={lens[:8]} hq={hq} hk={hk} d={d}")
    return a, fgg.prompt_attention(**a)


def _check_prompt(a, out, what="prompt"):
    s = a["scale"] if a["scale"] is not None else a["q"].shape[2] ** -0.5
    want, mag = oa.prompt_attention(_f64(a["q"]), _f64(a["k"]), _f64(a["v"]), a["starts"].cpu().numpy(), s)
    _close(out, want, mag, what)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1], [2, 31, 32, 33], [63, 64, 65, 1], [127, 128, 129], [0, 5, 0, 0, 70, 0],
                                  [255, 256, 257], [513]])
def test_prompt_lengths(d, lens):
    a, out = _prompt(lens, 2, 1, d, seed=len(lens))
    _check_prompt(a, out)


@pytest.mark.parametrize("lens,hq,hk,d", [([1100], 32, 8, 64), ([30] * 20, 32, 8, 128), ([200] * 4, 30, 5, 128),
                                          ([97, 0, 33], 32, 32, 64), ([900, 700], 20, 4, 64)])
def test_prompt_long_and_short_of_many_heads(lens, hq, hk, d):
    """Both sides of the choice between whole tiles and halves split over the keys."""
    a, out = _prompt(lens, hq, hk, d, seed=hq)
    _check_prompt(a, out)


@pytest.mark.parametrize("hq,hk", [(1, 1), (7, 1), (6, 3), (16, 2), (3, 3), (40, 8)])
def test_prompt_head_groups(hq, hk):
    for d in (64, 128):
        a, out = _prompt([100, 45], hq, hk, d, seed=hq)
        _check_prompt(a, out)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(16, 4), (24, 4), (14, 2), (16, 16)])
def test_prompt_batches_that_fill_the_card(hq, hk, d):
    """Enough rows for whole tiles, whose waves take four, two or one heads of a
    KV head: every length of the last tile, short and long prompts."""
    lens = [1, 2, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 160, 0, 191, 192, 193, 224, 255, 257, 288, 321,
            480, 1, 640, 17]
    a, out = _prompt(lens, hq, hk, d, seed=hq + d)
    keep = sorted({0, 1, hq // 2, hq - 1})
    want, mag = oa.prompt_attention(_f64(a["q"])[:, keep], _f64(a["k"])[:, [h // (hq // hk) for h in keep]],
                                    _f64(a["v"])[:, [h // (hq // hk) for h in keep]], a["starts"].cpu().numpy(), d ** -0.5)
    _close(out[:, keep], want, mag, f"hq={hq} hk={hk}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(16, 4), (16, 8), (16, 16)])
def test_prompt_later_tokens_never_arrive_in_whole_tiles(hq, hk, d):
    torch = _torch()
    a, base = _prompt([900, 1000, 300], hq, hk, d, seed=8)
    per = hq // hk
    for at in (900, 900 + 33, 900 + 130, 900 + 999):
        v = a["v"].clone()
        v[at, 1, 5], v[at, 1, 6] = float("inf"), float("nan")
        out = fgg.prompt_attention(**dict(a, v=v))
        want = base.clone()
        want[at:1900, per:2 * per, 5], want[at:1900, per:2 * per, 6] = float("inf"), float("nan")
        same = (out == want) | (torch.isnan(out) & torch.isnan(want))
        assert same.all(), f"value at {at}: {(~same).sum()} differ"


def test_prompt_many_short_ones():
    """More prompts than a workgroup has threads."""
    lens = [int(x) for x in np.random.default_rng(0).integers(0, 9, 600)]
    a, out = _prompt(lens, 2, 1, 64, seed=1)
    _check_prompt(a, out)


def test_prompt_tokens_of_no_prompt_are_zero():
    torch = _torch()
    a, out = _prompt([50, 140], 4, 2, 64, seed=2, before=70, after=200)
    _check_prompt(a, out)
    assert not out[:70].any() and not out[260:].any()
    a["starts"] = _int([-3, 120, 120, 1 << 30])  # clamped to [0, T]
    out = fgg.prompt_attention(**a)
    _check_prompt(a, out)
    assert torch.isfinite(out).all()


def test_prompt_sharp_and_reversed_scores():
    for kw in (dict(qscale=4.0), dict(scale=-0.1), dict(scale=0.0)):
        a, out = _prompt([200, 65], 4, 2, 128, seed=3, **kw)
        _check_prompt(a, out, str(kw))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("odd", [float("nan"), float("inf"), float("-inf")])
def test_prompt_later_tokens_never_arrive(d, odd):
    """A key and a value that are not finite reach the queries from their token
    on, in their KV head and prompt, and no other."""
    torch = _torch()
    a, base = _prompt([90, 300, 40], 4, 2, d, seed=4)
    for at in (90, 90 + 129, 90 + 299):
        v = a["v"].clone()
        v[at, 1, 5] = odd
        out = fgg.prompt_attention(**dict(a, v=v))
        want = base.clone()
        want[at:390, 2:, 5] = odd
        same = (out == want) | (torch.isnan(out) & torch.isnan(want))
        assert same.all(), f"value at {at}: {(~same).sum()} differ"
        k = a["k"].clone()
        k[at, 0, 7] = odd
        out = fgg.prompt_attention(**dict(a, k=k))
        keep = torch.ones(out.shape, dtype=torch.bool, device="cuda")
        keep[at:390, :2] = False
        assert torch.equal(out[keep], base[keep])


def test_prompt_strided_operands_and_stream():
    torch = _torch()
    a, base = _prompt([150, 77], 6, 2, 128, seed=5)
    joint = torch.full((227, 12, 136), float("nan"), dtype=torch.bfloat16, device="cuda")
    q, k, v = joint[:, :6, :128], joint[:, 7:9, :128], joint[:, 9:11, 8:]
    for x, n in ((q, "q"), (k, "k"), (v, "v")):
        x.copy_(a[n])
    out = torch.full((227, 6, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fgg.prompt_attention(q, k, v, a["starts"], out=out, stream=s)
    s.synchronize()
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, base)
    # heads first in memory, and one KV head broadcast to two
    qt = a["q"].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(fgg.prompt_attention(qt, a["k"], a["v"], a["starts"]), base)
    one = a["k"][:, :1].expand(-1, 2, -1)
    assert torch.equal(fgg.prompt_attention(a["q"], one, a["v"], a["starts"]),
                       fgg.prompt_attention(a["q"], one.contiguous(), a["v"], a["starts"]))


def test_prompt_graph_replays_reread_starts():
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
    log("prompt graph")
    with torch.cuda.graph(g):
        fgg.prompt_attention(**a, out=out)
    for starts in ([0, 200, 256], [0, 1, 100], [30, 31, 256]):
        a["starts"].copy_(_int(starts))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, fgg.prompt_attention(**a))
        _check_prompt(a, out, f"replay {starts}")


# ------------------------------------------------- the operators with each other
def test_decode_of_the_last_token_is_the_prompts_last_row():
    """A prompt through append and prompt_attention, and its last token again
    through paged_decode_attention on the cache that append filled."""
    torch = _torch()
    n = 333
    a = _append(n, 8, 2, 128, 128, 16, positions=list(range(n)), seq_ids=[0] * n, seed=7)
    q, k = fgg.rope_kv_append(**a, return_k=True)
    whole = fgg.prompt_attention(q, k, a["v"], _int([0, n]))
    last = fgg.paged_decode_attention(q[-1:], a["k_cache"], a["v_cache"], a["page_table"], _int([n]))
    mag = _f64(a["v"].abs().float().mean())
    err = (whole[-1:].float() - last.float()).abs().max().item()
    assert err <= 4 * 2.0 ** -8 * max(float(mag) * 4, whole[-1].abs().max().item())


def test_empty_batches_launch_nothing():
    torch = _torch()
    a, _ = _decode([3, 4], 2, 1, 64, 16, seed=1, check=False)
    none = dict(a, q=a["q"][:0], page_table=a["page_table"][:0], lengths=a["lengths"][:0])
    assert fgg.paged_decode_attention(**none).shape == (0, 2, 64)
    p, _ = _prompt([3], 2, 1, 64)
    z = {n: p[n][:0] for n in ("q", "k", "v")}
    assert fgg.prompt_attention(**z, starts=_int([0, 0])).shape == (0, 2, 64)


def test_refusals_of_the_binding():
    torch = _torch()
    a, _ = _decode([20, 30], 4, 2, 64, 16, seed=1, check=False)
    d = fgg.paged_decode_attention
    for bad, needle in (
            (dict(q=a["q"].float()), "bfloat16"), (dict(q=a["q"][:1]), "q must be"),
            (dict(q=a["q"][:, :3]), "q_heads"), (dict(q=a["q"][:, :, ::2]), "contiguous"),
            (dict(lengths=a["lengths"].long()), "lengths"), (dict(lengths=a["lengths"][:1]), "lengths"),
            (dict(lengths=a["lengths"].cpu()), "GPU"), (dict(page_table=a["page_table"].long()), "page_table"),
            (dict(k_cache=a["k_cache"].half()), "dtype"), (dict(k_cache=a["k_cache"].half(), v_cache=a["v_cache"].half()), "E4M3"),
            (dict(k_cache=a["k_cache"][:, :, :, :32]), "shape"), (dict(k_scale=torch.ones(2, device="cuda")), "E4M3"),
            (dict(k_cache=a["k_cache"].cpu(), v_cache=a["v_cache"].cpu()), "k_cache"),
            (dict(k_cache=a["k_cache"][:, :, :12], v_cache=a["v_cache"][:, :, :12]), "powers of two"),
            (dict(scale=float("nan")), "scale"), (dict(out=torch.empty(2, 4, 64, device="cuda")), "out")):
        with pytest.raises(ValueError, match=needle):
            d(**dict(a, **bad))
    p, _ = _prompt([20], 4, 2, 64)
    for bad, needle in ((dict(starts=p["starts"][:1]), "starts"), (dict(k=p["k"][:19]), "k and v"),
                        (dict(v=p["v"][:, :1]), "k and v"), (dict(q=p["q"][:, :3]), "q_heads"),
                        (dict(q=p["q"][..., :56], k=p["k"][..., :56], v=p["v"][..., :56]), "head_dim")):
        with pytest.raises(ValueError, match=needle):
            fgg.prompt_attention(**dict(p, **bad))
    w = _append(4, 2, 1, 64, 64, 16, positions=[0, 1, 2, 3], seq_ids=[0] * 4)
    for bad, needle in ((dict(seq_ids=None), "seq_ids"), (dict(cos_sin=w["cos_sin"][:, :24].contiguous()), "rot_dim"),
                        (dict(cos_sin=w["cos_sin"].double()), "cos_sin"), (dict(k=w["k"][:3]), "q must be"),
                        (dict(positions=w["positions"][:3]), "positions")):
        with pytest.raises(ValueError, match=needle):
            fgg.rope_kv_append(**dict(w, **bad))
