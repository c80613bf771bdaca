"""residual_norm on the GPU against the float64 oracle."""
import numpy as np
import pytest

import fp4_grouped_gemm_amd as fgg
from oracle import mxfp4 as om
from oracle.formats import bf16_rne_bits
from tests.gpu_util import c_to_f64, log
from tests.mxfp4_cases import STEP, bf16, check_bf16, check_mxfp4

pytestmark = pytest.mark.gpu


def dev16(x):
    import torch
    bits = np.ascontiguousarray(bf16_rne_bits(x))
    return torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)


def norm_bound(u, residual, weight, y, h, rows=1):
    """What FP32 may lose of y: of h, four roundings of its two terms; of the root mean square, at most log2(H) + H / 2048 + 8
    roundings of a sum of squares, which no sum of positive terms magnifies, halved by the root, and h's own; three more."""
    terms = np.abs(u) + (0 if residual is None else np.abs(residual))
    H = y.shape[1]
    dh = 8 * STEP * terms
    rms = np.sqrt((h * h).mean(-1, keepdims=True))
    drms = np.sqrt((dh * dh).mean(-1, keepdims=True))
    with np.errstate(divide="ignore", invalid="ignore"):
        rel = np.where(rms > 0, drms / rms, 0) + (np.log2(H) + H / 2048 + 16) * STEP
        back = np.where(h != 0, np.abs(y) / np.abs(h), 0)
    return np.abs(y) * rel + back * dh


def case(T, H, post, gate, seed=0, loud=1.0):
    rng = np.random.default_rng(T + H + seed)
    x = bf16(rng.standard_normal((T, H)) * loud)
    r = bf16(rng.standard_normal((T, H)) * 3)
    w = bf16(1 + 0.3 * rng.standard_normal(H))
    p = bf16(1 + 0.3 * rng.standard_normal(H)) if post else None
    g = {"": None, "channel": bf16(rng.random(H)), "token": bf16(rng.random((T, H)))}[gate]
    return x, r, w, p, g


def inner(x, p, g, scale, eps=1e-6):
    u = x if p is None else om.rms_normed(x, p, eps)
    return u * scale * (1.0 if g is None else g)


def up(v):
    return None if v is None else dev16(v)


# every form of the kernel (a row a wave, a row a workgroup of up to 8 pieces a lane, longer rows) and its edges
SHAPES = [(1, 8), (3, 64), (5, 512), (6, 520), (9, 1024), (2, 1032), (4, 2048), (3, 2056), (1, 4096), (7, 4104), (2, 7168), (2, 8192), (3, 8200),
          (2, 16384), (2, 16392), (1, 40000), (5, 50001 * 8), (1025, 256)]


@pytest.mark.parametrize("post,gate", [(False, ""), (True, "channel"), (False, "token"), (True, "token")])
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm(T, H, post, gate):
    x, r, w, p, g = case(T, H, post, gate)
    log(f"residual_norm {T} {H} {post} {gate}")
    y, h = fgg.residual_norm(up(x), up(r), up(w), post_weight=up(p), gate=up(g), scale=0.75)
    wy, wh = om.norm(x, r, w, p, g, 0.75)
    u = inner(x, p, g, 0.75)
    # (the post norm's own root mean square has the same roundings)
    loss = (np.log2(H) + H / 2048 + 16) * STEP * np.abs(u)
    check_bf16(c_to_f64(h), wh, loss + 8 * STEP * (np.abs(u) + np.abs(r)))
    check_bf16(c_to_f64(y), wy, norm_bound(u * (2 + np.log2(H) / 8 + H / 16384), r, w, wy, wh))


@pytest.mark.parametrize("T,H", [(1, 128), (3, 512), (5, 640), (2, 1024), (1, 2048), (9, 4096), (2, 7168), (3, 16384), (2, 16512), (700, 256)])
def test_norm_quantized(T, H):
    x, r, w, p, g = case(T, H, True, "channel")
    log(f"residual_norm quantized {T} {H}")
    (q, s), h = fgg.residual_norm(up(x), up(r), up(w), post_weight=up(p), gate=up(g), quantize=True)
    wy, wh = om.norm(x, r, w, p, g)
    u = inner(x, p, g, 1.0)
    check_bf16(c_to_f64(h), wh, (np.log2(H) + H / 2048 + 24) * STEP * (np.abs(u) + np.abs(r)))
    check_mxfp4(q.cpu().numpy(), s.cpu().numpy(), wy, norm_bound(u * (2 + np.log2(H) / 8 + H / 16384), r, w, wy, wh))


def test_plain_norm():
    """Without a residual h is x itself."""
    x, _, w, _, _ = case(33, 768, False, "")
    y, h = fgg.residual_norm(up(x), None, up(w), eps=1e-3)
    wy, wh = om.norm(x, None, w, eps=1e-3)
    assert np.array_equal(c_to_f64(h), x)
    check_bf16(c_to_f64(y), wy, norm_bound(x, None, w, wy, wh))


def test_rows_apart():
    """Rows of a wider tensor (a joint projection's part), a repeated residual row, one row."""
    import torch
    x, r, w, _, g = case(40, 384, False, "token")
    wide = torch.zeros((40, 1000), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:392] = up(x)
    base = torch.zeros((40, 1024), dtype=torch.bfloat16, device="cuda")
    base[:, 640:] = up(r)
    y, h = fgg.residual_norm(wide[:, 8:392], base[:, 640:], up(w), gate=up(g))
    want = fgg.residual_norm(up(x), up(r), up(w), gate=up(g))
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    one = up(r)[:1]
    a = fgg.residual_norm(up(x), one.expand(40, 384), up(w), gate=up(g)[:1].expand(40, 384))
    b = fgg.residual_norm(up(x), one.repeat(40, 1), up(w), gate=up(g)[0].contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    y1, h1 = fgg.residual_norm(wide[3:4, 8:392], base[3:4, 640:], up(w), gate=up(g)[3:4])
    assert torch.equal(y1, want[0][3:4]) and torch.equal(h1, want[1][3:4])


def test_zeros_and_values_that_are_not_finite():
    import torch
    x = torch.zeros((6, 256), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    x[3] = 2.0 ** 100  # whose squares are past FP32
    x[4, 3] = 2.0 ** -100
    y, h = fgg.residual_norm(x, None, w)
    assert not y[0].any() and torch.isnan(y[1]).all() and torch.equal(h[3:], x[3:]) and not y[3].any() and not y[5].any()
    assert torch.isnan(y[2, 9]) and not y[2, :9].any()
    (q, s), _ = fgg.residual_norm(x, None, w, quantize=True)
    assert (s[1] == 255).all() and not q[1].any() and s[2, 0] == 255 and not q[0].any() and not s[0].any()
    y, _ = fgg.residual_norm(x[:1], None, w, eps=0.0)
    assert torch.isnan(y).all()  # 0 / 0


def test_nothing_to_do():
    import torch
    x, w = torch.zeros((0, 256), dtype=torch.bfloat16, device="cuda"), torch.ones(256, dtype=torch.bfloat16, device="cuda")
    y, h = fgg.residual_norm(x, x, w)
    assert y.shape == h.shape == (0, 256)
    (q, s), h = fgg.residual_norm(x, None, w, quantize=True)
    assert q.shape == (0, 128) and s.shape == (0, 8)


def test_refusals():
    import torch
    x, w = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda"), torch.ones(256, dtype=torch.bfloat16, device="cuda")
    bad = [((x.float(), x, w), {}), ((x, x[:3], w), {}), ((x, x, w[:128]), {}), ((x, x, w.float()), {}), ((x.t(), x.t(), w[:4]), {}),
           ((x, x, w), dict(gate=w[:8])), ((x, x, w), dict(gate=x[:2])), ((x, x, w), dict(post_weight=w[::2])), ((x, x, None), {}),
           ((x, x, w), dict(eps=-1.0)), ((x, x, w), dict(scale=float("nan"))), ((x[:, :100], x[:, :100], w[:100]), {}),
           ((x[:, :96].contiguous(), None, w[:96].contiguous()), dict(quantize=True)), ((x[:, 1:9], None, w[:8]), {}),
           ((x.cpu(), None, w), {}), ((x, x.cpu(), w), {})]
    for args, kw in bad:
        with pytest.raises(ValueError):
            fgg.residual_norm(*args, **kw)
