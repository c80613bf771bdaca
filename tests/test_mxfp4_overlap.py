"""Results of the MXFP4 operators and of residual_norm lie apart from the operands and from each other: workgroups
write them while others still read.  Overlapping calls are refused before a device is touched; calls that are not
refused end there for want of one."""
import ctypes

import pytest
import torch

import fp4_grouped_gemm_amd as fgg

# a map of addresses that are never read: each operand has a GiB of its own
PLACE = {name: (i + 1) << 30 for i, name in enumerate(
    ["X", "Q", "scale", "rows", "A", "B", "a_scale", "b_scale", "m_indices", "C", "c_scale", "x", "residual", "gate", "post_weight",
     "weight", "h", "y", "y_scale"])}

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on addresses that are not there")


def refused(status):
    """What the overlapping pair is called, or None where something else, or nothing, stopped the call."""
    msg = fgg.load_library().fgg_last_error().decode()
    if status == 1 and "must not overlap" in msg:
        a, _, b = msg.split(": ", 1)[1].partition(" must not overlap ")
        return a, b
    return None


def run(which, at, **kw):
    """Calls entry point `which`, its operands at their places but for those in `at`."""
    lib, p = fgg.load_library(), {**PLACE, **at}
    if which == "quantize_mxfp4":
        return refused(lib.quantize_mxfp4(p["X"], p["Q"], p["scale"], 8, 256, None))
    if which == "quantize_mxfp4_rows":
        return refused(lib.quantize_mxfp4_rows(p["X"], p["rows"], p["Q"], p["scale"], 8, 5, 256, None))
    if which == "dequantize_mxfp4":
        return refused(lib.dequantize_mxfp4(p["Q"], p["scale"], p["X"], 8, 256, None))
    if which == "residual_norm":
        strides = (ctypes.c_longlong * 3)(*kw.get("strides", (256, 256, 0)))
        return refused(lib.residual_norm(p["x"], p["residual"], p["gate"], strides, p["post_weight"], p["weight"], 1.0, 1e-6,
                                         p["h"], p["y"], p["y_scale"], 4, 256, None))
    args = [p["A"], p["B"], p["a_scale"], p["b_scale"]] + ([p["m_indices"]] if "grouped" in which else []) + [p["C"]]
    args += [p["c_scale"]] if "gated" in which else []
    return refused(getattr(lib, which)(*args, 8, 64, 256, *([4] if "grouped" in which else []), None))


# bytes of each operand at the sizes above (products: M 8, N or F 64, K 256, G 4 or 1; the gated ones' C in MXFP4)
def sizes(which):
    if which == "quantize_mxfp4_rows":
        return dict(X=5 * 512, Q=8 * 128, scale=8 * 8, rows=32), ["Q", "scale"]
    if which == "quantize_mxfp4":
        return dict(X=8 * 512, Q=8 * 128, scale=8 * 8), ["Q", "scale"]
    if which == "dequantize_mxfp4":
        return dict(X=8 * 512, Q=8 * 128, scale=8 * 8), ["X"]
    if which == "residual_norm":
        return dict(x=2048, residual=2048, gate=512, post_weight=512, weight=512, h=2048, y=512, y_scale=32), ["h", "y", "y_scale"]
    gated = "gated" in which
    rows = 64 * (4 if "grouped" in which else 1) * (2 if gated else 1)
    s = dict(A=8 * 128, B=rows * 128, a_scale=64, b_scale=rows * 8, C=8 * 32 if gated else 8 * 128)
    if gated:
        s["c_scale"] = 8 * 2
    if "grouped" in which:
        s["m_indices"] = 32
    return s, ["C", "c_scale"] if gated else ["C"]


ALL = ["quantize_mxfp4", "quantize_mxfp4_rows", "dequantize_mxfp4", "mxfp4_gemm", "grouped_mxfp4_gemm", "mxfp4_gated_gemm",
       "grouped_mxfp4_gated_gemm", "residual_norm"]


def pairs():
    for which in ALL:
        size, results = sizes(which)
        for r in results:
            for other in size:
                if other != r:
                    yield which, r, other, size[r], size[other]


@pytest.mark.parametrize("which,r,other,n,m", list(pairs()))
def test_overlaps_are_refused(which, r, other, n, m):
    """The same place, the result's first bytes in the other's last, and its last in the other's first."""
    for at in (PLACE[other], PLACE[other] + m - 16, PLACE[other] - n + 16):
        got = run(which, {r: at})
        assert got is not None and set(got) == {r, other}, (at - PLACE[other], got)


@no_gpu
@pytest.mark.parametrize("which,r,other,n,m", list(pairs()))
def test_neighbours_are_not(which, r, other, n, m):
    for at in (PLACE[other] + m, PLACE[other] - n):
        assert run(which, {r: at}) is None


def test_rows_apart():
    """Strided rows are met where they lie: a result behind a row and before the next is apart from them."""
    gap = (4096, 4096, 0)  # rows of 512 bytes, 8192 apart
    for name in ("x", "residual"):
        for row in range(4):
            begin = PLACE[name] + row * 8192
            assert run("residual_norm", dict(h=begin + 496), strides=gap) == ("h", name)
            assert run("residual_norm", dict(h=begin - 2032), strides=gap) == ("h", name)
            assert run("residual_norm", dict(y_scale=begin + 480), strides=gap) == ("y_scale", name)
    # a gate of one row for all tokens, and one that is not there
    assert run("residual_norm", dict(h=PLACE["gate"] + 496), strides=gap) == ("h", "gate")


@no_gpu
def test_between_rows():
    for name in ("x", "residual"):
        for row in range(4):
            for at in (512, 8192 - 2048):
                assert run("residual_norm", dict(h=PLACE[name] + row * 8192 + at), strides=(4096, 4096, 0)) is None
    assert run("residual_norm", dict(h=PLACE["x"], x=PLACE["h"], residual=None, gate=None), strides=(256, 0, 0)) is None
