"""What the C ABI of the MXFP4 operators and residual_norm refuses; every call fails before a device is touched."""
import ctypes

import pytest

import fp4_grouped_gemm_amd as fgg

P = 0x10000  # an aligned address that is never read


def said(status):
    return status, fgg.load_library().fgg_last_error().decode()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(X=0), 1, "null"), (dict(Q=0), 1, "null"), (dict(M=0), 1, "M"), (dict(M=(1 << 24) + 1), 1, "M"),
    (dict(K=16), 1, "K"), (dict(K=144), 1, "K % 32"), (dict(K=160), 2, "K % 128"), (dict(K=1 << 21), 1, "K"),
    (dict(X=P + 8), 3, "aligned"), (dict(Q=P + 4), 3, "aligned")])
@pytest.mark.parametrize("which", ["quantize_mxfp4", "quantize_mxfp4_rows", "dequantize_mxfp4"])
def test_quantisers(which, kw, status, needle):
    a = dict(X=P, Q=P, S=P, M=8, K=256)
    a.update(kw)
    lib = fgg.load_library()
    if which == "quantize_mxfp4":
        st, msg = said(lib.quantize_mxfp4(a["X"], a["Q"], a["S"], a["M"], a["K"], None))
    elif which == "quantize_mxfp4_rows":
        st, msg = said(lib.quantize_mxfp4_rows(a["X"], P, a["Q"], a["S"], a["M"], 5, a["K"], None))
    else:
        st, msg = said(lib.dequantize_mxfp4(a["Q"], a["S"], a["X"], a["M"], a["K"], None))
    assert st == status and msg.startswith(which + ":") and needle in msg


def test_rows():
    lib = fgg.load_library()
    for args, status, needle in (((P, 0, P, P, 8, 4, 256), 1, "rows"), ((P, P + 2, P, P, 8, 4, 256), 3, "rows"),
                                 ((P, P, P, P, 8, 0, 256), 1, "T"), ((P, P, P, P, 1 << 24, 4, 1 << 13), 2, "2^31")):
        st, msg = said(lib.quantize_mxfp4_rows(*args, None))
        assert st == status and needle in msg


PRODUCTS = ["mxfp4_gemm", "grouped_mxfp4_gemm", "mxfp4_gated_gemm", "grouped_mxfp4_gated_gemm"]


def product(which, **kw):
    a = dict(A=P, B=P, sa=P, sb=P, ids=P, C=P, sc=None, M=8, N=256, K=256, G=4)
    a.update(kw)
    args = [a["A"], a["B"], a["sa"], a["sb"]] + ([a["ids"]] if "grouped" in which else []) + [a["C"]]
    args += ([a["sc"]] if "gated" in which else []) + [a["M"], a["N"], a["K"]] + ([a["G"]] if "grouped" in which else [])
    return said(getattr(fgg.load_library(), which)(*args, None))


@pytest.mark.parametrize("kw,status,needle", [
    (dict(A=0), 1, "null"), (dict(B=0), 1, "null"), (dict(sa=0), 1, "null"), (dict(sb=0), 1, "null"), (dict(C=0), 1, "null"),
    (dict(M=0), 1, "M"), (dict(M=(1 << 24) + 1), 1, "M"), (dict(N=0), 1, "<="), (dict(N=(1 << 19) + 16), 1, "<="),
    (dict(N=40), 2, "% 16"), (dict(K=0), 1, "K"), (dict(K=100), 1, "K % 32"), (dict(K=160), 2, "K % 128"),
    (dict(K=(1 << 20) + 128), 1, "K"), (dict(A=P + 8), 3, "aligned"), (dict(B=P + 8), 3, "aligned"), (dict(C=P + 8), 3, "aligned"),
    (dict(sa=P + 2), 3, "aligned"), (dict(sb=P + 2), 3, "aligned")])
@pytest.mark.parametrize("which", PRODUCTS)
def test_products(which, kw, status, needle):
    st, msg = product(which, **kw)
    assert st == status and msg.startswith(which + ":") and needle in msg


@pytest.mark.parametrize("which", ["grouped_mxfp4_gemm", "grouped_mxfp4_gated_gemm"])
def test_routing(which):
    for kw, status, needle in ((dict(ids=0), 1, "m_indices"), (dict(ids=P + 2), 3, "m_indices"), (dict(G=0), 1, "G"),
                               (dict(G=(1 << 16) + 1), 1, "G"), (dict(G=1 << 16, N=2048), 2, "2^23")):
        st, msg = product(which, **kw)
        assert st == status and needle in msg


def test_codes_out_need_whole_blocks():
    for which in PRODUCTS[2:]:
        st, msg = product(which, sc=P, N=48)
        assert st == 1 and "F % 32" in msg


def norm(**kw):
    a = dict(x=P, r=P, g=P, strides=(256, 256, 0), pw=P, w=P, scale=1.0, eps=1e-6, h=P, y=P, sy=None, T=4, H=256)
    a.update(kw)
    strides = (ctypes.c_longlong * 3)(*a["strides"]) if a["strides"] else None
    return said(fgg.load_library().residual_norm(a["x"], a["r"], a["g"], strides, a["pw"], a["w"], a["scale"], a["eps"],
                                                 a["h"], a["y"], a["sy"], a["T"], a["H"], None))


@pytest.mark.parametrize("kw,status,needle", [
    (dict(x=0), 1, "null"), (dict(strides=None), 1, "null"), (dict(w=0), 1, "null"), (dict(h=0), 1, "null"), (dict(y=0), 1, "null"),
    (dict(T=0), 1, "T"), (dict(T=1 << 24), 1, "T"), (dict(H=0), 1, "H"), (dict(H=(1 << 20) + 8), 1, "H"), (dict(H=100), 2, "H % 8"),
    (dict(H=40, sy=P), 1, "H % 32"), (dict(H=96, sy=P), 2, "H % 128"), (dict(scale=float("nan")), 1, "scale"),
    (dict(scale=float("inf")), 1, "scale"), (dict(eps=-1.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"),
    (dict(x=P + 8), 3, "x must"), (dict(strides=(260, 256, 0)), 3, "x must"), (dict(strides=(256, 260, 0)), 3, "residual"),
    (dict(strides=(256, 256, 4)), 3, "gate"), (dict(strides=(-8, 256, 0)), 1, "negative"), (dict(r=P + 2), 3, "residual"),
    (dict(g=P + 2), 3, "gate"), (dict(pw=P + 2), 3, "aligned"), (dict(w=P + 2), 3, "aligned"), (dict(h=P + 2), 3, "aligned"),
    (dict(y=P + 2), 3, "aligned")])
def test_norm(kw, status, needle):
    st, msg = norm(**kw)
    assert st == status and msg.startswith("residual_norm:") and needle in msg


def test_host_tensors_are_refused():
    torch = pytest.importorskip("torch")
    b, q, s = torch.zeros((4, 128), dtype=torch.bfloat16), torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 4), dtype=torch.uint8)
    ids = torch.zeros(4, dtype=torch.int32)
    for f in (lambda: fgg.quantize_mxfp4(b), lambda: fgg.dequantize_mxfp4(q, s), lambda: fgg.mxfp4_gemm(q, q, s, s),
              lambda: fgg.mxfp4_gated_gemm(q, q, s, s), lambda: fgg.grouped_mxfp4_gemm(q, q[None], s, s[None], ids),
              lambda: fgg.grouped_mxfp4_gated_gemm(q, q[None], s, s[None], ids), lambda: fgg.residual_norm(b, b, b[0])):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError, match="m_indices"):
        fgg.grouped_mxfp4_gemm(q, q[None], s, s[None], None)
