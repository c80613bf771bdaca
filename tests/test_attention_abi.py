"""Refusals of the attention entry points: the C ABI's checks (before any
device is touched) and the binding's."""
import ctypes
import struct

import pytest

import fp4_grouped_gemm_amd as fgg

torch = pytest.importorskip("torch")

_KV_CACHE = struct.Struct("@PPPPPqqqqqqqiiiiiii")  # fgg_kv_cache
_STRIDES = struct.Struct("@6q")


def _lib():
    lib = fgg.load_library()
    P, I, L, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
    B = ctypes.c_char_p  # packed structures and arrays
    for name, args in (
        ("rope_kv_append", [B, P, P, P, B, P, I, I, I, P, P, P, P, I, I, P]),
        ("paged_decode_attention_workspace", [B, I, ctypes.POINTER(ctypes.c_size_t)]),
        ("paged_decode_attention", [B, P, L, L, P, F, P, I, P, ctypes.c_size_t, P]),
        ("prompt_attention", [P, P, P, B, P, F, P, I, I, I, I, I, P]),
    ):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = args
    return lib


P = 0x10000  # 16-byte aligned and never dereferenced: every call below is refused


def _cache(**kw):
    f = dict(k=P, v=P, k_scale=None, v_scale=None, page_table=P, table_stride=8,
             k_strides=(4096, 1024, 128), v_strides=(4096, 1024, 128), dtype=0, num_pages=10, kv_heads=4,
             page_size=8, head_dim=128, batch=3, table_width=8)
    f.update(kw)
    return _KV_CACHE.pack(*(f[n] or 0 for n in ("k", "v", "k_scale", "v_scale", "page_table", "table_stride")),
                          *f["k_strides"], *f["v_strides"],
                          *(f[n] for n in ("dtype", "num_pages", "kv_heads", "page_size", "head_dim", "batch",
                                           "table_width")))


CACHE = [
    (dict(k=0), 1, "null"),
    (dict(page_table=0), 1, "page_table"),
    (dict(dtype=2), 1, "dtype"),
    (dict(num_pages=0), 1, "num_pages"),
    (dict(page_size=0), 1, "page_size"),
    (dict(page_size=24), 2, "powers of two"),
    (dict(page_size=1 << 17), 1, "page_size"),
    (dict(batch=0), 1, "batch"),
    (dict(table_width=0), 1, "table_width"),
    (dict(table_width=1 << 28, page_size=16), 2, "2^31"),
    (dict(table_stride=-1), 1, "negative"),
    (dict(k_scale=P), 1, "E4M3"),
    (dict(dtype=1, k_scale=P + 2), 3, "4-byte"),
    (dict(k_strides=(4096, 1024, 132)), 3, "strides"),
    (dict(v_strides=(-8, 1024, 128)), 1, "negative"),
    (dict(dtype=1, v_strides=(4096, 1024, 136)), 3, "strides"),
    (dict(v=P + 8), 3, "aligned"),
    (dict(kv_heads=0), 1, "kv_heads"),
    (dict(kv_heads=3), 1, "q_heads"),
    (dict(head_dim=96), 2, "head_dim"),
]


def _append(cache=None, q=P, k=P, v=P, strides=(1024, 128, 512, 128, 512, 128), turns=P, num=100, rot=128,
            pos=P, ids=P, q_out=P, k_out=None, T=3, q_heads=8):
    lib = _lib()
    st = lib.rope_kv_append(cache or _cache(), q, k, v, _STRIDES.pack(*strides), turns, num, rot, 0, pos, ids,
                            q_out, k_out, T, q_heads, None)
    return st, lib.fgg_last_error().decode()


def _decode(cache=None, q=P, qs=1024, qh=128, lens=P, scale=0.1, out=P, q_heads=8, work=P, n=1 << 30):
    lib = _lib()
    st = lib.paged_decode_attention(cache or _cache(), q, qs, qh, lens, scale, out, q_heads, work, n, None)
    return st, lib.fgg_last_error().decode()


def _prompt(q=P, k=P, v=P, strides=(1024, 128, 512, 128, 512, 128), starts=P, scale=0.1, out=P, T=5,
            batch=2, hq=8, hk=4, d=128):
    lib = _lib()
    st = lib.prompt_attention(q, k, v, _STRIDES.pack(*strides), starts, scale, out, T, batch, hq, hk, d, None)
    return st, lib.fgg_last_error().decode()


@pytest.mark.parametrize("kw,status,needle", CACHE)
def test_cache_refusals(kw, status, needle):
    for fn, call in (("rope_kv_append", _append), ("paged_decode_attention", _decode)):
        st, msg = call(cache=_cache(**kw))
        assert st == status and msg.startswith(fn + ":") and needle in msg
    n = ctypes.c_size_t()
    lib = _lib()
    assert lib.paged_decode_attention_workspace(_cache(**kw), 8, ctypes.byref(n)) == status
    assert lib.paged_decode_attention_workspace(None, 8, ctypes.byref(n)) == 1


@pytest.mark.parametrize("kw,status,needle", [
    (dict(q=0), 1, "q is null"),
    (dict(v=P + 8), 3, "v must be"),
    (dict(strides=(1024, 128, 516, 128, 512, 128)), 3, "k must be"),
    (dict(strides=(1024, -128, 512, 128, 512, 128)), 1, "negative"),
    (dict(turns=0), 1, "cos_sin"),
    (dict(turns=P + 4), 3, "cos_sin"),
    (dict(num=0), 1, "no rows"),
    (dict(rot=0), 1, "rot_dim"),
    (dict(rot=130), 1, "rot_dim"),
    (dict(rot=63), 1, "rot_dim"),
    (dict(rot=24), 2, "rot_dim"),
    (dict(pos=0), 1, "positions"),
    (dict(pos=P + 2), 3, "positions"),
    (dict(q_out=0), 1, "q_out"),
    (dict(k_out=P + 8), 3, "k_out"),
    (dict(T=0), 1, "T"),
    (dict(T=(1 << 24) + 1), 1, "T"),
    (dict(T=1 << 24, q_heads=16), 2, "2^31"),
    (dict(ids=None, T=4), 1, "seq_ids"),
    (dict(q_heads=6), 1, "q_heads"),
])
def test_append_refusals(kw, status, needle):
    st, msg = _append(**kw)
    assert st == status and needle in msg


@pytest.mark.parametrize("kw,status,needle", [
    (dict(q=0), 1, "q is null"),
    (dict(q=P + 4), 3, "q must be"),
    (dict(qs=1028), 3, "strides"),
    (dict(lens=0), 1, "lengths"),
    (dict(lens=P + 2), 3, "lengths"),
    (dict(out=P + 8), 3, "out"),
    (dict(work=0), 1, "workspace"),
    (dict(work=P + 8), 3, "workspace"),
    (dict(scale=float("nan")), 1, "scale"),
    (dict(scale=float("inf")), 1, "scale"),
    (dict(q_heads=2), 1, "q_heads"),
    (dict(cache=_cache(batch=1 << 20, table_width=1 << 18, page_size=1), q_heads=4), 2, "2^30"),
])
def test_decode_refusals(kw, status, needle):
    st, msg = _decode(**kw)
    assert st == status and needle in msg


@pytest.mark.parametrize("kw,status,needle", [
    (dict(k=0), 1, "k is null"),
    (dict(out=0), 1, "out"),
    (dict(out=P + 8), 3, "out"),
    (dict(starts=0), 1, "starts"),
    (dict(starts=P + 2), 3, "starts"),
    (dict(T=0), 1, "T"),
    (dict(batch=0), 1, "batch"),
    (dict(scale=float("-inf")), 1, "scale"),
    (dict(d=80), 2, "head_dim"),
    (dict(hq=10), 1, "q_heads"),
    (dict(strides=(1024, 128, 512, 128, 512, 60)), 3, "v must be"),
    (dict(T=1 << 24, hq=1 << 12, hk=1 << 10), None, "2^31"),
])
def test_prompt_refusals(kw, status, needle):
    if status is None:  # (2^18 tiles) x 2^12 heads stays below 2^31: more prompts pass it
        kw, status = dict(kw, batch=1 << 20), 2
    st, msg = _prompt(**kw)
    assert st == status and msg.startswith("prompt_attention:") and needle in msg


def test_binding_refuses_cpu_tensors_and_wrong_types():
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        fgg.prompt_attention(q, q, q, torch.tensor([0, 2], dtype=torch.int32))
    with pytest.raises(ValueError, match="bfloat16"):
        fgg.prompt_attention(q.float(), q, q, torch.tensor([0, 2], dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        fgg.paged_decode_attention(q, q, q, q, q)
    with pytest.raises(ValueError, match="3-D"):
        fgg.rope_kv_append(q[0], q, q, q, q, q, q, q)
    with pytest.raises(AttributeError):
        fgg.no_such_entry
