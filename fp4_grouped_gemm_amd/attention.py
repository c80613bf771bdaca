"""Attention entry points of the binding: the append of new keys and values to
a paged cache, single-token attention over that cache, and causal attention
over packed prompts (C ABI: rope_kv_append, paged_decode_attention,
prompt_attention in include/fgg.h).

As the rest of the binding these functions check types, shapes and devices,
derive sizes and strides and pass raw pointers and a HIP stream on.  Nothing
is read back to the host, so calls can be captured in a HIP graph and replayed
after positions, lengths, page tables or their contents change.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _check, load_library

KV_BF16, KV_E4M3 = 0, 1  # FGG_KV_*


class _KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_longlong), ("k_strides", ctypes.c_longlong * 3),
                ("v_strides", ctypes.c_longlong * 3), ("dtype", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("page_size", ctypes.c_int), ("head_dim", ctypes.c_int), ("batch", ctypes.c_int),
                ("table_width", ctypes.c_int)]


_Strides6 = ctypes.c_longlong * 6
_CODES = (torch.float8_e4m3fn, torch.uint8)
_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        lib = load_library()
        P, I, L, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
        C, S = ctypes.POINTER(_KvCache), ctypes.POINTER(ctypes.c_longlong)
        for name, args in (
            ("rope_kv_append", [C, P, P, P, S, P, I, I, I, P, P, P, P, I, I, P]),
            ("paged_decode_attention_workspace", [C, I, ctypes.POINTER(ctypes.c_size_t)]),
            ("paged_decode_attention", [C, P, L, L, P, F, P, I, P, ctypes.c_size_t, P]),
            ("prompt_attention", [P, P, P, S, P, F, P, I, I, I, I, I, P]),
        ):
            fn = getattr(lib, name)
            fn.restype = ctypes.c_int
            fn.argtypes = args
        _LIB = lib
    return _LIB


def _gpu(t, name, dtype, dim, device=None):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != dim:
        raise ValueError(f"{name} must be a {dim}-D {dtype} tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _heads(t, name, device=None):
    """A BF16 [rows, heads, head_dim] operand; head_dim contiguous."""
    _gpu(t, name, torch.bfloat16, 3, device)
    if t.stride(2) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t


def _vector(t, name, n, device, dtype=torch.int32):
    _gpu(t, name, dtype, 1, device)
    if t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape ({n},)")
    return t.data_ptr()


def _cache(k_cache, v_cache, page_table, k_scale, v_scale, device):
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{name} must be a tensor [pages, kv_heads, page_size, head_dim]")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
    if k_cache.dtype != v_cache.dtype or k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have one dtype and shape")
    fp8 = k_cache.dtype in _CODES
    if not fp8 and k_cache.dtype != torch.bfloat16:
        raise ValueError(f"a cache holds bfloat16 or E4M3 codes (float8_e4m3fn / uint8), got {k_cache.dtype}")
    ks, vs = k_cache.stride(), v_cache.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("k_cache and v_cache must be contiguous in their last dimension")
    pages, heads, page_size, dim = k_cache.shape
    _gpu(page_table, "page_table", torch.int32, 2, device)
    if page_table.stride(1) != 1 and page_table.shape[1] != 1:
        raise ValueError("page_table must be contiguous in its last dimension")
    scales = []
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t is not None and not fp8:
            raise ValueError(f"{name} goes with an E4M3 cache")
        scales.append(None if t is None else _vector(t, name, heads, device, torch.float32))
    return _KvCache(k_cache.data_ptr(), v_cache.data_ptr(), scales[0], scales[1],
                    page_table.data_ptr(), page_table.stride(0), ks[:3], vs[:3],
                    KV_E4M3 if fp8 else KV_BF16, pages, heads, page_size, dim,
                    page_table.shape[0], page_table.shape[1])


@contextlib.contextmanager
def _launch(device, stream):
    """The device of the call current; `stream` too if one is given, so that
    memory allocated for the call belongs to the stream that uses it.  Gives the
    raw stream."""
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device).cuda_stream
        else:
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


def _result(out, shape, name, device):
    if out is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=device)
    if out.dtype != torch.bfloat16 or tuple(out.shape) != tuple(shape) or out.device != device \
            or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bfloat16 tensor of shape {tuple(shape)} on {device}")
    return out


def rope_kv_append(q, k, v, cos_sin, positions, page_table, k_cache, v_cache, *, seq_ids=None,
                   interleaved=False, k_scale=None, v_scale=None, return_k=False, out=None,
                   stream=None):
    """Rotate new tokens' queries and keys and append keys and values to a paged cache.

    q [T, Hq, D], k and v [T, Hkv, D]: bfloat16, any strides of multiples of 8
    with D contiguous (views of a joint projection are taken as they are).
    cos_sin: float32 [P, R], row p the cosines of position p's R / 2 angles and
    then their sines.  positions: int32 [T]; a negative one is padding (nothing
    appended, zero rows in the results).  page_table: int32 [B, W];
    seq_ids: int32 [T], the table row of each token (None: token t is row t).
    k_cache, v_cache: [pages, Hkv, page_size, D] in any strides, bfloat16 or
    E4M3 codes with float32 scales k_scale, v_scale [Hkv].  They are updated in
    place.

    Returns the rotated queries [T, Hq, D] (into `out` if given), or with
    return_k (rotated queries, rotated keys): what prompt_attention reads.
    See include/fgg.h for the exact definition."""
    dev = _heads(q, "q").device
    _heads(k, "k", dev)
    _heads(v, "v", dev)
    cache = _cache(k_cache, v_cache, page_table, k_scale, v_scale, dev)
    T, hq, d = q.shape
    hk = cache.kv_heads
    if d != cache.head_dim or tuple(k.shape) != (T, hk, d) or tuple(v.shape) != (T, hk, d):
        raise ValueError(f"q must be [T, Hq, {cache.head_dim}], k and v [T, {hk}, {cache.head_dim}] as the cache")
    _gpu(cos_sin, "cos_sin", torch.float32, 2, dev)
    if not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be contiguous")
    pos = _vector(positions, "positions", T, dev)
    ids = None if seq_ids is None else _vector(seq_ids, "seq_ids", T, dev)
    strides = _Strides6(*q.stride()[:2], *k.stride()[:2], *v.stride()[:2])
    with _launch(dev, stream) as s:
        q_out = _result(out, (T, hq, d), "out", dev)
        k_out = torch.empty((T, hk, d), dtype=torch.bfloat16, device=dev) if return_k else None
        if T == 0:
            return (q_out, k_out) if return_k else q_out
        _check(_lib().rope_kv_append(
            cache, q.data_ptr(), k.data_ptr(), v.data_ptr(), strides, cos_sin.data_ptr(),
            cos_sin.shape[0], cos_sin.shape[1], bool(interleaved), pos, ids, q_out.data_ptr(),
            k_out.data_ptr() if return_k else None, T, hq, s))
    return (q_out, k_out) if return_k else q_out


def paged_decode_attention(q, k_cache, v_cache, page_table, lengths, *, scale=None, k_scale=None,
                           v_scale=None, out=None, stream=None):
    """Attention of one new token a sequence over its cached tokens.

    q: bfloat16 [B, Hq, D]; the cache as for rope_kv_append, Hq a multiple of
    its heads; page_table: int32 [B, W]; lengths: int32 [B], the cached tokens
    of each sequence (the new one among them); 0 gives zeros.  scale: of the
    scores, D ** -0.5 if None.  Returns bfloat16 [B, Hq, D]."""
    dev = _heads(q, "q").device
    cache = _cache(k_cache, v_cache, page_table, k_scale, v_scale, dev)
    B, hq, d = q.shape
    if d != cache.head_dim or B != cache.batch:
        raise ValueError(f"q must be [{cache.batch}, Hq, {cache.head_dim}] as the page table and the cache")
    lens = _vector(lengths, "lengths", B, dev)
    scale = d ** -0.5 if scale is None else float(scale)
    lib = _lib()
    with _launch(dev, stream) as s:
        res = _result(out, (B, hq, d), "out", dev)
        if B == 0:
            return res
        n = ctypes.c_size_t()
        _check(lib.paged_decode_attention_workspace(cache, hq, ctypes.byref(n)))
        work = torch.empty(n.value, dtype=torch.uint8, device=dev)
        _check(lib.paged_decode_attention(cache, q.data_ptr(), q.stride(0), q.stride(1), lens, scale,
                                          res.data_ptr(), hq, work.data_ptr(), n.value, s))
    return res


def prompt_attention(q, k, v, starts, *, scale=None, out=None, stream=None):
    """Causal attention over whole prompts packed one after the other.

    q [T, Hq, D], k and v [T, Hkv, D]: bfloat16, any strides of multiples of 8
    with D contiguous, Hq a multiple of Hkv.  starts: int32 [B + 1],
    non-decreasing: prompt i is the tokens [starts[i], starts[i + 1]); tokens
    of no prompt give zeros.  scale: of the scores, D ** -0.5 if None.
    Returns bfloat16 [T, Hq, D]."""
    dev = _heads(q, "q").device
    _heads(k, "k", dev)
    _heads(v, "v", dev)
    T, hq, d = q.shape
    hk = k.shape[1]
    if tuple(k.shape) != (T, hk, d) or tuple(v.shape) != (T, hk, d):
        raise ValueError(f"k and v must be [{T}, Hkv, {d}] as q")
    _gpu(starts, "starts", torch.int32, 1, dev)
    if starts.shape[0] < 2 or not starts.is_contiguous():
        raise ValueError("starts must be a contiguous int32 tensor of shape (B + 1,), B >= 1")
    scale = d ** -0.5 if scale is None else float(scale)
    strides = _Strides6(*q.stride()[:2], *k.stride()[:2], *v.stride()[:2])
    with _launch(dev, stream) as s:
        res = _result(out, (T, hq, d), "out", dev)
        if T == 0:
            return res
        _check(_lib().prompt_attention(q.data_ptr(), k.data_ptr(), v.data_ptr(), strides,
                                       starts.data_ptr(), scale, res.data_ptr(), T,
                                       starts.shape[0] - 1, hq, hk, d, s))
    return res
