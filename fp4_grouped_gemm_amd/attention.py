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

import ctypes
import struct

import torch

from . import _check, load_library

KV_BF16, KV_E4M3 = 0, 1  # FGG_KV_*

# fgg_kv_cache and the strides arrays, packed with the struct module: a call on
# one token takes about 3 us on the GPU, and filling a ctypes structure field by
# field would cost the host as much.
_KV_CACHE = struct.Struct("@PPPPPqqqqqqqiiiiiii")
_STRIDES = struct.Struct("@6q")
_CODES = (torch.float8_e4m3fn, torch.uint8)
_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
_LIB = None
_WORKSPACE = {}  # bytes by device and sizes


def _lib():
    global _LIB
    if _LIB is None:
        lib = load_library()
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
        _LIB = lib
    return _LIB


def _bad(t, name, dtype, dim, device):
    """Raises what is wrong with a tensor that is not `dim`-D of `dtype` on
    `device` (None: any GPU)."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != dim:
        raise ValueError(f"{name} must be a {dim}-D {dtype} tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")


# (The checks read each attribute once: they are most of a small call's time.)
def _heads(t, name, device=None):
    """Checks a BF16 [rows, heads, head_dim] operand, head_dim contiguous: its
    device and its strides."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _BF16:
        _bad(t, name, _BF16, 3, device)
    d, st = t.get_device(), t.stride()
    if len(st) != 3 or d < 0 or (device is not None and d != device):
        _bad(t, name, _BF16, 3, device)
    if st[2] != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return d, st


def _matrix(t, name, dtype, device):
    """Checks a 2-D tensor, its last dimension contiguous: shape and row stride."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != device:
        _bad(t, name, dtype, 2, device)
    shape, st = t.shape, t.stride()
    if len(shape) != 2:
        _bad(t, name, dtype, 2, device)
    if st[1] != 1 and shape[1] != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return shape, st[0]


def _vector(t, name, n, device, dtype=_I32):
    """Checks a contiguous vector of n values (None: of any length): its address."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != device or t.dim() != 1:
        _bad(t, name, dtype, 1, device)
    if (n is not None and t.shape[0] != n) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape ({n},)")
    return t.data_ptr()


def _cache(k_cache, v_cache, page_table, k_scale, v_scale, device):
    """Checks a cache: the packed fgg_kv_cache and its kv_heads, page_size,
    head_dim, batch and table width."""
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{name} must be a tensor [pages, kv_heads, page_size, head_dim]")
        if t.get_device() != device:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    shape, dtype = k_cache.shape, k_cache.dtype
    if dtype is not v_cache.dtype or shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have one dtype and shape")
    fp8 = dtype in _CODES
    if not fp8 and dtype is not _BF16:
        raise ValueError(f"a cache holds bfloat16 or E4M3 codes (float8_e4m3fn / uint8), got {dtype}")
    ks, vs = k_cache.stride(), v_cache.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("k_cache and v_cache must be contiguous in their last dimension")
    pages, heads, page_size, dim = shape
    (batch, width), row = _matrix(page_table, "page_table", _I32, device)
    if not fp8 and (k_scale is not None or v_scale is not None):
        raise ValueError("k_scale and v_scale go with an E4M3 cache")
    k_sc = 0 if k_scale is None else _vector(k_scale, "k_scale", heads, device, _F32)
    v_sc = 0 if v_scale is None else _vector(v_scale, "v_scale", heads, device, _F32)
    packed = _KV_CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), k_sc, v_sc,
                            page_table.data_ptr(), row, ks[0], ks[1], ks[2], vs[0], vs[1], vs[2],
                            KV_E4M3 if fp8 else KV_BF16, pages, heads, page_size, dim, batch, width)
    return packed, heads, page_size, dim, batch, width


def _elsewhere(device, stream):
    """None if the call's device and stream are the current ones; else a context
    that makes them so, so that memory allocated for the call belongs to the
    stream that uses it."""
    if stream is None:
        return None if _current_device() == device else torch.cuda.device(device)
    if stream.device.index != device:
        raise ValueError(f"stream is on {stream.device}, expected cuda:{device}")
    return torch.cuda.stream(stream)


def _result(out, q, shape, device):
    if out is None:
        return q.new_empty(shape)
    if out.dtype != _BF16 or tuple(out.shape) != shape or out.get_device() != device \
            or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous bfloat16 tensor of shape {shape} on cuda:{device}")
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
    dev, qs = _heads(q, "q")
    ks, vs = _heads(k, "k", dev)[1], _heads(v, "v", dev)[1]
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return rope_kv_append(q, k, v, cos_sin, positions, page_table, k_cache, v_cache,
                                  seq_ids=seq_ids, interleaved=interleaved, k_scale=k_scale,
                                  v_scale=v_scale, return_k=return_k, out=out)
    cache, hk, _, dim, _, _ = _cache(k_cache, v_cache, page_table, k_scale, v_scale, dev)
    T, hq, d = q.shape
    if d != dim or k.shape != (T, hk, d) or v.shape != (T, hk, d):
        raise ValueError(f"q must be [T, Hq, {dim}], k and v [T, {hk}, {dim}] as the cache")
    (turns, rot), row = _matrix(cos_sin, "cos_sin", _F32, dev)
    if row != rot and turns != 1:
        raise ValueError("cos_sin must be contiguous")
    pos = _vector(positions, "positions", T, dev)
    ids = None if seq_ids is None else _vector(seq_ids, "seq_ids", T, dev)
    res = _result(out, q, (T, hq, d), dev)
    k_out = q.new_empty((T, hk, d)) if return_k else None
    if T:
        strides = _STRIDES.pack(qs[0], qs[1], ks[0], ks[1], vs[0], vs[1])
        _check(_lib().rope_kv_append(
            cache, q.data_ptr(), k.data_ptr(), v.data_ptr(), strides, cos_sin.data_ptr(), turns, rot,
            1 if interleaved else 0, pos, ids, res.data_ptr(),
            k_out.data_ptr() if return_k else None, T, hq, _raw_stream(dev)))
    return (res, k_out) if return_k else res


def paged_decode_attention(q, k_cache, v_cache, page_table, lengths, *, scale=None, k_scale=None,
                           v_scale=None, out=None, stream=None):
    """Attention of one new token a sequence over its cached tokens.

    q: bfloat16 [B, Hq, D]; the cache as for rope_kv_append, Hq a multiple of
    its heads; page_table: int32 [B, W]; lengths: int32 [B], the cached tokens
    of each sequence (the new one among them); 0 gives zeros.  scale: of the
    scores, D ** -0.5 if None.  Returns bfloat16 [B, Hq, D]."""
    dev, qs = _heads(q, "q")
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return paged_decode_attention(q, k_cache, v_cache, page_table, lengths, scale=scale,
                                          k_scale=k_scale, v_scale=v_scale, out=out)
    cache, hk, page_size, dim, batch, width = _cache(k_cache, v_cache, page_table, k_scale, v_scale, dev)
    B, hq, d = q.shape
    if d != dim or B != batch:
        raise ValueError(f"q must be [{batch}, Hq, {dim}] as the page table and the cache")
    lens = _vector(lengths, "lengths", B, dev)
    res = _result(out, q, (B, hq, d), dev)
    if B:
        lib, sizes = _lib(), (dev, B, hq, hk, d, page_size * width)
        n = _WORKSPACE.get(sizes)
        if n is None:
            need = ctypes.c_size_t()
            _check(lib.paged_decode_attention_workspace(cache, hq, ctypes.byref(need)))
            if len(_WORKSPACE) >= 4096:
                _WORKSPACE.clear()
            n = _WORKSPACE[sizes] = need.value
        # (a call that needs no workspace is given its output's address)
        work = torch.empty(n, dtype=torch.uint8, device=q.device) if n else res
        _check(lib.paged_decode_attention(cache, q.data_ptr(), qs[0], qs[1], lens,
                                          d ** -0.5 if scale is None else float(scale),
                                          res.data_ptr(), hq, work.data_ptr(), n, _raw_stream(dev)))
    return res


def prompt_attention(q, k, v, starts, *, scale=None, out=None, stream=None):
    """Causal attention over whole prompts packed one after the other.

    q [T, Hq, D], k and v [T, Hkv, D]: bfloat16, any strides of multiples of 8
    with D contiguous, Hq a multiple of Hkv.  starts: int32 [B + 1],
    non-decreasing: prompt i is the tokens [starts[i], starts[i + 1]); tokens
    of no prompt give zeros.  scale: of the scores, D ** -0.5 if None.
    Returns bfloat16 [T, Hq, D]."""
    dev, qs = _heads(q, "q")
    ks, vs = _heads(k, "k", dev)[1], _heads(v, "v", dev)[1]
    elsewhere = _elsewhere(dev, stream)
    if elsewhere is not None:
        with elsewhere:
            return prompt_attention(q, k, v, starts, scale=scale, out=out)
    T, hq, d = q.shape
    hk = k.shape[1]
    if k.shape != (T, hk, d) or v.shape != (T, hk, d):
        raise ValueError(f"k and v must be [{T}, Hkv, {d}] as q")
    starts_ptr = _vector(starts, "starts", None, dev)
    batch = starts.shape[0] - 1
    if batch < 1:
        raise ValueError("starts must be an int32 tensor of shape (B + 1,), B >= 1")
    res = _result(out, q, (T, hq, d), dev)
    if T:
        strides = _STRIDES.pack(qs[0], qs[1], ks[0], ks[1], vs[0], vs[1])
        _check(_lib().prompt_attention(q.data_ptr(), k.data_ptr(), v.data_ptr(), strides,
                                       starts_ptr, d ** -0.5 if scale is None else float(scale),
                                       res.data_ptr(), T, batch, hq, hk, d, _raw_stream(dev)))
    return res
