"""Attention entry points of the binding: the append of new keys and values to
a paged cache, single-token attention over that cache, and causal attention
over packed prompts (C ABI: rope_kv_append, paged_decode_attention,
prompt_attention in include/fgg.h).

As the rest of the binding these functions check types, shapes and devices,
derive sizes and strides and pass raw pointers and a HIP stream on; they do so
in a compiled module (csrc/attention_binding.cpp), because a call on one token
takes about 3 us on the GPU.  Nothing is read back to the host, so calls can be
captured in a HIP graph and replayed after positions, lengths, page tables or
their contents change.
"""
from __future__ import annotations

from . import compiled


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
    if stream is not None:
        with compiled.on(stream, q):
            return rope_kv_append(q, k, v, cos_sin, positions, page_table, k_cache, v_cache,
                                  seq_ids=seq_ids, interleaved=interleaved, k_scale=k_scale,
                                  v_scale=v_scale, return_k=return_k, out=out)
    return (compiled.C or compiled.load()).rope_kv_append(q, k, v, cos_sin, positions, page_table, k_cache, v_cache,
                                             seq_ids, interleaved, k_scale, v_scale, return_k, out)


def paged_decode_attention(q, k_cache, v_cache, page_table, lengths, *, scale=None, k_scale=None,
                           v_scale=None, out=None, stream=None):
    """Attention of one new token a sequence over its cached tokens.

    q: bfloat16 [B, Hq, D]; the cache as for rope_kv_append, Hq a multiple of
    its heads; page_table: int32 [B, W]; lengths: int32 [B], the cached tokens
    of each sequence (the new one among them); 0 gives zeros.  scale: of the
    scores, D ** -0.5 if None.  Returns bfloat16 [B, Hq, D]."""
    if stream is not None:
        with compiled.on(stream, q):
            return paged_decode_attention(q, k_cache, v_cache, page_table, lengths, scale=scale,
                                          k_scale=k_scale, v_scale=v_scale, out=out)
    return (compiled.C or compiled.load()).paged_decode_attention(q, k_cache, v_cache, page_table, lengths, scale,
                                                     k_scale, v_scale, out)


def prompt_attention(q, k, v, starts, *, scale=None, out=None, stream=None):
    """Causal attention over whole prompts packed one after the other.

    q [T, Hq, D], k and v [T, Hkv, D]: bfloat16, any strides of multiples of 8
    with D contiguous, Hq a multiple of Hkv.  starts: int32 [B + 1],
    non-decreasing: prompt i is the tokens [starts[i], starts[i + 1]); tokens
    of no prompt give zeros (a start before an earlier one counts as the largest
    of those).  scale: of the scores, D ** -0.5 if None.
    Returns bfloat16 [T, Hq, D]."""
    if stream is not None:
        with compiled.on(stream, q):
            return prompt_attention(q, k, v, starts, scale=scale, out=out)
    return (compiled.C or compiled.load()).prompt_attention(q, k, v, starts, scale, out)
