"""A mixture-of-experts decoder layer served with the library: prompts in one
packed batch, then tokens one by one against the paged cache.

    python examples/moe_decoder.py

Random weights in NVFP4 (grouped_w4a16_gemm, projections as one expert),
rotated heads, BF16 or E4M3 cache.  Per layer and call:

    prompt   rope_kv_append (q, k rotated; k, v to the cache) -> prompt_attention
    token    rope_kv_append -> paged_decode_attention

The torch operations between (norms, residuals, router, SiLU) stand for the
rest of a model.  Nothing is read back to the host between the calls.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp4_grouped_gemm_amd as fgg  # noqa: E402


class PagedCache:
    """K and V pages of one layer, handed out to sequences from a free list."""

    def __init__(self, pages, kv_heads, page_size, head, sequences, max_len, fp8, device):
        shape = (pages, kv_heads, page_size, head)
        dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
        self.k, self.v = (torch.zeros(shape, device=device).to(dtype) for _ in range(2))
        # calibrated for values of a few units: codes reach 448
        self.scales = {n: torch.full((kv_heads,), 8.0 / 448, device=device) if fp8 else None
                       for n in ("k_scale", "v_scale")}
        self.table = torch.full((sequences, -(-max_len // page_size)), -1, dtype=torch.int32, device=device)
        self.free = list(range(pages))
        self.held = [0] * sequences
        self.page_size = page_size

    def reserve(self, sequence, length):
        """Pages for a sequence's first `length` tokens."""
        while self.held[sequence] * self.page_size < length:
            self.table[sequence, self.held[sequence]] = self.free.pop()
            self.held[sequence] += 1


class Linear:
    """NVFP4 weights [experts, out, in] for grouped_w4a16_gemm."""

    def __init__(self, experts, out, inp, gen):
        w = torch.randn((experts * out, inp), generator=gen, device=gen.device) * inp ** -0.5
        q, s, g = fgg.quantize_nvfp4(w.to(torch.bfloat16))
        self.q, self.s = q.view(experts, out, inp // 2), s.view(experts, out, inp // 16)
        self.scale = float(g)

    def __call__(self, x, expert):
        return fgg.grouped_w4a16_gemm(x, self.q, self.s, expert, self.scale)


def norm(x):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Layer:
    def __init__(self, hidden=512, q_heads=8, kv_heads=2, head=64, experts=4, ffn=256, top=2, positions=4096, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.q_heads, self.kv_heads, self.head, self.top = q_heads, kv_heads, head, top
        self.qkv = Linear(1, (q_heads + 2 * kv_heads) * head, hidden, gen)
        self.out = Linear(1, hidden, q_heads * head, gen)
        self.router = torch.randn((experts, hidden), generator=gen, device="cuda") * hidden ** -0.5
        self.up, self.down = Linear(experts, 2 * ffn, hidden, gen), Linear(experts, hidden, ffn, gen)
        angle = torch.arange(positions, device="cuda")[:, None] * \
            10000.0 ** (-torch.arange(0, head, 2, device="cuda") / head)
        self.turns = torch.cat([angle.cos(), angle.sin()], dim=1)

    def experts(self, x):
        """Each token through its `top` experts, weighted."""
        p, e = torch.softmax(x.float() @ self.router.t(), dim=-1).topk(self.top)
        rows = x.repeat_interleave(self.top, dim=0)
        ids = e.reshape(-1).int()
        gate, up = self.up(rows, ids).chunk(2, dim=-1)
        y = self.down(torch.nn.functional.silu(gate) * up, ids).view(len(x), self.top, -1)
        return (y * (p / p.sum(-1, keepdim=True))[..., None]).sum(1).to(torch.bfloat16)

    def __call__(self, x, cache, positions, seq_ids, *, starts=None, lengths=None):
        """x [T, hidden]: whole packed prompts (starts), or a token of each
        sequence (lengths: cached tokens, the new ones among them)."""
        one = torch.zeros(len(x), dtype=torch.int32, device=x.device)
        heads = self.qkv(norm(x), one).view(len(x), -1, self.head)
        q, k, v = heads.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)  # views
        q, k = fgg.rope_kv_append(q, k, v, self.turns, positions, cache.table, cache.k, cache.v, seq_ids=seq_ids,
                                  return_k=True, **cache.scales)
        if starts is not None:
            y = fgg.prompt_attention(q, k, v, starts)
        else:
            y = fgg.paged_decode_attention(q, cache.k, cache.v, cache.table, lengths, **cache.scales)
        x = x + self.out(y.flatten(1), one)
        return x + self.experts(norm(x))


def packed(lens, device="cuda"):
    """positions, sequence ids and starts of packed prompts."""
    pos = torch.cat([torch.arange(n) for n in lens]).int()
    ids = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).int()
    starts = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)
    return pos.to(device), ids.to(device), starts.to(device)


def serve(layers, inputs, prompt_lens, steps, fp8):
    """Runs prompts and then `steps` tokens a sequence; inputs [sequences,
    longest, hidden] holds what enters the first layer at each position.  Returns
    what leaves the last one: per sequence, prompt_lens + steps rows."""
    n, longest, _ = inputs.shape
    c = layers[0]
    caches = [PagedCache(n * -(-longest // 16), c.kv_heads, 16, c.head, n, longest, fp8, inputs.device) for _ in layers]
    for cache in caches:
        for b, length in enumerate(prompt_lens):
            cache.reserve(b, length + steps)
    pos, ids, starts = packed(prompt_lens, inputs.device)
    x = inputs[ids.long(), pos.long()]
    for layer, cache in zip(layers, caches):
        x = layer(x, cache, pos, ids, starts=starts)
    outs = [list(p) for p in x.split(prompt_lens)]
    length = torch.tensor(prompt_lens, dtype=torch.int32, device=inputs.device)
    rows = torch.arange(n, dtype=torch.int32, device=inputs.device)
    for _ in range(steps):
        x = inputs[rows.long(), length.long()]
        for layer, cache in zip(layers, caches):
            x = layer(x, cache, length, rows, lengths=length + 1)
        length = length + 1
        for b in range(n):
            outs[b].append(x[b])
    return [torch.stack(o) for o in outs]


def main():
    torch.manual_seed(0)
    layers = [Layer(seed=i) for i in range(2)]
    lens, steps = [37, 5, 130], 6
    inputs = torch.randn((len(lens), max(lens) + steps, 512), device="cuda").to(torch.bfloat16)
    whole = serve(layers, inputs, [n + steps for n in lens], 0, False)
    off = {}
    for fp8 in (False, True):
        got = serve(layers, inputs, lens, steps, fp8)
        off[fp8] = max(((g - w).float().norm() / w.float().norm()).item() for g, w in zip(got, whole))
        print(f"{sum(lens)} prompt tokens, then {steps} of each sequence, {'E4M3' if fp8 else 'BF16'} cache: "
              f"relative difference to the whole sequences as prompts {off[fp8]:.2e}", flush=True)
    return off


if __name__ == "__main__":
    main()
