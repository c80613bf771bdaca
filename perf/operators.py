"""Cases of the attention operators: position rotation with the append to a paged key-value cache
(op "append"), attention of one new token over that cache (op "decode") and causal attention over
whole packed prompts (op "prompt").

Each case is a call as a serving loop of a mixture-of-experts layer makes it.  `run` computes it
with elementary torch operations in FP32 (own = False) or by the library's entry points (own =
True); `exact` computes it in FP64, sequence by sequence.

Keys of a case: op; q_heads, kv_heads, head (size of a head); fp8 (the cache holds E4M3 codes with
one scale per KV head, else BF16); page (tokens of a page); and
  append: seqs x new (new tokens of each of seqs sequences; new = 1 is decode), context (tokens
          already cached: lowest and highest of the batch), rot (rotated part of a head),
          interleaved (pairs (2i, 2i + 1) instead of (i, i + rot / 2)), padding (rows at the end of
          the batch that are no token), keys (the rotated keys are returned too, for
          prompt_attention)
  decode: seqs, low, high (cached tokens of the sequences: spread between them over the logarithm)
  prompt: seqs, low, high (lengths of the packed prompts, spread likewise)
"""
import math

import torch

own = False

POSITIONS = 1 << 18  # rows of the rotation table: the longest context served
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    append = dict(op="append", page=16, rot=128, interleaved=False, padding=0, keys=False)
    decode = dict(op="decode", page=16, fp8=False)
    return [
        # one user's next token: the call is all latency
        dict(append, name="append one token", q_heads=32, kv_heads=8, head=128, fp8=False, seqs=1, new=1, low=1000, high=1000),
        # a decode batch padded to its captured size, E4M3 cache, half of each head rotated
        dict(append, name="append batch fp8", q_heads=64, kv_heads=8, head=128, fp8=True, seqs=250, new=1, low=1, high=20000,
             page=64, rot=64, interleaved=True, padding=6),
        # prompts enter the cache; their rotated keys go on to the prompt's attention
        dict(append, name="append prompts", q_heads=32, kv_heads=8, head=128, fp8=False, seqs=5, new=3333, low=0, high=0, keys=True),
        # one user, a short chat: few tokens to spread over the card
        dict(decode, name="decode one short", q_heads=32, kv_heads=8, head=128, seqs=1, low=517, high=517),
        # one user, a long document: few heads, split over the length
        dict(decode, name="decode one long", q_heads=32, kv_heads=4, head=128, seqs=1, low=130001, high=130001),
        # a serving batch of mixed ages, from the first token on
        dict(decode, name="decode ragged", q_heads=64, kv_heads=8, head=128, seqs=96, low=1, high=6000, page=64),
        # a large batch with the cache in E4M3
        dict(decode, name="decode fp8", q_heads=64, kv_heads=8, head=128, seqs=128, low=2000, high=8191, fp8=True, page=32),
        # the card filled with long contexts; heads of 64 with a key head each second query head
        dict(decode, name="decode large", q_heads=32, kv_heads=16, head=64, seqs=64, low=12000, high=32768, page=128),
        # one short prompt: latency
        dict(op="prompt", name="prompt short", q_heads=32, kv_heads=8, head=128, seqs=1, low=77, high=77),
        # many prompts of a chat service packed without padding, odd lengths
        dict(op="prompt", name="prompts packed", q_heads=32, kv_heads=8, head=64, seqs=24, low=17, high=1501),
        # a prompt of a few pages on the heads of one of several GPUs
        dict(op="prompt", name="prompt few heads", q_heads=8, kv_heads=1, head=128, seqs=1, low=4001, high=4001),
        # long documents, all heads
        dict(op="prompt", name="prompts long", q_heads=32, kv_heads=8, head=128, seqs=2, low=4096, high=8192),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "decode", "prompt"])
    kv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, kv_heads=kv, q_heads=kv * rng.choice([1, 2, 4, 7, 8]), head=rng.choice([64, 128]))
    if op == "append":
        new = rng.choice([1, 1, spread(2, 2000)])
        c.update(fp8=rng.random() < 0.5, page=rng.choice([1, 16, 32, 64, 256]), new=new,
                 seqs=spread(1, 300) if new == 1 else spread(1, max(2, 12000 // new)), low=0, high=spread(1, 30000),
                 rot=rng.choice([32, c["head"]]), interleaved=rng.random() < 0.5, padding=rng.choice([0, 0, rng.randint(1, 9)]),
                 keys=rng.random() < 0.5)
        if new > 1:
            c.update(high=c["low"])
    elif op == "decode":
        high = spread(1, 60000)
        c.update(fp8=rng.random() < 0.5, page=rng.choice([1, 16, 32, 64, 256]), low=rng.randint(1, high), high=high,
                 seqs=spread(1, max(2, min(256, 600000 // high))))
    else:
        high = spread(1, 6000)
        c.update(low=rng.randint(1, high), high=high, seqs=spread(1, max(1, min(64, 9000 // high))))
    return c


def lengths_of(case):
    """The lengths of the case's sequences (cached tokens, or prompts): its lowest and highest, and
    the others between them over the logarithm, in an order that mixes them."""
    n, lo, hi = case["seqs"], max(case["low"], 0), case["high"]
    if n == 1:
        return [hi]
    got = [int(round(math.exp(math.log(lo + 1) + (math.log(hi + 1) - math.log(lo + 1)) * i / (n - 1)))) - 1 for i in range(n)]
    step = next(s for s in range(max(1, int(n * 0.618)), n + 1) if math.gcd(s, n) == 1)
    return [got[i * step % n] for i in range(n)]


def work(case):
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head"]
    code = 1 if case.get("fp8") else 2
    if case["op"] == "append":
        tokens = case["seqs"] * case["new"]
        rows = tokens + case["padding"]
        read = tokens * ((hq + 2 * hk) * d * 2 + case["rot"] * 4 + 4) + rows * 8
        write = rows * hq * d * 2 + tokens * 2 * hk * d * code + (rows * hk * d * 2 if case["keys"] else 0)
        return {"bytes": read + write, "flops": 3 * tokens * (hq + hk) * case["rot"]}
    lens = lengths_of(case)
    if case["op"] == "decode":
        pages = sum(-(-n // case["page"]) for n in lens)
        return {"bytes": 2 * sum(lens) * hk * d * code + 2 * len(lens) * hq * d * 2 + 4 * (pages + len(lens)),
                "flops": 4 * sum(lens) * hq * d}
    tokens = sum(lens)
    return {"bytes": 2 * tokens * (hq + hk) * d * 2 + 4 * (len(lens) + 1),
            "flops": 4 * hq * d * sum(n * (n + 1) // 2 for n in lens)}


# ----------------------------------------------------------------- inputs
def rotation_table(rot, device):
    """FP32 [POSITIONS, rot]: the cosines of a position's rot / 2 angles, then the sines."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    angle = torch.arange(POSITIONS, device=device, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head"]

    def bf16(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)

    s = {"case": case, "scale": d ** -0.5}
    lens = lengths_of(case)
    if case["op"] == "prompt":
        n = sum(lens)
        s["q"], s["k"], s["v"] = bf16(n, hq, d), bf16(n, hk, d), bf16(n, hk, d)
        s["starts"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=dev)
        return s
    # a pool whose pages the sequences hold in shuffled order; the last page belongs to nobody
    page = case["page"]
    new = case.get("new", 0)
    need = [-(-(n + new) // page) for n in lens]
    width = max(need)
    # an append writes into its sequences' last pages only: its pool holds no others
    first = [n // page if case["op"] == "append" else 0 for n in lens]
    pool = sum(need) - sum(first) + 1
    order = torch.randperm(pool - 1, generator=g, device=dev, dtype=torch.int32)
    own_pages = torch.tensor([n - f for n, f in zip(need, first)], device=dev)
    ends = own_pages.cumsum(0)
    col = torch.arange(width, device=dev)[None, :] - torch.tensor(first, device=dev)[:, None]
    mine = (col >= 0) & (col < own_pages[:, None])
    s["table"] = torch.where(mine, order[((ends - own_pages)[:, None] + col).clamp(0, pool - 2)], torch.full_like(col, -1, dtype=torch.int32)).int().contiguous()
    for name in ("k_cache", "v_cache"):
        x = bf16(pool, hk, page, d)
        s[name] = (x * 64).to(torch.float8_e4m3fn) if case["fp8"] else x
        # calibrated scales: values of a few units fill the codes' range
        s[name[0] + "_scale"] = (0.8 + 0.4 * torch.rand(hk, generator=g, device=dev)) / 64 if case["fp8"] else None
    if case["op"] == "decode":
        s["q"] = bf16(len(lens), hq, d)
        s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        return s
    rows = len(lens) * new + case["padding"]
    # q, k and v as one projection leaves them: side by side in each token's row
    qkv = bf16(rows, hq + 2 * hk, d)
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    s["turns"] = rotation_table(case["rot"], dev)
    pos = (torch.tensor(lens, device=dev)[:, None] + torch.arange(new, device=dev)[None, :]).reshape(-1)
    ids = torch.arange(len(lens), device=dev)[:, None].expand(-1, new).reshape(-1)
    s["positions"] = torch.cat([pos, torch.full((case["padding"],), -1, device=dev)]).int()
    s["seq_ids"] = torch.cat([ids, torch.zeros(case["padding"], dtype=ids.dtype, device=dev)]).int()
    return s


# -------------------------------------------------------------- operators
def run(s):
    op = s["case"]["op"]
    if own:
        import fp4_grouped_gemm_amd as fgg
        if op == "append":
            got = fgg.rope_kv_append(s["q"], s["k"], s["v"], s["turns"], s["positions"], s["table"], s["k_cache"],
                                     s["v_cache"], seq_ids=s["seq_ids"], interleaved=s["case"]["interleaved"],
                                     k_scale=s["k_scale"], v_scale=s["v_scale"], return_k=s["case"]["keys"])
            q, k = got if s["case"]["keys"] else (got, None)
            return {"q": q, "k": k, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if op == "decode":
            return fgg.paged_decode_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], scale=s["scale"],
                                              k_scale=s["k_scale"], v_scale=s["v_scale"])
        return fgg.prompt_attention(s["q"], s["k"], s["v"], s["starts"], scale=s["scale"])
    return {"append": plain_append, "decode": plain_decode, "prompt": plain_prompt}[op](s)


def turned(x, turn, rot, interleaved):
    """x [T, H, D] with the first rot values of each head rotated by turn [T, rot]; FP32."""
    x = x.float()
    cos, sin = turn[:, None, :rot // 2], turn[:, None, rot // 2:]
    part, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([part, rest], dim=-1)


def put(cache, scale, x, page, slot, valid):
    """Writes x [T, H, D] (FP32) to its slots; rows that are no token leave the spare page as it is."""
    if scale is not None:
        x = (x / scale[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        cache = cache.view(torch.uint8)
    else:
        x = x.to(cache.dtype)
    cache[page, :, slot] = torch.where(valid[:, None, None], x, cache[page, :, slot])


def plain_append(s):
    case, pos = s["case"], s["positions"].long()
    valid = pos >= 0
    at = pos.clamp(min=0)
    turn = s["turns"][at]
    q = turned(s["q"], turn, case["rot"], case["interleaved"])
    k = turned(s["k"], turn, case["rot"], case["interleaved"])
    page = s["table"][s["seq_ids"].long(), at // case["page"]].long()
    page = torch.where(valid, page, s["k_cache"].shape[0] - 1)
    slot = torch.where(valid, at % case["page"], 0)
    put(s["k_cache"], s["k_scale"], k, page, slot, valid)
    put(s["v_cache"], s["v_scale"], s["v"].float(), page, slot, valid)
    q = torch.where(valid[:, None, None], q, 0.0).to(torch.bfloat16)
    k = torch.where(valid[:, None, None], k, 0.0).to(torch.bfloat16) if case["keys"] else None
    return {"q": q, "k": k, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def gathered(cache, scale, table):
    """FP32 [B, H, tokens, D] of the pages that table [B, W] names."""
    b, w = table.shape
    x = cache.view(torch.uint8)[table].view(cache.dtype) if scale is not None else cache[table]
    x = x.float().transpose(1, 2).flatten(2, 3)
    return x * scale[None, :, None, None] if scale is not None else x


def softmaxed(x, mask):
    """Softmax over the last axis of the values that mask admits; rows without any give zeros."""
    x = torch.where(mask, x, -torch.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -torch.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total)


def plain_decode(s):
    q, lens = s["q"], s["lengths"]
    b, hq, d = q.shape
    table = s["table"].clamp(min=0).long()
    k = gathered(s["k_cache"], s["k_scale"], table)
    x = torch.matmul(q.float().view(b, k.shape[1], -1, d), k.transpose(-1, -2)) * s["scale"]
    del k
    mask = torch.arange(x.shape[-1], device=q.device)[None, :] < lens[:, None]
    p = softmaxed(x, mask[:, None, None, :])
    v = gathered(s["v_cache"], s["v_scale"], table)
    return torch.matmul(p, v).view(b, hq, d).to(torch.bfloat16)


def plain_prompt(s):
    q, k, v, starts = s["q"], s["k"], s["v"], s["starts"]
    t, hq, d = q.shape
    hk = k.shape[1]
    at = torch.arange(t, device=q.device)
    seq = torch.bucketize(at, starts[1:-1].long(), right=True)
    mask = (seq[:, None] == seq[None, :]) & (at[None, :] <= at[:, None])
    qh = q.float().view(t, hk, -1, d).permute(1, 2, 0, 3).flatten(1, 2)
    kh, vh = k.float().permute(1, 2, 0), v.float().transpose(0, 1)
    x = torch.matmul(qh, kh).view(hk, -1, t, t) * s["scale"]
    p = softmaxed(x, mask)
    o = torch.matmul(p.view(hk, -1, t), vh).view(hq, t, d)
    return o.transpose(0, 1).to(torch.bfloat16).contiguous()


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The same in FP64, one sequence (or token) at a time.  E4M3 caches: the values before they
    are rounded to codes."""
    s = prepare(case, seed)
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head"]
    group = hq // hk
    if case["op"] == "append":
        half = case["rot"] // 2
        pos = s["positions"].tolist()
        ids = s["seq_ids"].tolist()
        table = s["table"].tolist()
        real = [t for t, p in enumerate(pos) if p >= 0]
        turn = s["turns"].double()[[pos[t] for t in real]]
        first, second = (list(range(0, 2 * half, 2)), list(range(1, 2 * half, 2))) if case["interleaved"] else (list(range(half)), list(range(half, 2 * half)))

        def rotate(x):
            y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
            z = x[real].double()
            w = z.clone()
            for i in range(half):
                c, n = turn[:, i, None], turn[:, half + i, None]
                w[:, :, first[i]] = z[:, :, first[i]] * c - z[:, :, second[i]] * n
                w[:, :, second[i]] = z[:, :, second[i]] * c + z[:, :, first[i]] * n
            y[real] = w
            return y

        pages = [table[ids[t]][pos[t] // case["page"]] for t in real]
        slots = [pos[t] % case["page"] for t in real]
        q, k = rotate(s["q"]), rotate(s["k"])
        out = {"q": q, "k": k if case["keys"] else None}
        for name, x, scale in (("k_cache", k, s["k_scale"]), ("v_cache", s["v"].double(), s["v_scale"])):
            cache = s[name].double()
            y = x[real]
            if scale is not None:
                y = (y / scale.double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
            cache[torch.tensor(pages, device=q.device), :, torch.tensor(slots, device=q.device)] = y
            out[name] = cache
        return out
    lens = lengths_of(case)
    if case["op"] == "decode":
        out = torch.zeros((len(lens), hq, d), dtype=torch.float64, device=s["q"].device)
        for b, n in enumerate(lens):
            if n == 0:
                continue
            pages = s["table"][b, :-(-n // case["page"])].long()
            k, v = s["k_cache"][pages].double(), s["v_cache"][pages].double()
            if case["fp8"]:
                k, v = k * s["k_scale"].double()[:, None, None], v * s["v_scale"].double()[:, None, None]
            k, v = (x.permute(1, 0, 2, 3).reshape(hk, -1, d)[:, :n] for x in (k, v))
            z = s["q"][b].double().view(hk, group, d) @ k.transpose(1, 2) * s["scale"]
            out[b] = (torch.softmax(z, dim=-1) @ v).view(hq, d)
        return out
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    at = 0
    for n in lens:
        for h in range(hk):
            q = s["q"][at:at + n, h * group:(h + 1) * group].double().transpose(0, 1)
            k, v = s["k"][at:at + n, h].double(), s["v"][at:at + n, h].double()
            z = (q @ k.t() * s["scale"]).masked_fill(torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1), -torch.inf)
            out[at:at + n, h * group:(h + 1) * group] = (torch.softmax(z, dim=-1) @ v).transpose(0, 1)
        at += n
    return out
