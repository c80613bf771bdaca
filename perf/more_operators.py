"""Cases of the MXFP4 operators: quantisation of activations to microscaled 4-bit values (op
"quantise"), their products with MXFP4 weights (op "product"), the gated feed-forward product (op
"gated") and the norms, gate and residual sum at a block's border (op "norm").

MXFP4: E2M1 codes, and for each 32 of them along a row one power of two (E8M0, code - 127).  A block's
scale is 2 ** (floor(log2(largest magnitude)) - 2), at least 2 ** -127; codes round to nearest, ties to
even, and saturate at 6.

Each case is a call as a serving loop of a mixture-of-experts layer makes it.  `run` computes it
with elementary torch operations in FP32 (own = False) or by the library's entry points (own =
True); `exact` computes it in FP64, expert by expert.

Keys of a case: op; and
  quantise: tokens, width; top > 0: the rows are the tokens' copies for `top` of `experts` experts, in
            their order, runs padded to a multiple of `pad` rows (0: the tokens as they are)
  product:  tokens x top rows, each for one of `experts` experts (1: no routing) of unequal load (skew),
            in runs padded to a multiple of `pad` rows, or unsorted (pad = 0); n, k: the weights' shape
  gated:    rows as for product; inner (columns of gate, and of up), k; down: the result goes on in
            MXFP4 through the second product, to k columns
  norm:     tokens, width; post (a norm of the block's output before the sum), gate ("", "channel" or
            "token"); project > 0: the result goes on in MXFP4 through a product with that many columns
"""
import math

import torch

own = False

BLOCK = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6
SCALE = 0.5


# ------------------------------------------------------------------ cases
def listed():
    dense = dict(experts=1, top=1, skew=0.0, pad=0)
    return [
        # one user's next token before a projection: all latency
        dict(op="quantise", name="quantise one token", tokens=1, width=4096, experts=1, top=0, skew=0.0, pad=0),
        # a prompt batch expanded to its experts' rows, padded as the products like it
        dict(op="quantise", name="quantise expanded", tokens=4001, width=7168, experts=32, top=2, skew=0.6, pad=128),
        # one user's next token through a projection
        dict(op="product", name="product one token", tokens=1, n=4096, k=4096, **dense),
        # a decode batch over large experts, rows as the router leaves them
        dict(op="product", name="product decode", tokens=64, top=2, experts=8, skew=0.3, pad=0, n=8192, k=8192),
        # prompts over many experts of very unequal load
        dict(op="product", name="product experts", tokens=6111, top=2, experts=32, skew=1.0, pad=128, n=2048, k=7168),
        # a wide dense layer over a prompt batch
        dict(op="product", name="product dense", tokens=2048, n=36864, k=4608, **dense),
        # one user's next token through two experts' gate and up projections
        dict(op="gated", name="gated one token", tokens=1, top=2, experts=8, skew=0.0, pad=0, inner=2048, k=4096, down=False),
        # a decode batch through whole feed-forward blocks of small experts
        dict(op="gated", name="feed forward decode", tokens=48, top=4, experts=64, skew=0.5, pad=0, inner=1024, k=2048, down=True),
        # prompts through whole feed-forward blocks, runs as they fall
        dict(op="gated", name="feed forward prompts", tokens=2777, top=2, experts=8, skew=0.4, pad=1, inner=2048, k=7168, down=True),
        # one user's next token between two blocks
        dict(op="norm", name="norm one token", tokens=1, width=4096, post=False, gate="", project=0),
        # a prompt batch between two blocks, normed on both sides and gated
        dict(op="norm", name="norm prompts", tokens=8192, width=7168, post=True, gate="channel", project=0),
        # a prompt between two blocks, and on into the queries', keys' and values' projection
        dict(op="norm", name="norm and projection", tokens=777, width=4096, post=False, gate="", project=6144),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quantise", "product", "product", "gated", "gated", "norm"])
    if op == "norm":
        width = 128 * spread(2, 64)
        c = dict(op=op, tokens=spread(1, min(16384, 50000000 // width)), width=width, post=rng.random() < 0.5,
                 gate=rng.choice(["", "channel", "token"]), project=0)
        if rng.random() < 0.4:
            c.update(project=16 * spread(4, 512), tokens=min(c["tokens"], 4096))
        return c
    experts = rng.choice([1, 4, 8, 16, 32, 64])
    c = dict(op=op, experts=experts, top=1 if experts == 1 else rng.choice([1, 2, 4]), skew=rng.choice([0.0, 0.3, 0.6, 1.0]))
    if op == "quantise":
        width = 128 * spread(1, 64)
        c.update(width=width, tokens=spread(1, min(16384, 20000000 // width)), top=rng.choice([0, c["top"]]), pad=rng.choice([1, 16, 128]))
        return c
    c.update(tokens=spread(1, 3000), k=128 * spread(1, 56))
    few = c["tokens"] * c["top"] <= 256
    c.update(pad=0 if few or experts == 1 else rng.choice([1, 16, 128]))
    # the weights of all experts stay within those of the largest listed case
    room = 500000000 // (experts * c["k"])
    if op == "product":
        c.update(n=16 * spread(1, max(2, min(512, room // 16))))
    else:
        c.update(inner=128 * spread(1, max(2, min(32, room // 384))), down=rng.random() < 0.5)
    return c


def loads(case):
    """Rows of each expert: the copies of the tokens shared out by (rank + 1) ** -skew, the experts in an order that mixes them."""
    rows, g = case["tokens"] * case["top"], case["experts"]
    share = [(i + 1) ** -case["skew"] for i in range(g)]
    ends = [round(rows * sum(share[:i]) / sum(share)) for i in range(g + 1)]
    got = [b - a for a, b in zip(ends, ends[1:])]
    step = next(s for s in range(max(1, int(g * 0.618)), g + 1) if math.gcd(s, g) == 1)
    return [got[i * step % g] for i in range(g)]


def routing(case):
    """Expert of each row, -1 for padding: runs in the experts' order, each padded to a multiple of `pad` rows."""
    ids = []
    for e, n in enumerate(loads(case)):
        ids += [e] * n + [-1] * (-n % max(1, case["pad"]))
    return ids


def packed(n):
    """Bytes of n values in MXFP4."""
    return n // 2 + n // BLOCK


def work(case):
    op = case["op"]
    if op == "norm":
        t, w = case["tokens"], case["width"]
        gate = {"": 0, "channel": w, "token": t * w}[case["gate"]]
        got = {"bytes": 2 * (3 * t * w + w * (2 if case["post"] else 1) + gate), "flops": t * w * (14 if case["post"] else 8)}
        if case["project"]:
            got["bytes"] += packed(t * w) * 2 + packed(case["project"] * w) + 2 * t * case["project"]
            got["flops"] += 2 * t * w * case["project"]
        else:
            got["bytes"] += 2 * t * w
        return got
    if op == "quantise":
        rows = len(routing(case)) if case["top"] else case["tokens"]
        n = rows * case["width"]
        return {"bytes": 2 * case["tokens"] * case["width"] + (4 * rows if case["top"] else 0) + 2 * packed(n) + 2 * n, "flops": 3 * n}
    rows, k = len(routing(case)), case["k"]
    real, used = case["tokens"] * case["top"], sum(n > 0 for n in loads(case))
    ids = 4 * rows if case["experts"] > 1 else 0
    if op == "product":
        return {"bytes": ids + packed(rows * k) + used * packed(case["n"] * k) + 2 * rows * case["n"], "flops": 2 * real * case["n"] * k}
    f = case["inner"]
    got = {"bytes": ids + packed(rows * k) + used * packed(2 * f * k), "flops": 4 * real * f * k}
    if case["down"]:
        got["bytes"] += 2 * packed(rows * f) + ids + used * packed(f * k) + 2 * rows * k
        got["flops"] += 2 * real * f * k
    else:
        got["bytes"] += 2 * rows * f
    return got


# ----------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def activations(rows, width):
        """Values of a few units, with channels that are larger than others."""
        x = torch.randn((rows, width), generator=g, device=dev)
        return (x * torch.exp(0.7 * torch.randn((width,), generator=g, device=dev))).to(torch.bfloat16)

    def weights(experts, n, k):
        """MXFP4 weights [experts, n, k] whose products with values of one unit are of one unit."""
        w = torch.randn((experts * n, k), generator=g, device=dev, dtype=torch.bfloat16) * k ** -0.5
        codes, scales = quantised(w)
        return codes.view(experts, n, k // 2), scales.view(experts, n, k // BLOCK)

    s = {"case": case}
    op = case["op"]
    if op == "norm":
        t, w = case["tokens"], case["width"]
        s["x"], s["residual"] = activations(t, w), 4 * activations(t, w)
        s["weight"] = (1 + 0.2 * torch.randn((w,), generator=g, device=dev)).to(torch.bfloat16)
        s["post"] = (1 + 0.2 * torch.randn((w,), generator=g, device=dev)).to(torch.bfloat16) if case["post"] else None
        shape = {"": None, "channel": (w,), "token": (t, w)}[case["gate"]]
        s["gate"] = None if shape is None else torch.rand(shape, generator=g, device=dev).to(torch.bfloat16)
        if case["project"]:
            s["b"], s["b_scale"] = (x[0] for x in weights(1, case["project"], w))
        return s
    if op == "quantise":
        s["x"], s["rows"] = activations(case["tokens"], case["width"]), None
        if case["top"]:
            ids = torch.tensor(routing(case), device=dev)
            copies = torch.randperm(case["tokens"] * case["top"], generator=g, device=dev) // case["top"]
            s["rows"] = torch.full_like(ids, -1)
            s["rows"][ids >= 0] = copies
            s["rows"] = s["rows"].int()
        return s
    ids = torch.tensor(routing(case), dtype=torch.int32, device=dev)
    if case["pad"] == 0:
        ids = ids[torch.randperm(len(ids), generator=g, device=dev)].contiguous()
    s["ids"] = ids if case["experts"] > 1 else None
    # the rows of each expert, which a program without grouped products sorts out beforehand
    s["mine"] = [(ids == e).nonzero()[:, 0] for e in range(case["experts"])]
    s["a"], s["a_scale"] = quantised(activations(len(ids), case["k"]))
    if op == "product":
        s["b"], s["b_scale"] = weights(case["experts"], case["n"], case["k"])
    else:
        s["b"], s["b_scale"] = weights(case["experts"], 2 * case["inner"], case["k"])
        if case["down"]:
            s["b2"], s["b2_scale"] = weights(case["experts"], case["k"], case["inner"])
    return s


# -------------------------------------------------------------- operators
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"quantise": plain_quantise, "product": plain_product, "gated": plain_gated, "norm": plain_norm}[op](s)
    import fp4_grouped_gemm_amd as fgg
    if op == "quantise":
        return fgg.dequantize_mxfp4(*fgg.quantize_mxfp4(s["x"], rows=s["rows"]))
    if op == "norm":
        y, h = fgg.residual_norm(s["x"], s["residual"], s["weight"], post_weight=s["post"], gate=s["gate"],
                                 scale=SCALE, eps=EPS, quantize=case["project"] > 0)
        if case["project"]:
            y = fgg.mxfp4_gemm(y[0], s["b"], y[1], s["b_scale"])
        return {"y": y, "h": h}
    if op == "product":
        if s["ids"] is None:
            return fgg.mxfp4_gemm(s["a"], s["b"][0], s["a_scale"], s["b_scale"][0])
        return fgg.grouped_mxfp4_gemm(s["a"], s["b"], s["a_scale"], s["b_scale"], s["ids"])
    if s["ids"] is None:
        y = fgg.mxfp4_gated_gemm(s["a"], s["b"][0], s["a_scale"], s["b_scale"][0], quantize=case["down"])
        return fgg.mxfp4_gemm(y[0], s["b2"][0], y[1], s["b2_scale"][0]) if case["down"] else y
    y = fgg.grouped_mxfp4_gated_gemm(s["a"], s["b"], s["a_scale"], s["b_scale"], s["ids"], quantize=case["down"])
    return fgg.grouped_mxfp4_gemm(y[0], s["b2"], y[1], s["b2_scale"], s["ids"]) if case["down"] else y


def powers(codes):
    """FP32 2 ** (code - 127) of E8M0 codes 0 .. 254."""
    codes = codes.int()
    return torch.where(codes == 0, 1 << 22, codes << 23).view(torch.float32)


def rounded(x):
    """MXFP4 magnitudes and scales of FP32 x [rows, width]: E2M1 codes with their sign, E8M0 codes."""
    x = x.view(x.shape[0], -1, BLOCK)
    top = x.abs().amax(-1, keepdim=True)
    code = ((top.view(torch.int32) >> 23) - 2).clamp(min=0)
    a = x.abs() / powers(code)
    c = (a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    return (c + 8 * torch.signbit(x).byte()).flatten(1), code[..., 0].byte()


def quantised(x):
    """The codes two a byte, the first in the low half, and the scales."""
    codes, scales = rounded(x.float())
    return codes[:, 0::2] + 16 * codes[:, 1::2], scales


def values(codes, scales):
    """FP32 values of E2M1 codes [..., rows, width] and their scales."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    return (table[codes.int()].unflatten(-1, (-1, BLOCK)) * powers(scales)[..., None]).flatten(-2)


def unpacked(codes, scales):
    return values(torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2), scales)


def plain_quantise(s):
    x = s["x"].float()
    if s["rows"] is not None:
        rows = s["rows"].long()
        x = torch.where((rows >= 0)[:, None], x[rows.clamp(min=0)], 0.0)
    return values(*rounded(x)).to(torch.bfloat16)


def routed(a, b, b_scale, mine):
    """FP32 products of the rows of a with their experts' weights; zeros in rows without one."""
    y = torch.zeros((a.shape[0], b.shape[1]), device=a.device)
    for e, rows in enumerate(mine):
        if len(rows):
            y[rows] = a[rows] @ unpacked(b[e], b_scale[e]).t()
    return y


def plain_product(s):
    return routed(unpacked(s["a"], s["a_scale"]), s["b"], s["b_scale"], s["mine"]).to(torch.bfloat16)


def plain_gated(s):
    y = routed(unpacked(s["a"], s["a_scale"]), s["b"], s["b_scale"], s["mine"])
    gate, up = y.chunk(2, dim=1)
    y = gate / (1 + torch.exp(-gate)) * up
    if s["case"]["down"]:
        y = routed(values(*rounded(y)), s["b2"], s["b2_scale"], s["mine"])
    return y.to(torch.bfloat16)


def normed(x, weight):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()


def plain_norm(s):
    x = s["x"].float()
    if s["post"] is not None:
        x = normed(x, s["post"])
    if s["gate"] is not None:
        x = x * s["gate"].float()
    h = s["residual"].float() + SCALE * x
    y = normed(h, s["weight"])
    if s["case"]["project"]:
        y = values(*rounded(y)) @ unpacked(s["b"], s["b_scale"]).t()
    return {"y": y.to(torch.bfloat16), "h": h.to(torch.bfloat16)}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The same in FP64, one expert at a time."""
    s = prepare(case, seed)

    def decoded(codes, scales):
        c = codes.long()
        c = torch.stack([c % 16, c // 16], dim=2).reshape(c.shape[0], -1)
        e, m = c // 2 % 4, (c % 2).double()
        v = torch.where(e == 0, m * 0.5, (1 + m * 0.5) * 2.0 ** (e - 1).double())
        v = torch.where(c >= 8, -v, v)
        return v * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, dim=1)

    def mx(x):
        """x [rows, width] rounded to MXFP4."""
        y = x.reshape(-1, BLOCK)
        top = y.abs().max(dim=1, keepdim=True).values
        step = torch.exp2((torch.frexp(top).exponent.double() - 3).clamp(min=-127))
        step = torch.where(top == 0, 2.0 ** -127, step)
        table = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
        a = y.abs() / step
        hi = torch.searchsorted(table, a).clamp(max=7)
        lo = (hi - 1).clamp(min=0)
        d = (table[hi] - a) - (a - table[lo])
        up = (d < 0) | ((d == 0) & (hi % 2 == 0))
        return (torch.where(up, table[hi], table[lo]) * torch.sign(y) * step).reshape(x.shape)

    def product(a, b, b_scale):
        out = torch.zeros((a.shape[0], b.shape[1]), dtype=torch.float64, device=a.device)
        for e in range(case["experts"]):
            rows = s["mine"][e]
            if len(rows):
                out[rows] = torch.mm(a[rows], decoded(b[e], b_scale[e]).t())
        return out

    op = case["op"]
    if op == "quantise":
        x = s["x"].double()
        if s["rows"] is not None:
            y = torch.zeros((len(s["rows"]), x.shape[1]), dtype=torch.float64, device=x.device)
            real = s["rows"] >= 0
            y[real] = x[s["rows"][real].long()]
            x = y
        return mx(x)
    if op == "norm":
        x, h = s["x"].double(), s["residual"].double()
        if s["post"] is not None:
            x = x / (x.pow(2).sum(1, keepdim=True) / x.shape[1] + EPS).sqrt() * s["post"].double()
        h = h + x * (1.0 if s["gate"] is None else s["gate"].double()) * SCALE
        y = h / (h.pow(2).sum(1, keepdim=True) / h.shape[1] + EPS).sqrt() * s["weight"].double()
        if case["project"]:
            y = torch.mm(mx(y), decoded(s["b"], s["b_scale"]).t())
        return {"y": y, "h": h}
    y = product(decoded(s["a"], s["a_scale"]), s["b"], s["b_scale"])
    if op == "gated":
        f = case["inner"]
        y = y[:, :f] * torch.sigmoid(y[:, :f]) * y[:, f:]
        if case["down"]:
            y = product(mx(y), s["b2"], s["b2_scale"])
    return y
