"""The MXFP4 operators on the GPU against the float64 oracle.

Codes with scales within a few powers of two of one have sums that FP32 holds exactly, whatever their order
(mxfp4_cases.exact_spread): those results are compared bit by bit.  Wider scales and the gated products are
compared within bounds that are made of the sums' magnitudes."""
import numpy as np
import pytest

import fp4_grouped_gemm_amd as fgg
from oracle import mxfp4 as om
from oracle.formats import bf16_bits_to_float, bf16_rne_bits
from tests.gpu_util import c_bits, c_to_f64, log
from tests.mxfp4_cases import (bf16, check_bf16, check_mxfp4, coded, exact_spread, gated_bound, routed,
                               sum_bound)

pytestmark = pytest.mark.gpu


def dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def dev16(bits):
    import torch
    return dev(np.ascontiguousarray(bits, np.uint16).view(np.int16)).view(torch.bfloat16)


def host(t):
    return t.cpu().numpy()


# ------------------------------------------------------------ quantisation
def every_value():
    """Blocks around every way a value can meet its block's scale: each finite BF16 below it, both signs."""
    rows = []
    for top in (0x0080, 0x0100, 0x0180, 0x0233, 0x3F80, 0x3FFF, 0x40C0, 0x7F00, 0x7F7F, 0x0003, 0x4000):
        low = np.arange(max(0, top - 1500), top + 1, dtype=np.uint16)
        low = np.concatenate([low, low | 0x8000, np.arange(0, top, 97, dtype=np.uint16)])
        low = np.resize(low, -(-len(low) // 31) * 31).reshape(-1, 31)
        rows.append(np.concatenate([low, np.full((len(low), 1), top, np.uint16)], 1))
    x = np.concatenate(rows)
    x = x[:len(x) // 4 * 4].reshape(-1, 128)
    special = np.zeros((8, 128), np.uint16)
    special[1, 5], special[1, 40], special[1, 70], special[1, 127] = 0x7F80, 0xFF80, 0x7FC1, 0xFFFF
    special[2, ::2] = 0x8000
    special[3, 64] = 1
    special[4] = 0x7F7F
    special[5] = np.arange(128)
    special[6] = bf16_rne_bits(np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 4], 16))
    special[7] = bf16_rne_bits(np.tile([-0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, 7.9], 16))
    return np.concatenate([special, x])


def test_quantize_every_value():
    bits = every_value()
    log(f"quantize_mxfp4 {bits.shape}")
    Q, S = fgg.quantize_mxfp4(dev16(bits))
    q, s = om.quantize(bf16_bits_to_float(bits))
    assert np.array_equal(host(S), s) and np.array_equal(host(Q), q)


@pytest.mark.parametrize("M,K", [(1, 128), (1, 4096), (3, 384), (77, 1152), (1000, 512), (5, 1 << 20), (70001, 128)])
def test_quantize(M, K):
    rng = np.random.default_rng(M + K)
    bits = bf16_rne_bits(rng.standard_normal((M, K), dtype=np.float32) * np.exp(3 * rng.standard_normal((1, K))))
    log(f"quantize_mxfp4 {M} {K}")
    Q, S = fgg.quantize_mxfp4(dev16(bits))
    q, s = om.quantize(bf16_bits_to_float(bits))
    assert np.array_equal(host(S), s) and np.array_equal(host(Q), q)
    x = om.dequantize(q, s)
    assert np.array_equal(c_to_f64(fgg.dequantize_mxfp4(Q, S)), x)


@pytest.mark.parametrize("T,R,K", [(1, 1, 128), (5, 3, 256), (9, 1000, 640), (300, 777, 1024)])
def test_quantize_rows(T, R, K):
    rng = np.random.default_rng(T + R)
    bits = bf16_rne_bits(rng.standard_normal((T, K)))
    rows = rng.integers(-2, T + 2, R).astype(np.int32)
    log(f"quantize_mxfp4 rows {T} {R} {K}")
    Q, S = fgg.quantize_mxfp4(dev16(bits), rows=dev(rows))
    real = (rows >= 0) & (rows < T)
    x = np.where(real[:, None], bf16_bits_to_float(bits)[np.where(real, rows, 0)], 0.0)
    q, s = om.quantize(x)
    assert np.array_equal(host(S), s) and np.array_equal(host(Q), q)


def test_dequantize_every_code():
    q = np.tile(np.arange(256, dtype=np.uint8), (256, 1))[:, :256]
    q = np.concatenate([q, q], 1)  # 16 blocks of 32 a row half: every byte under every scale
    s = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, 32))
    log("dequantize_mxfp4")
    X = c_bits(fgg.dequantize_mxfp4(dev(q), dev(s)))
    x = om.dequantize(q, s)
    want = bf16_rne_bits(x)
    nan = np.isnan(x)
    assert np.array_equal(X[~nan], want[~nan]) and np.isnan(bf16_bits_to_float(X[nan])).all()


# ---------------------------------------------------------------- products
SHAPES = [(1, 16, 128), (1, 4096, 4096), (2, 32, 256), (15, 48, 384), (16, 128, 512), (17, 144, 640), (33, 256, 1152),
          (64, 80, 2048), (100, 272, 896), (129, 512, 1024), (250, 384, 4096), (257, 336, 128), (513, 528, 1536), (1100, 144, 384),
          (2049, 784, 256)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_dense(M, N, K):
    rng = np.random.default_rng(M + N + K)
    A, sA = coded((M, K), rng, exact_spread(K))
    B, sB = coded((N, K), rng, exact_spread(K))
    log(f"mxfp4_gemm {M} {N} {K}")
    C = fgg.mxfp4_gemm(dev(A), dev(B), dev(sA), dev(sB))
    want, _ = om.gemm(A, B, sA, sB)
    assert np.array_equal(bf16_bits_to_float(c_bits(C)), bf16(want))


GROUPED = [(1, 32, 128, 3, "any"), (2, 64, 512, 8, "any"), (5, 144, 384, 1, "any"), (64, 256, 1024, 4, "any"), (130, 96, 640, 16, "any"),
           (130, 128, 640, 16, "none"), (40, 128, 256, 5, "one"), (300, 272, 512, 3, "runs"), (700, 528, 384, 4, "padded"),
           (1500, 48, 256, 2, "any"), (2300, 256, 1152, 7, "runs"), (1030, 16, 128, 70, "any"), (4097, 144, 256, 4, "padded"),
           (3000, 336, 128, 5, "one"), (260, 2064, 384, 2, "runs")]


@pytest.mark.parametrize("M,N,K,G,kind", GROUPED)
def test_grouped(M, N, K, G, kind):
    rng = np.random.default_rng(M + N + K + G)
    A, sA = coded((M, K), rng, exact_spread(K))
    B, sB = coded((G, N, K), rng, exact_spread(K))
    ids = routed(M, G, rng, kind)
    # what rows of padding hold reaches nothing
    sA[(ids < 0) | (ids >= G)] = 255
    log(f"grouped_mxfp4_gemm {M} {N} {K} {G} {kind}")
    C = fgg.grouped_mxfp4_gemm(dev(A), dev(B), dev(sA), dev(sB), dev(ids))
    sA[(ids < 0) | (ids >= G)] = 0
    want, _ = om.gemm(A, B, sA, sB, ids)
    assert np.array_equal(bf16_bits_to_float(c_bits(C)), bf16(want))


@pytest.mark.parametrize("M,N,K", [(1, 256, 4096), (20, 96, 1152), (300, 272, 2048)])
def test_scales_of_every_size(M, N, K):
    """Scales over the whole range at which results are BF16 numbers; blocks that vanish beside others."""
    rng = np.random.default_rng(M)
    A, sA = coded((M, K), rng, 60)
    B, sB = coded((N, K), rng, 55)
    log(f"mxfp4_gemm scales {M} {N} {K}")
    C = fgg.mxfp4_gemm(dev(A), dev(B), dev(sA), dev(sB))
    want, S = om.gemm(A, B, sA, sB)
    check_bf16(c_to_f64(C), want, sum_bound(S, K))


@pytest.mark.parametrize("M", [3, 400])
def test_small_and_large_scales(M):
    """Code 0 (2^-127) against a scale that brings the product back, and the other way round."""
    rng = np.random.default_rng(M)
    for a, b in ((0, 200), (1, 253), (0, 254), (254, 0), (120, 7)):
        A, sA = coded((M, 256), rng, 0)
        B, sB = coded((48, 256), rng, 0)
        sA[:], sB[:] = a, b
        log(f"mxfp4_gemm scales {a} {b}")
        C = fgg.mxfp4_gemm(dev(A), dev(B), dev(sA), dev(sB))
        want, _ = om.gemm(A, B, sA, sB)
        assert np.array_equal(bf16_bits_to_float(c_bits(C)), bf16(want))


@pytest.mark.parametrize("M", [2, 300])
def test_nan_scales(M):
    rng = np.random.default_rng(M)
    A, sA = coded((M, 512), rng, 1)
    B, sB = coded((3, 64, 512), rng, 1)
    ids = routed(M, 3, rng, "any")
    ids[0] = 1
    sA[0, 5] = 255
    sB[2, 7, 15] = 255
    sB[2, 33, 0] = 255
    log("grouped_mxfp4_gemm NaN")
    C = c_to_f64(fgg.grouped_mxfp4_gemm(dev(A), dev(B), dev(sA), dev(sB), dev(ids)))
    want, _ = om.gemm(A, B, sA, sB, ids)
    nan = np.zeros(C.shape, bool)
    nan[0] = True
    for n in (7, 33):
        nan[ids == 2, n] = True
    assert np.array_equal(np.isnan(C), nan) and np.array_equal(C[~nan], bf16(want[~nan]))


# ------------------------------------------------------------------- gated
GATED = [(1, 32, 128, 1, "dense"), (1, 2048, 4096, 1, "dense"), (37, 96, 640, 1, "dense"), (300, 416, 512, 1, "dense"), (2, 256, 1024, 8, "any"),
         (70, 64, 384, 5, "any"), (200, 32, 256, 16, "none"), (600, 160, 1152, 3, "runs"), (1300, 224, 384, 4, "padded"), (2100, 288, 128, 2, "any")]


def gated_case(M, F, K, G, kind):
    rng = np.random.default_rng(M + F + K + G)
    A, sA = coded((M, K), rng, 1)
    B, sB = coded((G, 2 * F, K), rng, 1)
    # sums of a few units: what silu bends
    sB = (sB - int(np.log2(10 * K ** 0.5)) + 1).astype(np.uint8)
    ids = None if kind == "dense" else routed(M, G, rng, kind)
    if ids is None:
        B, sB = B[0], sB[0]
    return A, sA, B, sB, ids


def call_gated(A, sA, B, sB, ids, **kw):
    if ids is None:
        return fgg.mxfp4_gated_gemm(dev(A), dev(B), dev(sA), dev(sB), **kw)
    return fgg.grouped_mxfp4_gated_gemm(dev(A), dev(B), dev(sA), dev(sB), dev(ids), **kw)


@pytest.mark.parametrize("M,F,K,G,kind", GATED + [(5, 16, 128, 1, "dense"), (90, 80, 256, 3, "any"), (700, 176, 256, 2, "runs")])
def test_gated(M, F, K, G, kind):
    case = gated_case(M, F, K, G, kind)
    log(f"gated {M} {F} {K} {G} {kind}")
    C = c_to_f64(call_gated(*case))
    A, sA, B, sB, ids = case
    z, halves, S = om.gated(A, B, sA, sB, ids)
    check_bf16(C, z, gated_bound(z, halves, S, K))


@pytest.mark.parametrize("M,F,K,G,kind", GATED)
def test_gated_quantized(M, F, K, G, kind):
    case = gated_case(M, F, K, G, kind)
    log(f"gated quantized {M} {F} {K} {G} {kind}")
    Q, S = call_gated(*case, quantize=True)
    A, sA, B, sB, ids = case
    z, halves, mags = om.gated(A, B, sA, sB, ids)
    check_mxfp4(host(Q), host(S), z, gated_bound(z, halves, mags, K))
    if ids is not None:
        nobody = (ids < 0) | (ids >= G)
        assert not host(Q)[nobody].any() and not host(S)[nobody].any()


@pytest.mark.parametrize("M", [1, 260])
def test_gated_values_that_are_not_finite(M):
    """NaN scales, gates of large magnitude either way, results past BF16."""
    rng = np.random.default_rng(M)
    A, sA = coded((M, 256), rng, 0)
    B, sB = coded((128, 256), rng, 0)
    sB[3] = 255             # a gate
    sB[64 + 40] = 255       # an up
    sB[10], sB[11] = 140, 190   # gates of 2^17, and of 2^67
    sB[64 + 11] = 190       # products of 2^134
    log("gated not finite")
    C = c_to_f64(fgg.mxfp4_gated_gemm(dev(A), dev(B), dev(sA), dev(sB)))
    z, _, _ = om.gated(A, B, sA, sB)
    nan = np.isnan(z)
    assert np.array_equal(np.isnan(C), nan) and nan[:, [3, 40]].all()
    big = np.abs(z) > 2.0 ** 128
    assert big.any() and np.array_equal(C[big], np.sign(z[big]) * np.inf)
    zero = ~nan & (np.abs(z) < 1e-30)
    assert (np.abs(C[zero]) < 2e-30).all()
    Q, S = fgg.mxfp4_gated_gemm(dev(A), dev(B), dev(sA), dev(sB), quantize=True)
    assert (host(S) == 255).all() and not host(Q).any()


# ------------------------------------------------------------------ calls
def test_chain():
    """A feed-forward block as it is used: norm, expansion to the experts' rows, both products, on a stream of
    its own and replayed from a graph with other inputs."""
    import torch
    from tests.test_gpu_norm import norm_bound
    T, H, F, G, top = 37, 256, 384, 4, 2
    rng = np.random.default_rng(7)
    x, r = (bf16(rng.standard_normal((T, H))) for _ in range(2))
    w = bf16(1 + 0.1 * rng.standard_normal(H))
    order = rng.permutation(T * top)
    ids = np.sort(rng.integers(0, G, T * top)).astype(np.int32)
    rows = (order // top).astype(np.int32)
    W1, W2 = rng.standard_normal((G * 2 * F, H)) * H ** -0.5, rng.standard_normal((G * H, F)) * F ** -0.5
    (B1, s1), (B2, s2) = (om.quantize(bf16(W)) for W in (W1, W2))
    B1, s1, B2, s2 = B1.reshape(G, 2 * F, -1), s1.reshape(G, 2 * F, -1), B2.reshape(G, H, -1), s2.reshape(G, H, -1)
    d = [dev16(bf16_rne_bits(v)) for v in (x, r, w)] + [dev(v) for v in (rows, ids, B1, s1, B2, s2)]

    def block(x, r, w, rows, ids, B1, s1, B2, s2):
        y, h = fgg.residual_norm(x, r, w)
        q, s = fgg.quantize_mxfp4(y, rows=rows)
        q2, t2 = fgg.grouped_mxfp4_gated_gemm(q, B1, s, s1, ids, quantize=True)
        return y, h, q, s, q2, t2, fgg.grouped_mxfp4_gemm(q2, B2, t2, s2, ids)

    def check(out, x, r, w):
        """Each step against the oracle on what the step before gave."""
        y, h, q, s, q2, t2, z = out
        wy, wh = om.norm(x, r, w)
        check_bf16(c_to_f64(h), wh, 2.0 ** -22 * (np.abs(x) + np.abs(r)))
        check_bf16(c_to_f64(y), wy, norm_bound(x, r, w, wy, wh))
        eq, es = om.quantize(c_to_f64(y)[rows])
        assert np.array_equal(host(q), eq) and np.array_equal(host(s), es)
        v, halves, mags = om.gated(eq, B1, es, s1, ids)
        check_mxfp4(host(q2), host(t2), v, gated_bound(v, halves, mags, H))
        want, mag = om.gemm(host(q2), B2, host(t2), s2, ids)
        check_bf16(c_to_f64(z), want, sum_bound(mag, F))

    log("chain")
    check(block(*d), x, r, w)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        out = block(*d)
    stream.synchronize()
    check(out, x, r, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(*d)
    for seed in range(3):
        x, r = (bf16(rng.standard_normal((T, H)) * (seed + 1)) for _ in range(2))
        d[0].copy_(dev16(bf16_rne_bits(x)))
        d[1].copy_(dev16(bf16_rne_bits(r)))
        graph.replay()
        torch.cuda.synchronize()
        check(out, x, r, w)


def test_stream_argument():
    import torch
    rng = np.random.default_rng(1)
    A, sA = coded((50, 512), rng, 1)
    B, sB = coded((96, 512), rng, 1)
    stream = torch.cuda.Stream()
    args = [dev(v) for v in (A, B, sA, sB)]
    bits = bf16_rne_bits(rng.standard_normal((50, 512)))
    x = dev16(bits)
    torch.cuda.synchronize()
    C = fgg.mxfp4_gemm(*args, stream=stream)
    D = fgg.mxfp4_gated_gemm(*args, stream=stream)
    Q, S = fgg.quantize_mxfp4(x, stream=stream)
    X = fgg.dequantize_mxfp4(Q, S, stream=stream)
    y, h = fgg.residual_norm(x, None, x[0].clone(), stream=stream)
    stream.synchronize()
    want, _ = om.gemm(A, B, sA, sB)
    assert np.array_equal(c_to_f64(C), bf16(want))
    z, halves, mags = om.gated(A, B, sA, sB)
    check_bf16(c_to_f64(D), z, gated_bound(z, halves, mags, 512))
    q, s = om.quantize(bf16_bits_to_float(bits))
    assert np.array_equal(host(Q), q) and np.array_equal(c_to_f64(X), om.dequantize(q, s))
    assert np.array_equal(c_to_f64(h), bf16_bits_to_float(bits))


def test_out_and_types():
    import torch
    rng = np.random.default_rng(2)
    A, sA = coded((50, 512), rng, 1)
    B, sB = coded((96, 512), rng, 1)
    a, b, u, v = (dev(x) for x in (A, B, sA, sB))
    out = torch.full((50, 96), float("nan"), dtype=torch.bfloat16, device="cuda")
    want, _ = om.gemm(A, B, sA, sB)
    assert fgg.mxfp4_gemm(a, b, u, v, out) is out and np.array_equal(c_to_f64(out), bf16(want))
    C = fgg.mxfp4_gemm(a.view(torch.float4_e2m1fn_x2), b.view(torch.int8), u.view(torch.float8_e8m0fnu), v)
    assert np.array_equal(c_to_f64(C), bf16(want))
    # slices of larger tensors, as long as they are whole rows
    big = torch.zeros((60, 256), dtype=torch.uint8, device="cuda")
    big[3:53] = a
    assert np.array_equal(c_to_f64(fgg.mxfp4_gemm(big[3:53], b, u, v)), bf16(want))


def test_results_do_not_depend_on_timing():
    rng = np.random.default_rng(3)
    A, sA = coded((300, 4096), rng, 20)
    B, sB = coded((2, 160, 4096), rng, 20)
    ids = routed(300, 2, rng, "any")
    args = [dev(v) for v in (A, B, sA, sB, ids)]
    first = c_bits(fgg.grouped_mxfp4_gemm(*args))
    for _ in range(5):
        assert np.array_equal(c_bits(fgg.grouped_mxfp4_gemm(*args)), first)


def test_nothing_to_do():
    import torch
    e = lambda *shape, d=torch.uint8: torch.empty(shape, dtype=d, device="cuda")  # noqa: E731
    Q, S = fgg.quantize_mxfp4(e(0, 256, d=torch.bfloat16))
    assert Q.shape == (0, 128) and S.shape == (0, 8)
    assert fgg.quantize_mxfp4(e(3, 256, d=torch.bfloat16), rows=e(0, d=torch.int32))[0].shape == (0, 128)
    assert fgg.dequantize_mxfp4(Q, S).shape == (0, 256)
    b, sb = e(64, 128), e(64, 8)
    assert fgg.mxfp4_gemm(Q, b, S, sb).shape == (0, 64)
    C, s = fgg.grouped_mxfp4_gated_gemm(Q, b[None], S, sb[None], e(0, d=torch.int32), quantize=True)
    assert C.shape == (0, 16) and s.shape == (0, 1)


def test_refusals():
    import torch
    a, s, b, sb = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for shape in ((4, 128), (4, 8), (64, 128), (64, 8)))
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    bad = [
        (fgg.quantize_mxfp4, (x.float(),), {}), (fgg.quantize_mxfp4, (x.t(),), {}), (fgg.quantize_mxfp4, (x[:, :144].contiguous(),), {}),
        (fgg.quantize_mxfp4, (x,), dict(rows=ids.long())), (fgg.quantize_mxfp4, (x[:0],), dict(rows=ids)),
        (fgg.dequantize_mxfp4, (a, s[:, :4].contiguous()), {}), (fgg.dequantize_mxfp4, (a.float(), s), {}),
        (fgg.mxfp4_gemm, (a, b, s, sb[:32]), {}), (fgg.mxfp4_gemm, (a, b[:, :64].contiguous(), s, sb[:, :4].contiguous()), {}),
        (fgg.mxfp4_gemm, (a, b[:40], s, sb[:40]), {}), (fgg.mxfp4_gemm, (a, b, s.float(), sb), {}), (fgg.mxfp4_gemm, (a, b[None], s, sb[None]), {}),
        (fgg.mxfp4_gemm, (a, b, s, sb, x), {}), (fgg.mxfp4_gemm, (a[:, ::2], b, s, sb), {}), (fgg.mxfp4_gemm, (a.cpu(), b, s, sb), {}),
        (fgg.grouped_mxfp4_gemm, (a, b[None], s, sb[None], ids[:3]), {}), (fgg.grouped_mxfp4_gemm, (a, b[None], s, sb[None], ids.long()), {}),
        (fgg.grouped_mxfp4_gemm, (a, b[:0][None], s, sb[:0][None], ids), {}), (fgg.grouped_mxfp4_gemm, (a, b[None], s, sb[None], None), {}),
        (fgg.mxfp4_gated_gemm, (a, b[:33], s, sb[:33]), {}), (fgg.mxfp4_gated_gemm, (a, b[:32], s, sb[:32]), dict(quantize=True)),
        (fgg.mxfp4_gated_gemm, (a, b, s, sb, x), dict(quantize=True)),
    ]
    for f, args, kw in bad:
        with pytest.raises(ValueError):
            f(*args, **kw)
