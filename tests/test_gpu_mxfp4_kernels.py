"""The MXFP4 products where what runs them changes: few rows and many, rows of few of many experts, more tiles
than the card takes at once, the edges of steps, tiles and windows.  Codes whose sums FP32 holds exactly, compared
bit by bit with the float64 oracle."""
import numpy as np
import pytest

import fp4_grouped_gemm_amd as fgg
from oracle import mxfp4 as om
from oracle.formats import bf16_bits_to_float
from tests.gpu_util import c_bits, c_to_f64, log
from tests.mxfp4_cases import bf16, check_bf16, check_mxfp4, coded, exact_spread, gated_bound, routed, sum_bound
from tests.test_gpu_mxfp4 import call_gated, dev, gated_case, host

pytestmark = pytest.mark.gpu


def compare(M, N, K, G, ids, rng):
    A, sA = coded((M, K), rng, exact_spread(K))
    B, sB = coded((G, N, K), rng, exact_spread(K))
    if ids is None:
        C = fgg.mxfp4_gemm(dev(A), dev(B[0]), dev(sA), dev(sB[0]))
        want, _ = om.gemm(A, B[0], sA, sB[0])
    else:
        sA[(ids < 0) | (ids >= G)] = 255  # what rows of padding hold reaches nothing
        C = fgg.grouped_mxfp4_gemm(dev(A), dev(B), dev(sA), dev(sB), dev(ids))
        sA[(ids < 0) | (ids >= G)] = 0
        want, _ = om.gemm(A, B, sA, sB, ids)
    assert np.array_equal(bf16_bits_to_float(c_bits(C)), bf16(want))


# rows about the chunks of 16 and 32, K of one to many steps and odd multiples of 128, columns of a part of a
# workgroup, of many; the last where few rows end and many begin
DENSE = [(16, 16, 128), (17, 8192, 128), (31, 64, 256), (32, 8208, 384), (33, 48, 1408), (48, 16400, 256), (49, 16400, 256), (64, 4096, 640),
         (97, 1040, 3456), (127, 8192, 256), (128, 8192, 256), (128, 8208, 256), (129, 8192, 384), (129, 32, 1152), (255, 16400, 128), (256, 33280, 128),
         (257, 33280, 128), (385, 176, 2176), (2048, 4096, 128), (2049, 4112, 384), (2100, 8704, 128), (1537, 16656, 256), (4100, 8208, 128)]


@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense(M, N, K):
    log(f"mxfp4_gemm {M} {N} {K}")
    compare(M, N, K, 1, None, np.random.default_rng(M + N + K))


# fewer rows than experts, a wave's lanes full and one more; more than a scan of m_indices; windows of many
# experts and of one; more tiles than workgroups
GROUPED = [(1, 48, 256, 300, "any"), (3, 4096, 384, 8, "any"), (63, 272, 128, 64, "any"), (64, 80, 640, 65, "any"), (64, 80, 640, 64, "any"),
           (65, 80, 640, 66, "any"), (40, 64, 256, 50, "one"), (40, 64, 256, 50, "none"), (1024, 48, 256, 40, "any"), (1025, 48, 384, 40, "runs"),
           (2300, 32, 128, 64, "one"), (96, 4112, 256, 2, "any"), (97, 4112, 256, 2, "any"), (1500, 8208, 128, 7, "runs"), (1500, 528, 384, 12, "any"),
           (2048, 2064, 256, 3, "padded"), (4100, 2064, 384, 3, "runs"), (4100, 2064, 128, 5, "any"), (2600, 8208, 128, 4, "runs"), (2304, 4112, 128, 2, "none"),
           (3000, 3856, 128, 2, "one")]


@pytest.mark.parametrize("M,N,K,G,kind", GROUPED)
def test_grouped(M, N, K, G, kind):
    rng = np.random.default_rng(M + N + K + G)
    log(f"grouped_mxfp4_gemm {M} {N} {K} {G} {kind}")
    compare(M, N, K, G, routed(M, G, rng, kind), rng)


def test_windows_of_padding():
    """Runs that end within windows, whole windows of padding between them, unequal loads."""
    rng = np.random.default_rng(3)
    for M, N, loads in ((2400, 4112, {3: 700, 0: 5, 1: 512}), (1300, 80, {0: 1, 2: 300, 3: 257})):
        ids = np.full(M, -1, np.int32)
        at = 130
        for e, n in loads.items():
            ids[at:at + n] = e
            at += n + 260
        log(f"windows of padding {M} {N}")
        compare(M, N, 384, 4, ids, rng)


GATED = [(17, 4096, 128, 1, "dense"), (33, 48, 1408, 1, "dense"), (128, 4128, 128, 1, "dense"), (129, 160, 640, 1, "dense"), (1100, 8224, 128, 1, "dense"),
         (2049, 2080, 256, 1, "dense"), (5, 96, 384, 40, "any"), (64, 2080, 128, 65, "any"), (1030, 32, 256, 30, "runs"), (500, 96, 384, 5, "any"),
         (1500, 4128, 128, 7, "runs"), (2600, 2080, 256, 3, "runs"), (2304, 2080, 128, 2, "one")]


@pytest.mark.parametrize("M,F,K,G,kind,quantize", [c + (q,) for c in GATED for q in (False, True) if not q or c[1] % 32 == 0])
def test_gated(M, F, K, G, kind, quantize):
    case = gated_case(M, F, K, G, kind)
    log(f"gated {M} {F} {K} {G} {kind} {quantize}")
    out = call_gated(*case, quantize=quantize)
    A, sA, B, sB, ids = case
    z, halves, S = om.gated(A, B, sA, sB, ids)
    if quantize:
        check_mxfp4(host(out[0]), host(out[1]), z, gated_bound(z, halves, S, K))
    else:
        check_bf16(c_to_f64(out), z, gated_bound(z, halves, S, K))


def random_codes(shape, spread):
    import torch
    q = torch.randint(0, 256, shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8, device="cuda")
    return q, torch.randint(127 - spread, 128 + spread, shape[:-1] + (shape[-1] // 32,), dtype=torch.uint8, device="cuda")


def picked(C, A, B, sA, sB, rows, cols, e=None):
    """The oracle's product of some rows and columns against C's."""
    import torch
    r, n = torch.tensor(rows, device="cuda"), torch.tensor(cols, device="cuda")
    want, _ = om.gemm(*(host(v) for v in (A[r], (B if e is None else B[e])[n], sA[r], (sB if e is None else sB[e])[n])))
    assert np.array_equal(c_to_f64(C[r][:, n]), bf16(want))


@pytest.mark.parametrize("M", [3, 600])
def test_weights_past_32_bits(M):
    import torch
    G, N, K = 9, 16384, 65536
    (A, sA), (B, sB) = random_codes((M, K), 0), random_codes((G, N, K), 0)
    assert B.numel() > 2 ** 32
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    ids[:M // 2], ids[M - 1] = 8, 7
    log(f"weights past 32 bits {M}")
    C = fgg.grouped_mxfp4_gemm(A, B, sA, sB, ids)
    cols = [0, 1, 31, 8000, N - 1]
    picked(C, A, B, sA, sB, [0, M // 2 - 1], cols, 8)
    picked(C, A, B, sA, sB, [M - 1], cols, 7)
    assert not C[M // 2:M - 1].any()


def test_rows_past_32_bits():
    """More than 2^32 bytes of A, and of C."""
    for M, N, K in ((2 ** 20 + 77, 16, 8320), (2 ** 17 + 3, 16656, 128)):
        (A, sA), (B, sB) = random_codes((M, K), 0), random_codes((N, K), 0)
        log(f"rows past 32 bits {M} {N} {K}")
        C = fgg.mxfp4_gemm(A, B, sA, sB)
        assert max(A.numel(), C.numel() * 2) > 2 ** 32
        picked(C, A, B, sA, sB, [0, 1, M // 2, M - 129, M - 1], [0, 7, N // 2, N - 1])


def test_two_streams_at_once():
    import torch
    rng = np.random.default_rng(11)
    M, N, K = 40, 1024, 2048
    cases = []
    for m in (M, 40 * M):
        A, sA = coded((m, K), rng, exact_spread(K))
        B, sB = coded((N, K), rng, exact_spread(K))
        cases.append(([dev(v) for v in (A, B, sA, sB)], bf16(om.gemm(A, B, sA, sB)[0])))
    torch.cuda.synchronize()
    log("two streams")
    streams, out = [torch.cuda.Stream() for _ in cases], [[], []]
    for _ in range(10):
        for i, (args, _) in enumerate(cases):
            out[i].append(fgg.mxfp4_gemm(*args, stream=streams[i]))
    torch.cuda.synchronize()
    for i, (_, want) in enumerate(cases):
        for C in out[i]:
            assert np.array_equal(c_to_f64(C), want)


def runs(loads, rng, G):
    """Rows of (expert, rows) in turn, the experts out of range in several ways."""
    return np.concatenate([np.full(n, e if 0 <= e < G else rng.choice([-1, G, -7, 2 ** 31 - 1]), np.int32) for e, n in loads])


# runs that end at, before and behind half a span and a span; an expert with several runs; more runs than are
# taken as such; as many heavy spans as fill the card's last round by half, with and without light ones
RUNS = [(272, 384, 3, [(0, 128), (1, 129), (2, 127), (0, 256), (9, 1), (1, 257), (2, 255), (-1, 300), (0, 1)]),
        (4112, 256, 3, [(2, 1000), (0, 128), (-1, 129), (1, 897)]), (2064, 128, 2, [(0, 4100), (1, 1)]), (2064, 128, 2, [(-1, 700), (1, 4100)]),
        (528, 128, 4, [(g % 4, 5 + g) for g in range(60)]), (528, 640, 9, [(g % 9, 40 + 13 * g) for g in range(19)]),
        (528, 640, 9, [(g % 9, 40 + 13 * g) for g in range(20)]), (4112, 128, 9, [(g, 256 + 60 * (g % 2)) for g in range(9)]),
        (16, 128, 300, [(g, 100) for g in range(300)]), (48, 128, 600, [(g, 130) for g in range(600)]), (16, 256, 1100, [(g, 30) for g in range(1100)]),
        (8208, 128, 5, [(g, 513) for g in range(5)]), (1040, 256, 2, [(0, 129), (5, 2000), (1, 130)])]


@pytest.mark.parametrize("N,K,G,loads", RUNS)
def test_runs(N, K, G, loads):
    rng = np.random.default_rng(N + K + G)
    ids = runs(loads, rng, G)
    log(f"runs {len(ids)} {N} {K} {G} {len(loads)}")
    compare(len(ids), N, K, G, ids, rng)


@pytest.mark.parametrize("F,K,G,loads,quantize", [(c[0] - 16, *c[1:], q) for c in RUNS if c[0] > 100 for q in (False, True)])
def test_runs_gated(F, K, G, loads, quantize):
    rng = np.random.default_rng(F + K + G)
    ids = runs(loads, rng, G)
    A, sA, B, sB, _ = gated_case(len(ids), F, K, G, "one")
    log(f"runs gated {len(ids)} {F} {K} {G} {len(loads)} {quantize}")
    out = call_gated(A, sA, B, sB, ids, quantize=quantize)
    z, halves, S = om.gated(A, B, sA, sB, ids)
    if quantize:
        check_mxfp4(host(out[0]), host(out[1]), z, gated_bound(z, halves, S, K))
        nobody = (ids < 0) | (ids >= G)
        assert not host(out[0])[nobody].any() and not host(out[1])[nobody].any()
    else:
        check_bf16(c_to_f64(out), z, gated_bound(z, halves, S, K))


def test_result_over_an_operand():
    """A result that would overwrite what other workgroups still read is refused; one beside it is not."""
    import torch
    M, N, K = 64, 128, 512
    rng = np.random.default_rng(5)
    A, sA = coded((M, K), rng, exact_spread(K))
    B, sB = coded((N, K), rng, exact_spread(K))
    room = torch.zeros(2 * M * K, dtype=torch.uint8, device="cuda")
    a = room[:M * K // 2].view(M, K // 2)
    a.copy_(dev(A))
    args = [a, dev(B), dev(sA), dev(sB)]
    with pytest.raises(ValueError, match="overlap"):
        fgg.mxfp4_gemm(*args, out=room[M * K // 2 - 16:M * K // 2 - 16 + 2 * M * N].view(torch.bfloat16).view(M, N))
    out = room[M * K // 2:M * K // 2 + 2 * M * N].view(torch.bfloat16).view(M, N)
    log("result beside an operand")
    assert fgg.mxfp4_gemm(*args, out=out) is out
    assert np.array_equal(c_to_f64(out), bf16(om.gemm(A, B, sA, sB)[0]))


@pytest.mark.parametrize("quantize", [None, False, True])
def test_capacity(quantize):
    """Every expert's rows at the start of as many places, the rest of no expert, some of them empty or full."""
    G, places, N, K = 6, 400, 1056, 256
    rng = np.random.default_rng(8)
    ids = np.full((G, places), -1, np.int32)
    for e, n in enumerate((0, 400, 1, 129, 300, 256)):
        ids[e, :n] = e
    ids = ids.ravel()
    log(f"capacity {quantize}")
    if quantize is None:
        compare(len(ids), N, K, G, ids, rng)
        return
    A, sA, B, sB, _ = gated_case(len(ids), N, K, G, "one")
    out = call_gated(A, sA, B, sB, ids, quantize=quantize)
    z, halves, S = om.gated(A, B, sA, sB, ids)
    if quantize:
        check_mxfp4(host(out[0]), host(out[1]), z, gated_bound(z, halves, S, K))
        assert not host(out[0])[ids < 0].any() and not host(out[1])[ids < 0].any()
    else:
        check_bf16(c_to_f64(out), z, gated_bound(z, halves, S, K))


@pytest.mark.parametrize("M,N,K,G", [(2, 32, 1 << 20, 1), (150, 32, 1 << 20, 1), (3, 1 << 19, 128, 1), (140, 1 << 19, 128, 1),
                                     (40, 16, 128, 1 << 16), (300, 16, 128, 1 << 16)])
def test_largest_sizes(M, N, K, G):
    """The largest K, N and G that are taken; sums within their bound where FP32 does not hold them."""
    rng = np.random.default_rng(M)
    A, sA = coded((M, K), rng, 0)
    B, sB = coded((G, N, K), rng, 0)
    log(f"largest sizes {M} {N} {K} {G}")
    if G == 1:
        C = fgg.mxfp4_gemm(dev(A), dev(B[0]), dev(sA), dev(sB[0]))
        want, S = om.gemm(A, B[0], sA, sB[0])
    else:
        ids = rng.integers(-1, G, M).astype(np.int32)
        ids[-1] = G - 1
        C = fgg.grouped_mxfp4_gemm(dev(A), dev(B), dev(sA), dev(sB), dev(ids))
        used = np.unique(ids[ids >= 0])
        want, S = om.gemm(A, B[used], sA, sB[used], np.where(ids < 0, -1, np.searchsorted(used, ids)))
    check_bf16(c_to_f64(C), want, sum_bound(S, K))


@pytest.mark.parametrize("M,G", [(1 << 24, 2), (700001, 3)])
def test_most_rows(M, G):
    """More rows than fit the search for runs."""
    import torch
    (A, sA), (B, sB) = random_codes((M, 128), 1), random_codes((G, 16, 128), 1)
    ids = (torch.arange(M, device="cuda") * G // M).int()
    ids[M // 3:M // 3 + 1000] = -1
    log(f"most rows {M}")
    C = fgg.grouped_mxfp4_gemm(A, B, sA, sB, ids)
    assert not C[M // 3:M // 3 + 1000].any()
    for rows, e in (([0, 200, M // 4], 0), ([M - 1, M - 300], G - 1)):
        picked(C, A, B, sA, sB, rows, list(range(16)), e)


def test_graphs_when_the_routing_changes():
    """Two captured calls, replayed in turn while the rows' experts change from runs to no order, to one expert,
    to none: which kernel runs was fixed at capture, where its tiles lie is found at each replay."""
    import torch
    rng = np.random.default_rng(21)
    cases = []
    for M, N, K, G in ((2600, 2064, 256, 4), (40, 144, 384, 60)):
        A, sA = coded((M, K), rng, exact_spread(K))
        B, sB = coded((G, N, K), rng, exact_spread(K))
        ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
        out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        args = [dev(v) for v in (A, B, sA, sB)]
        fgg.grouped_mxfp4_gemm(*args, ids, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fgg.grouped_mxfp4_gemm(*args, ids, out=out)
        cases.append((graph, ids, out, args, (A, B, sA, sB), G))
    for kind in ("runs", "any", "one", "padded", "none", "runs", "any"):
        for graph, ids, out, _, host_args, G in cases:
            new = routed(len(ids), G, rng, kind)
            ids.copy_(dev(new))
            out.fill_(float("nan"))
            log(f"graph {len(ids)} {kind}")
            graph.replay()
            want, _ = om.gemm(*host_args, new)
            assert np.array_equal(c_to_f64(out), bf16(want)), kind
