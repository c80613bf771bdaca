"""The MXFP4 products of few rows an expert in batches of more rows than one scan of m_indices takes (1024): rows of
an expert in several scans, runs that a scan's end cuts, chunks of 16 and 32 rows in a later scan, padding in each.
Codes whose sums FP32 holds exactly, compared bit by bit with the float64 oracle; the gated ones within their bounds.
(tests/test_mx_rule.py holds these cases to the kernel that scans.)"""
import numpy as np
import pytest

import fp4_grouped_gemm_amd as fgg
from tests.gpu_util import c_bits, c_to_f64, log
from oracle import mxfp4 as om
from tests.mxfp4_cases import check_bf16, check_mxfp4, coded, gated_bound, routed
from tests.test_gpu_mxfp4 import call_gated, dev, gated_case, host
from tests.test_gpu_mxfp4_kernels import compare

pytestmark = pytest.mark.gpu

GROUPED = [(1025, 48, 384, 43, "any"), (1025, 48, 1408, 43, "runs"), (1025, 48, 256, 43, "one"), (2300, 32, 1152, 96, "one"),
           (2049, 272, 2176, 86, "runs"), (2049, 272, 640, 86, "any"), (2100, 144, 640, 88, "padded"), (3100, 1040, 384, 130, "any"),
           (3100, 16, 3456, 130, "runs"), (6144, 80, 1152, 256, "any"), (6144, 80, 640, 256, "runs"), (1500, 4112, 256, 70, "none"),
           (1536, 32, 128, 64, "any"), (1100, 16, 1 << 14, 46, "one")]
GATED = [(1030, F, K, 44, kind, q) for F, K in ((96, 640), (32, 1408)) for kind in ("any", "runs", "one") for q in (False, True)]
GATED += [(2100, 2080, 384, 90, kind, q) for kind in ("any", "padded") for q in (False, True)]
GATED += [(3100, 16, 256, 130, "runs", False), (2600, 160, 2176, 110, "any", True), (1100, 32, 256, 50, "none", True)]


@pytest.mark.parametrize("M,N,K,G,kind", GROUPED)
def test_grouped(M, N, K, G, kind):
    rng = np.random.default_rng(M + N + K + G)
    log(f"grouped_mxfp4_gemm {M} {N} {K} {G} {kind}")
    compare(M, N, K, G, routed(M, G, rng, kind), rng)


@pytest.mark.parametrize("M,F,K,G,kind,quantize", GATED)
def test_gated(M, F, K, G, kind, quantize):
    A, sA, B, sB, ids = gated_case(M, F, K, G, kind)
    nobody = (ids < 0) | (ids >= G)
    loud = sA.copy()
    loud[nobody] = 255  # what rows of padding hold reaches nothing
    log(f"gated {M} {F} {K} {G} {kind} {quantize}")
    out = call_gated(A, loud, B, sB, ids, quantize=quantize)
    z, halves, S = om.gated(A, B, sA, sB, ids)
    if quantize:
        check_mxfp4(host(out[0]), host(out[1]), z, gated_bound(z, halves, S, K))
        assert not host(out[0])[nobody].any() and not host(out[1])[nobody].any()
    else:
        check_bf16(c_to_f64(out), z, gated_bound(z, halves, S, K))


def lists():
    """(N, K, G, ids): an expert with few rows in the first scan and 15 to 70 in the next; one whose last row is a scan's first,
    or a scan's last; scans without a row of any expert; the first expert's rows last."""
    out = []
    for n in (15, 16, 17, 31, 32, 33, 64, 70):
        ids = np.full(2200, -1, np.int32)
        ids[[3, 700, 1023]] = 2
        ids[1030:1030 + 3 * n:3] = 2
        ids[2047], ids[2048], ids[2199] = 1, 99, 0
        out.append((48, 640, 100, ids))
    for at in (1023, 1024, 1025):
        ids = np.full(1200, 5, np.int32)
        ids[:at] = 4
        ids[at + 1:] = np.arange(1200 - at - 1) % 50
        out.append((272, 896, 50, ids))
    ids = np.full(4200, -7, np.int32)
    ids[0], ids[3000:3040], ids[4199] = 174, 0, 0
    out.append((32, 1152, 175, ids))
    return out


@pytest.mark.parametrize("i", range(len(lists())))
def test_lists(i):
    N, K, G, ids = lists()[i]
    log(f"lists {i} {len(ids)} {N} {K} {G}")
    compare(len(ids), N, K, G, ids, np.random.default_rng(i))


# K over 4, 2 and 1 of a workgroup's waves
REPEATED = [(20, 160, 4096, 2, 4), (32, 9600, 2048, 2, 2), (20, 9600, 1024, 8, 1), (1030, 64, 2048, 44, 4), (1030, 512, 1024, 44, 2)]


@pytest.mark.parametrize("M,N,K,G,ksplit", REPEATED)
def test_results_do_not_depend_on_timing(M, N, K, G, ksplit):
    """Sums that FP32 rounds: the same bits from every call, beside another stream's work too."""
    import torch
    rng = np.random.default_rng(M + N)
    A, sA = coded((M, K), rng, 20)
    B, sB = coded((G, N, K), rng, 20)
    args = [dev(v) for v in (A, B, sA, sB, routed(M, G, rng, "any"))]
    log(f"repeated {M} {N} {K} {G}")
    first = c_bits(fgg.grouped_mxfp4_gemm(*args))
    other, x = torch.cuda.Stream(), torch.zeros(1 << 24, device="cuda")
    torch.cuda.synchronize()
    for i in range(6):
        with torch.cuda.stream(other):
            x.add_(1)
        assert np.array_equal(c_bits(fgg.grouped_mxfp4_gemm(*args)), first)
    torch.cuda.synchronize()
