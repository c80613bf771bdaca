"""The MXFP4 products' tests reach the kernels that they are written for: csrc/mx_rule.h, which the launchers call,
asked by tests/mx_rule_check.cpp."""
import os
import shutil
import subprocess

import pytest

from tests import test_gpu_mxfp4_scans as scans

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path_factory.mktemp("rule") / "mx_rule_check")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-I", os.path.join(ROOT, "fp4_grouped_gemm_amd", "csrc"),
                    os.path.join(ROOT, "tests", "mx_rule_check.cpp"), "-o", exe], check=True)

    def ask(cases, cus=256):
        """Kernels of (M, N, G, gated, MXFP4 result)."""
        lines = "".join("%d %d %d %d %d on %d\n" % (*map(int, c), cus) for c in cases)
        return subprocess.run([exe], input=lines, capture_output=True, text=True, timeout=60, check=True).stdout.splitlines()
    return ask


def test_the_rule_is_asked(kernels):
    assert kernels([(1, 4096, 1, 0, 0), (16, 64, 1, 1, 1), (2048, 4096, 1, 0, 0), (2100, 4096, 1, 0, 0), (300, 4096, 1, 0, 0)]) == [
        "rows 4", "rows 2", "tiles", "large tiles", "tiles"]


def test_scans_reach_the_stream(kernels):
    cases = [(M, N, G, 0, 0) for M, N, K, G, kind in scans.GROUPED] + [(M, F, G, 1, q) for M, F, K, G, kind, q in scans.GATED]
    cases += [(len(ids), N, G, 0, 0) for N, K, G, ids in scans.lists()]
    assert len(cases) >= 30 and all(c[0] > 1024 for c in cases)
    got = kernels(cases)
    assert all(k.startswith("rows") for k in got), [c for c, k in zip(cases, got) if not k.startswith("rows")]
    assert len(set(got)) == 3  # K whole, in two parts, in four


def test_repeated_calls_split_k(kernels):
    got = kernels([(M, N, G, 0, 0) for M, N, K, G, ksplit in scans.REPEATED])
    assert got == ["rows %d" % ksplit for M, N, K, G, ksplit in scans.REPEATED] and {k for *_, k in scans.REPEATED} == {1, 2, 4}


@pytest.mark.parametrize("cus", [256, 128, 32])
def test_k_is_split_by_the_card(kernels, cus):
    """One row: four waves a column block up to one wave a compute unit, two up to four; halves of a card as well."""
    got = kernels([(1, 32 * w, 1, 0, 0) for w in (cus, cus + 1, 4 * cus, 4 * cus + 1)], cus)
    assert got == ["rows 4", "rows 2", "rows 2", "rows 1"]
