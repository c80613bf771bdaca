"""The LDS layout and staging offsets of prompt_attention (csrc/attn_layout.h, the
arithmetic the kernel calls) checked on the host: tests/attn_layout_check.cpp
enumerates every load and fragment read."""
import os
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_staging_and_fragment_reads():
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "attn_layout_check")
        subprocess.run(["g++", "-O1", "-std=c++17", "-Wall",
                        "-I", os.path.join(ROOT, "fp4_grouped_gemm_amd", "csrc"),
                        os.path.join(ROOT, "tests", "attn_layout_check.cpp"), "-o", exe], check=True)
        r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    print(r.stdout)
    assert r.returncode == 0, r.stdout
    assert " 0 failed" in r.stdout and "seen" in r.stdout
