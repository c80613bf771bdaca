"""Host tests of the attention operators' definitions at the edges."""
import os
import shutil
import subprocess
import sys

import numpy as np
import pytest

from oracle import attention as oa
from tests.test_attention_abi import _prompt

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_start_before_an_earlier_one_counts_as_that_one():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((9, 2, 4)), rng.standard_normal((9, 1, 4)), rng.standard_normal((9, 1, 4))
    for starts, same in (([0, 9, 0, 9], [0, 9]), ([3, 7, 5, 8], [3, 7, 7, 8]), ([-4, 6, 2, 100, 1], [0, 6, 6, 9])):
        for got, want in zip(oa.prompt_attention(q, k, v, starts, 0.5), oa.prompt_attention(q, k, v, same, 0.5)):
            assert np.array_equal(got, want)
    out, _ = oa.prompt_attention(q, k, v, [3, 7, 5, 8], 0.5)
    assert not out[:3].any() and not out[8:].any() and out[3:8].all()


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_the_list_of_work_at_the_ends_of_its_range(tmp_path):
    """csrc/attn_list.h, the arithmetic the kernels call: tests/attn_list_check.cpp.
    (Overflows trap instead of wrapping.)"""
    exe = str(tmp_path / "attn_list_check")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-ftrapv", "-I", os.path.join(ROOT, "fp4_grouped_gemm_amd", "csrc"),
                    os.path.join(ROOT, "tests", "attn_list_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and " 0 failed" in r.stdout, (r.returncode, r.stdout)


@pytest.mark.parametrize("T,batch,hq,hk", [(1000, 1 << 20, 64, 16), (100, (1 << 19) - 2 - 1, 64, 32), (128, (1 << 18) - 3, 64, 64),
                                           (1 << 24, 1, 128, 32)])
def test_prompts_that_one_launch_cannot_take_are_refused(T, batch, hq, hk):
    """At 2^24 workgroups of 256 threads (2^32) and above, before any device is touched."""
    status, msg = _prompt(T=T, batch=batch, hq=hq, hk=hk)
    assert status == 2 and msg.startswith("prompt_attention:") and "2^24" in msg


@pytest.mark.parametrize("which", [2, 4])
def test_prompt_token_strides_past_32_bit_offsets_are_refused(which):
    strides = [1024, 128, 512, 128, 512, 128]
    strides[which] = (1 << 22) + 8
    status, msg = _prompt(strides=strides)
    assert status == 2 and "token strides" in msg


@pytest.mark.parametrize("missing", ["torch", "fp4_grouped_gemm_amd._attention"])
def test_the_package_imports_without_torch_or_the_compiled_binding(missing):
    """What they are needed for says so when it is called."""
    code = (f"import sys; sys.modules[{missing!r}] = None\n"
            "from fp4_grouped_gemm_amd import *\n"
            "import fp4_grouped_gemm_amd as fgg\n"
            "assert all(callable(f) for f in (grouped_fp8_gemm, rope_kv_append, prompt_attention))\n"
            "load_library()\n"
            "try:\n"
            "    prompt_attention(None, None, None, None)\n"
            "except ImportError as e:\n"
            "    print('refused:', e)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "refused:" in r.stdout, r.stderr
    if missing != "torch":
        assert "python -m fp4_grouped_gemm_amd.build" in r.stdout
