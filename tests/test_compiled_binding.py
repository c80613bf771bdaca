"""Without torch or the compiled module the calls that need it say what is missing; with them the modules share one."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALLS = ["quantize_mxfp4(None)", "dequantize_mxfp4(None, None)", "mxfp4_gemm(*4 * [None])", "grouped_mxfp4_gemm(*5 * [0])",
         "mxfp4_gated_gemm(*4 * [None])", "grouped_mxfp4_gated_gemm(*5 * [0])", "residual_norm(None, None, None)",
         "rope_kv_append(*8 * [None])", "paged_decode_attention(*5 * [None])", "prompt_attention(*4 * [None])"]


@pytest.mark.parametrize("missing", ["torch", "fp4_grouped_gemm_amd._attention"])
def test_what_is_missing_is_named(missing):
    code = f"import sys; sys.modules[{missing!r}] = None\nfrom fp4_grouped_gemm_amd import *\n"
    for call in CALLS:
        code += f"try:\n    {call}\nexcept ImportError as e:\n    print({call.partition('(')[0]!r}, e)\n"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    lines = r.stdout.splitlines()
    assert r.returncode == 0 and [line.split()[0] for line in lines] == [c.partition("(")[0] for c in CALLS], r.stderr
    if missing != "torch":
        for line in lines:
            assert "attention and MXFP4 operators, residual_norm" in line and "python -m fp4_grouped_gemm_amd.build" in line


def test_one_module():
    pytest.importorskip("torch")
    from fp4_grouped_gemm_amd import attention, compiled, mxfp4
    assert compiled.load() is compiled.load() is compiled.C
    assert attention.compiled is mxfp4.compiled is compiled
