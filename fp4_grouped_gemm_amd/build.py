"""Build libfgg.so (the HIP kernels and the C ABI) in-tree for gfx950, and
_attention.so (the compiled part of the Python binding, host code only; it
takes torch's headers, and is left out where there is no torch).

    python -m fp4_grouped_gemm_amd.build        (or fp4_grouped_gemm_amd.build.build())

Every source is compiled with hipcc for gfx950 only; packed FP32 VALU
instructions are disabled (-packed-fp32-ops) and MFMA results are kept in
VGPRs (-amdgpu-mfma-vgpr-form).  Objects go to _build/ at the
repository root, the shared libraries next to this file.
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfgg.so")

SOURCES = ["api.cpp", "fp8_grouped.hip", "fp4.hip", "quant.hip", "w4a16.hip",
           "attn_append.hip", "attn_decode.hip", "attn_prompt.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA results in VGPRs: the FP8 kernel promotes every partial with VALU
    # FMAs, which cannot read AGPRs directly.
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-Wall", "-Wno-unused-command-line-argument",
    "-I" + os.path.join(ROOT, "include"),
]
BINDING = os.path.join(PKG, "_attention.so")


def _run(cmd: list[str], what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _binding(lib: str) -> str | None:
    """Compile the binding against the installed torch and link it to `lib`
    (its host side only: there is no kernel in it); returns the built file, not yet in
    its place.  None if there is no torch: the C ABI does not need one."""
    if importlib.util.find_spec("torch") is None:
        return None
    import torch
    home = os.path.dirname(torch.__file__)
    tmp = BINDING + ".tmp"
    _run([HIPCC, "-x", "hip", "--offload-host-only", "-no-hip-rt", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
          "-DUSE_ROCM",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
          "-I" + os.path.join(ROOT, "include"),
          *(flag for d in (os.path.join(home, "include"),
                           os.path.join(home, "include", "torch", "csrc", "api", "include"),
                           sysconfig.get_path("include"))
            for flag in ("-isystem", d)),
          os.path.join(CSRC, "attention_binding.cpp"), "-x", "none", lib, "-o", tmp,
          "-L" + os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10_hip", "-lc10",
          "-Wl,-rpath,$ORIGIN"], "attention_binding.cpp")
    return tmp


def _compile(src: str) -> str:
    out = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    lang = ["-x", "hip"] if src.endswith(".cpp") else []
    cmd = [HIPCC, *FLAGS, *lang, "-c", os.path.join(CSRC, src), "-o", out]
    _run(cmd, f"hipcc for {src}")
    return out


PROBES = ["mfma_peak", "lds_banks"]
PROBE = os.path.join(ROOT, "bench", "mfma_peak")


def build_probe(verbose: bool = False) -> str:
    """Build the microbenchmarks in bench/ (standalone HIP programs, not part
    of the library): mfma_peak (roofline legs) and lds_banks (LDS
    bank-conflict patterns)."""
    for name in PROBES:
        src = os.path.join(ROOT, "bench", name + ".hip")
        exe = os.path.join(ROOT, "bench", name)
        cmd = [HIPCC, *[f for f in FLAGS if f not in ("-fPIC",) and not f.startswith("-I")],
               src, "-o", exe]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            print("built", exe)
    return PROBE


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-Wl,-soname,libfgg.so", *objs, "-o", tmp]
    _run(cmd, "link")
    # both are built before either is put in its place: a library never stands
    # beside a binding that was linked to another one
    binding = _binding(tmp)
    if binding:
        os.replace(binding, BINDING)
    elif os.path.exists(BINDING):
        os.remove(BINDING)
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
        print("built", BINDING) if binding else print("no torch: the attention binding is not built")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
