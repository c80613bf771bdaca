"""What a build leaves behind when a part of it cannot be built (no compiler runs)."""
import importlib.util
import os

import pytest

from fp4_grouped_gemm_amd import build as b


@pytest.fixture
def paths(tmp_path, monkeypatch):
    """An older build in tmp_path, and a toolchain that writes its output's name."""
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libfgg.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_attention.so"))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(b, "_compile", lambda src: src + ".o")
    failing = []

    def run(cmd, what):
        if what in failing:
            raise RuntimeError(f"{what} failed")
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write("new")

    monkeypatch.setattr(b, "_run", run)
    for p in (b.LIB, b.BINDING):
        with open(p, "w") as f:
            f.write("old")
    return failing


def _read(path):
    with open(path) as f:
        return f.read()


def test_both_libraries_are_replaced(paths):
    b.build()
    assert _read(b.LIB) == "new" and _read(b.BINDING) == "new"


def test_a_binding_that_fails_leaves_the_older_pair(paths):
    paths.append("attention_binding.cpp")
    with pytest.raises(RuntimeError, match="attention_binding"):
        b.build()
    assert _read(b.LIB) == "old" and _read(b.BINDING) == "old"


def test_without_torch_the_c_abi_is_built(paths, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    b.build()
    assert _read(b.LIB) == "new" and not os.path.exists(b.BINDING)
