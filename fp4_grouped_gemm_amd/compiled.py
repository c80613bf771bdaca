"""The compiled part of the binding (_attention.so: csrc/attention_binding.cpp and
csrc/mxfp4_binding.cpp), shared by the modules whose functions it holds."""
from __future__ import annotations

C = None  # the module, once a call has loaded it


def load():
    """The compiled module, loaded by the first call: importing the package needs
    neither torch nor a built library."""
    global C
    import torch  # noqa: F401  (its libraries come first)
    try:
        from . import _attention
    except ImportError as e:
        raise ImportError("the compiled binding (attention and MXFP4 operators, residual_norm) is missing or was "
                          "built for another torch: build it with `python -m fp4_grouped_gemm_amd.build`") from e
    C = _attention
    return C


def on(stream, q):
    """A context in which `stream` is the current one, so that memory allocated
    for the call belongs to the stream that uses it."""
    import torch
    if stream.device != q.device:
        raise ValueError(f"stream is on {stream.device}, expected {q.device}")
    return torch.cuda.stream(stream)
