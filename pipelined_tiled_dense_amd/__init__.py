"""bf16 GEMM for MI355X (gfx950): a persistent, circular-buffered, tiled kernel.

The compute path is the HIP library ``libgemm_bf16.so`` built from ``csrc/``;
``binding`` is a thin ctypes layer over its C ABI.  The binding is imported
lazily so that ``inputs`` can be used without loading the HIP library.
"""
from __future__ import annotations

import importlib

_FROM_BINDING = ("gemm", "gemm_fp8", "quantize_fp8", "rms_norm", "rms_norm_backward", "swiglu", "swiglu_backward",
                 "RmsNorm", "GemmError", "SYNC_MODES")
__all__ = ["binding", "inputs", "mlp", *_FROM_BINDING, "FeedForward"]


def __getattr__(name):
    if name in _FROM_BINDING:
        return getattr(importlib.import_module(__name__ + ".binding"), name)
    if name == "FeedForward":
        return importlib.import_module(__name__ + ".mlp").FeedForward
    raise AttributeError(name)
