"""bf16 GEMM for MI355X (gfx950): a persistent, circular-buffered, tiled kernel.

The compute path is the HIP library ``libgemm_bf16.so`` built from ``csrc/``;
``binding`` is a thin ctypes layer over its C ABI.  The binding is imported
lazily so that ``inputs`` can be used without loading the HIP library.
"""
from __future__ import annotations

import importlib

_FROM_BINDING = ("gemm", "gemm_fp8", "quantize_fp8", "rms_norm", "rms_norm_backward", "swiglu", "swiglu_backward",
                 "linear", "linear_backward_input", "linear_backward_weight", "gated_linear",
                 "gated_linear_backward_input", "RmsNorm", "GemmError", "SYNC_MODES")
_FROM_MLP = ("FeedForward", "FeedForwardBF16")
__all__ = ["binding", "inputs", "mlp", *_FROM_BINDING, *_FROM_MLP]


def __getattr__(name):
    if name in _FROM_BINDING:
        return getattr(importlib.import_module(__name__ + ".binding"), name)
    if name in _FROM_MLP:
        return getattr(importlib.import_module(__name__ + ".mlp"), name)
    raise AttributeError(name)
