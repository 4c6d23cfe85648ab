"""Thin ctypes binding over the C ABI of ``libgemm_bf16.so`` (include/gemm_bf16.h).

Every function here only marshals arguments: the GEMM itself runs in the HIP
kernels of the library.  There is no fallback: if the library is missing or
cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "libgemm_bf16.so")

GEMM_OK = 0
GEMM_ERR_INVALID_VALUE = -1
GEMM_ERR_MISALIGNED = -2
GEMM_ERR_UNSUPPORTED_SHAPE = -3
GEMM_ERR_STAGES = -4
GEMM_ERR_SYNC_MODE = -5
GEMM_ERR_DEVICE = -6
GEMM_ERR_LAUNCH = -7
GEMM_ERR_ALIAS = -8
GEMM_ERR_SCRATCH = -9
GEMM_NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024

SYNC_MODES = {"barrier": 0, "flags": 1, "wavespec": 2, "pingpong": 3}
STAGES_WINDOWS = 5          # GEMM_STAGES_WINDOWS: the split-window ring (barrier sync)
TYPE_BF16 = 0
TYPE_FP8 = 1
TYPE_FP32 = 2
FP8_EXACT = 256             # GEMM_FP8_EXACT, added to gemm_fp8_bt's c_type
LINEAR_PRODUCTS = {"linear": 0, "linear_bwd_input": 1, "linear_bwd_weight": 2, "gated_linear": 3,
                   "gated_linear_bwd_input": 4}   # GEMM_LINEAR, ...
ACTIVATIONS = {None: 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}   # GEMM_ACT_*
BLOCK = 128                 # values along k (and rows of a block) that share a scale
NORM_MAX_WIDTH = 32768      # GEMM_NORM_MAX_WIDTH


class GemmError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__("%s%s (status %d)" % (what + ": " if what else "", strerror(code), code))


class Plan(ctypes.Structure):
    _fields_ = [("bm", ctypes.c_int32), ("bn", ctypes.c_int32), ("bk", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("sync_mode", ctypes.c_int32),
                ("b_transposed", ctypes.c_int32), ("mfma_waves", ctypes.c_int32),
                ("producer_waves", ctypes.c_int32), ("threads", ctypes.c_int32),
                ("lds_bytes", ctypes.c_int32), ("tiles", ctypes.c_int64),
                ("k_steps", ctypes.c_int64), ("grid", ctypes.c_int64),
                ("k_splits", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
                ("tail_tiles", ctypes.c_int64), ("tail_splits", ctypes.c_int64),
                ("pad_bytes", ctypes.c_int64), ("mfma_block", ctypes.c_int64),
                ("pipelines", ctypes.c_int64)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class Fp8Plan(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("few_rows", ctypes.c_int32),
                ("exact", ctypes.c_int32), ("threads", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("tiles", ctypes.c_int64), ("k_splits", ctypes.c_int64), ("k_blocks", ctypes.c_int64),
                ("grid", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64), ("pad_bytes", ctypes.c_int64)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_ if name != "reserved"}


class LinearPlan(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("waves_share_k", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("tiles", ctypes.c_int64), ("k_splits", ctypes.c_int64),
                ("k_chunk", ctypes.c_int64), ("grid", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
                ("pad_bytes", ctypes.c_int64), ("scratch_bytes", ctypes.c_int64)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


_lib = None


def library() -> ctypes.CDLL:
    """The loaded HIP library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIBRARY):
            raise RuntimeError("HIP library %s is not built; run __graft_entry__.build() or "
                               "python -m pipelined_tiled_dense_amd.build" % LIBRARY)
        lib = ctypes.CDLL(LIBRARY)
        i64, p, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        sig = [i64, i64, i64, p, i64, p, i64, p, i64, i32, i32, p]
        lib.gemm_bf16.argtypes = sig
        lib.gemm_bf16.restype = i32
        lib.gemm_bf16_bt.argtypes = sig
        lib.gemm_bf16_bt.restype = i32
        lib.gemm_bf16_noalloc.argtypes = sig
        lib.gemm_bf16_noalloc.restype = i32
        lib.gemm_bf16_plan.argtypes = [i64, i64, i64, i32, i32, i32, ctypes.POINTER(Plan)]
        lib.gemm_bf16_plan.restype = i32
        lib.gemm_bf16_plan_cus.argtypes = [i64, i64, i64, i32, i32, i32, i32, ctypes.POINTER(Plan)]
        lib.gemm_bf16_plan_cus.restype = i32
        lib.gemm_bf16_strerror.argtypes = [i32]
        lib.gemm_bf16_strerror.restype = ctypes.c_char_p
        lib.gemm_bf16_sync_timeouts.argtypes = [i32]
        lib.gemm_bf16_sync_timeouts.restype = i64
        lib.gemm_bf16_set_sync_spin_limit.argtypes = [i64]
        lib.gemm_bf16_set_sync_spin_limit.restype = i64
        lib.gemm_bf16_set_clock_sampling.argtypes = [i32]
        lib.gemm_bf16_set_clock_sampling.restype = i32
        lib.gemm_bf16_clock_samples.argtypes = [ctypes.POINTER(ctypes.c_uint64), i32]
        lib.gemm_bf16_clock_samples.restype = i32
        lib.gemm_bf16_workspace_info.argtypes = [ctypes.POINTER(ctypes.c_int64)] * 3
        lib.gemm_bf16_workspace_info.restype = i32
        lib.gemm_bf16_release_workspaces.argtypes = []
        lib.gemm_bf16_release_workspaces.restype = i32
        lib.gemm_fp8_bt.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, p, i64, i32, p, i64, i32, p]
        lib.gemm_quantize_fp8.argtypes = [i64, i64, p, i64, p, i64, p, i64, i32, i32, p]
        lib.gemm_rms_norm.argtypes = [i64, i64, p, i64, p, i64, p, ctypes.c_float, p, i64, p, i64, i32, p, i64, p, p]
        lib.gemm_rms_norm_bwd.argtypes = [i64, i64, p, i64, p, i64, p, p, p, i64, p, i64, p, p]
        lib.gemm_rms_norm_bwd_given.argtypes = [i64, i64, p, i64, p, i64, p, p, p, i64, p, i64, p, p, i64, p]
        lib.gemm_rms_norm_bwd_scratch_cus.argtypes = [i64, i64, i32]
        lib.gemm_rms_norm_bwd_scratch_cus.restype = i64
        lib.gemm_swiglu.argtypes = [i64, i64, p, i64, p, i64, i32, p, i64, p]
        lib.gemm_swiglu_bwd.argtypes = [i64, i64, p, i64, p, i64, p, i64, p]
        lib.gemm_fp8_plan_cus.argtypes = [i64, i64, i64, i32, i32, i32, i32, i32, ctypes.POINTER(Fp8Plan)]
        lib.gemm_linear.argtypes = [i64, i64, i64, p, i64, p, i64, p, i32, p, i64, p, i64, p, i64, p, i64, p]
        lib.gemm_linear_bwd_input.argtypes = [i64, i64, i64, p, i64, p, i64, i32, p, i64, p, i64, p, i64, p, i64, p]
        lib.gemm_linear_bwd_weight.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, i32, p, p, i64, p]
        lib.gemm_gated_linear.argtypes = [i64, i64, i64, p, i64, p, i64, p, i32, p, i64, p, i64, p, i64, p]
        lib.gemm_gated_linear_bwd_input.argtypes = [i64, i64, i64, p, i64, p, i64, i32, p, i64, p, i64, p, i64, p, i64, p]
        lib.gemm_linear_plan_cus.argtypes = [i64, i64, i64, i32, i32, i32, i32, ctypes.POINTER(LinearPlan)]
        for name in ("gemm_fp8_bt", "gemm_fp8_plan_cus", "gemm_quantize_fp8", "gemm_rms_norm", "gemm_rms_norm_bwd",
                     "gemm_rms_norm_bwd_given",
                     "gemm_swiglu", "gemm_swiglu_bwd", "gemm_linear", "gemm_linear_bwd_input", "gemm_linear_bwd_weight",
                     "gemm_gated_linear", "gemm_gated_linear_bwd_input", "gemm_linear_plan_cus"):
            getattr(lib, name).restype = i32
        _lib = lib
    return _lib


# -- the C entry points, same names --------------------------------------------
def gemm_bf16(M, N, K, A, lda, B, ldb, C, ldc, stages, sync_mode, stream) -> int:
    return library().gemm_bf16(M, N, K, A, lda, B, ldb, C, ldc, stages, sync_mode, stream)


def gemm_bf16_bt(M, N, K, A, lda, B, ldb, C, ldc, stages, sync_mode, stream) -> int:
    return library().gemm_bf16_bt(M, N, K, A, lda, B, ldb, C, ldc, stages, sync_mode, stream)


def gemm_bf16_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stages, sync_mode, stream) -> int:
    return library().gemm_bf16_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stages, sync_mode, stream)


def gemm_bf16_plan(M, N, K, b_transposed, stages, sync_mode) -> dict:
    out = Plan()
    rc = library().gemm_bf16_plan(M, N, K, int(bool(b_transposed)), stages, sync_mode,
                                  ctypes.byref(out))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_bf16_plan")
    return out.as_dict()


def gemm_bf16_plan_cus(M, N, K, b_transposed, stages, sync_mode, compute_units) -> dict:
    out = Plan()
    rc = library().gemm_bf16_plan_cus(M, N, K, int(bool(b_transposed)), stages, sync_mode, compute_units,
                                      ctypes.byref(out))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_bf16_plan_cus")
    return out.as_dict()


def gemm_bf16_strerror(code: int) -> str:
    return library().gemm_bf16_strerror(code).decode()


def gemm_bf16_sync_timeouts(reset: bool = False) -> int:
    n = library().gemm_bf16_sync_timeouts(int(bool(reset)))
    if n < 0:
        raise GemmError(int(n), "gemm_bf16_sync_timeouts")
    return int(n)


def gemm_bf16_set_sync_spin_limit(polls: int) -> int:
    n = library().gemm_bf16_set_sync_spin_limit(int(polls))
    if n < 0:
        raise GemmError(int(n), "gemm_bf16_set_sync_spin_limit")
    return int(n)


def gemm_bf16_workspace_info() -> dict:
    """The temporary memory the library keeps on the current device: blocks,
    their total bytes, and how many are taken right now."""
    blocks, nbytes, busy = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    rc = library().gemm_bf16_workspace_info(ctypes.byref(blocks), ctypes.byref(nbytes), ctypes.byref(busy))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_bf16_workspace_info")
    return {"blocks": blocks.value, "bytes": nbytes.value, "busy": busy.value}


def gemm_bf16_release_workspaces() -> None:
    """Frees the temporary memory the library keeps on the current device
    (synchronises the device)."""
    rc = library().gemm_bf16_release_workspaces()
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_bf16_release_workspaces")


def gemm_bf16_set_clock_sampling(enable: bool) -> bool:
    """Turns the kernels' clock sampling on or off; returns the previous setting."""
    return bool(library().gemm_bf16_set_clock_sampling(int(bool(enable))))


def gemm_bf16_clock_samples(reset: bool = False) -> dict:
    """The current device's clock sums: shader-clock ticks, constant-rate ticks,
    samples, the constant rate in Hz, and the mean clock in GHz they give
    (None without samples)."""
    out = (ctypes.c_uint64 * 4)()
    rc = library().gemm_bf16_clock_samples(out, int(bool(reset)))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_bf16_clock_samples")
    shader, wall, n, hz = (int(v) for v in out)
    return {"shader_ticks": shader, "wall_ticks": wall, "samples": n, "wall_hz": hz,
            "clock_ghz": shader / wall * hz / 1e9 if wall > 0 else None}


def gemm_fp8_bt(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, b_block_rows, C, ldc, c_type, stream) -> int:
    return library().gemm_fp8_bt(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, b_block_rows, C, ldc, c_type, stream)


def gemm_fp8_plan_cus(M, N, K, b_block_rows, c_type, a_aligned, b_aligned, compute_units) -> dict:
    out = Fp8Plan()
    rc = library().gemm_fp8_plan_cus(M, N, K, b_block_rows, c_type, int(bool(a_aligned)), int(bool(b_aligned)),
                                     compute_units, ctypes.byref(out))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_fp8_plan_cus")
    return out.as_dict()


def gemm_quantize_fp8(M, K, X, ldx, Q, ldq, scale, lds, block_rows, transposed, stream) -> int:
    return library().gemm_quantize_fp8(M, K, X, ldx, Q, ldq, scale, lds, block_rows, transposed, stream)


def gemm_rms_norm(M, D, X, ldx, residual, ldr, weight, eps, H, ldh, Y, ldy, y_type, scale, lds, rstd, stream) -> int:
    return library().gemm_rms_norm(M, D, X, ldx, residual, ldr, weight, eps, H, ldh, Y, ldy, y_type, scale, lds,
                                   rstd, stream)


def gemm_rms_norm_bwd(M, D, dY, lddy, H, ldh, weight, rstd, dres, lddr, dX, lddx, dweight, stream) -> int:
    return library().gemm_rms_norm_bwd(M, D, dY, lddy, H, ldh, weight, rstd, dres, lddr, dX, lddx, dweight, stream)


def gemm_rms_norm_bwd_given(M, D, dY, lddy, H, ldh, weight, rstd, dres, lddr, dX, lddx, dweight, stream, workspace=None,
                            workspace_bytes=0) -> int:
    return library().gemm_rms_norm_bwd_given(M, D, dY, lddy, H, ldh, weight, rstd, dres, lddr, dX, lddx, dweight, workspace,
                                             workspace_bytes, stream)


def gemm_rms_norm_bwd_scratch_cus(M, D, compute_units) -> int:
    n = library().gemm_rms_norm_bwd_scratch_cus(M, D, compute_units)
    if n < 0:
        raise GemmError(n, "gemm_rms_norm_bwd_scratch_cus")
    return n


def gemm_swiglu(M, F, GU, ldgu, Y, ldy, y_type, scale, lds, stream) -> int:
    return library().gemm_swiglu(M, F, GU, ldgu, Y, ldy, y_type, scale, lds, stream)


def gemm_swiglu_bwd(M, F, dY, lddy, GU, ldgu, dGU, lddgu, stream) -> int:
    return library().gemm_swiglu_bwd(M, F, dY, lddy, GU, ldgu, dGU, lddgu, stream)


def gemm_linear(M, N, K, X, ldx, W, ldw, bias, act, residual, ldr, Z, ldz, Y, ldy, stream, workspace=None,
                workspace_bytes=0) -> int:
    return library().gemm_linear(M, N, K, X, ldx, W, ldw, bias, act, residual, ldr, Z, ldz, Y, ldy, workspace,
                                 workspace_bytes, stream)


def gemm_linear_bwd_input(M, N, K, dY, lddy, W, ldw, act, Z, ldz, dres, lddr, dX, lddx, stream, workspace=None,
                          workspace_bytes=0) -> int:
    return library().gemm_linear_bwd_input(M, N, K, dY, lddy, W, ldw, act, Z, ldz, dres, lddr, dX, lddx, workspace,
                                           workspace_bytes, stream)


def gemm_linear_bwd_weight(M, N, K, dY, lddy, X, ldx, dW, lddw, dw_type, dbias, stream, workspace=None,
                           workspace_bytes=0) -> int:
    return library().gemm_linear_bwd_weight(M, N, K, dY, lddy, X, ldx, dW, lddw, dw_type, dbias, workspace,
                                            workspace_bytes, stream)


def gemm_gated_linear(M, F, K, X, ldx, W, ldw, bias, act, GU, ldgu, Y, ldy, stream, workspace=None,
                      workspace_bytes=0) -> int:
    return library().gemm_gated_linear(M, F, K, X, ldx, W, ldw, bias, act, GU, ldgu, Y, ldy, workspace,
                                       workspace_bytes, stream)


def gemm_gated_linear_bwd_input(M, F, N, dY, lddy, W, ldw, act, GU, ldgu, dGU, lddgu, Y, ldy, stream, workspace=None,
                                workspace_bytes=0) -> int:
    return library().gemm_gated_linear_bwd_input(M, F, N, dY, lddy, W, ldw, act, GU, ldgu, dGU, lddgu, Y, ldy, workspace,
                                                 workspace_bytes, stream)


def gemm_linear_plan_cus(M, N, K, product, a_aligned, b_aligned, compute_units) -> dict:
    out = LinearPlan()
    rc = library().gemm_linear_plan_cus(M, N, K, LINEAR_PRODUCTS.get(product, product), int(bool(a_aligned)),
                                        int(bool(b_aligned)), compute_units, ctypes.byref(out))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_linear_plan_cus")
    return out.as_dict()


strerror = gemm_bf16_strerror


# -- tensor-level convenience ----------------------------------------------------
def _sync_code(sync) -> int:
    if isinstance(sync, str):
        if sync not in SYNC_MODES:
            raise ValueError("sync must be one of %s" % sorted(SYNC_MODES))
        return SYNC_MODES[sync]
    return int(sync)


def gemm(A, B, *, b_transposed: bool = False, stages: int = 0, sync="barrier", out=None,
         stream=None):
    """C = A @ B (or A @ B.T-stored when ``b_transposed``) for CUDA bf16 tensors
    with unit inner stride.  Returns ``out`` (allocated if None).  Runs on the
    current stream unless a torch stream is given."""
    import torch

    for name, X in (("A", A), ("B", B)):
        if X.dtype != torch.bfloat16 or X.dim() != 2 or not X.is_cuda:
            raise TypeError("%s must be a 2-D bfloat16 CUDA tensor" % name)
        if X.shape[0] * X.shape[1] > 0 and X.stride(1) != 1:
            raise ValueError("%s needs unit stride along its second dimension" % name)
    M, K = A.shape
    if b_transposed:
        N, KB = B.shape
    else:
        KB, N = B.shape
    if KB != K:
        raise ValueError("inner dimensions differ: %d vs %d" % (K, KB))
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    elif out.dtype != torch.bfloat16 or tuple(out.shape) != (M, N) or (M * N > 0 and out.stride(1) != 1):
        raise ValueError("out must be a bfloat16 tensor of shape (M, N) with unit inner stride")
    s = (stream or torch.cuda.current_stream(A.device)).cuda_stream
    fn = gemm_bf16_bt if b_transposed else gemm_bf16
    lda = A.stride(0) if M > 1 else max(K, 8)
    ldb = B.stride(0) if B.shape[0] > 1 else max(B.shape[1], 8)
    ldc = out.stride(0) if M > 1 else max(N, 8)
    rc = fn(M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, out.data_ptr(), ldc,
            int(stages), _sync_code(sync), s)
    if rc != GEMM_OK:
        raise GemmError(rc, fn.__name__)
    return out


# -- 8-bit operands and the operators around the product --------------------------
# 8-bit tensors are torch.float8_e4m3fn.  Scales are float32 with the k block
# first: shape (ceil(K / 128), rows) for row scales, (ceil(K / 128),
# ceil(rows / 128)) for blocks.  Every function runs on the current stream
# unless a torch stream is given; with one, results are allocated for that
# stream and the arguments are marked as used on it.
#
# For a few rows these calls take the host longer than the GPU, so the helpers
# below touch each tensor as little as they can.
class RmsNorm(NamedTuple):
    """What ``rms_norm`` returns; what was not asked for is None."""
    y: object               # bfloat16, or float8_e4m3fn with ``scale``
    scale: object = None    # float32 (ceil(D / 128), M)
    h: object = None        # bfloat16, x + residual
    rstd: object = None     # float32 (M,)


def _matrix(name, x, dtype):
    """Checks a 2-D CUDA operand with unit inner stride; returns its leading dimension."""
    if x.dtype is not dtype or x.ndim != 2 or not x.is_cuda:
        raise TypeError("%s must be a 2-D %s CUDA tensor" % (name, str(dtype).replace("torch.", "")))
    rows, cols = x.shape
    ld, inner = x.stride()
    if inner != 1 and cols > 1 and rows > 0:
        raise ValueError("%s needs unit stride along its second dimension" % name)
    return ld if rows > 1 else max(ld, cols)


def _shaped(name, x, rows, cols):
    r, c = x.shape
    if r != rows or c != cols:
        raise ValueError("%s must have shape %s, not %s" % (name, (rows, cols), tuple(x.shape)))


def _vector(name, x, dtype, n):
    if x.dtype is not dtype or x.ndim != 1 or not x.is_cuda:
        raise TypeError("%s must be a 1-D %s CUDA tensor" % (name, str(dtype).replace("torch.", "")))
    if x.shape[0] != n or (n > 1 and x.stride(0) != 1):
        raise ValueError("%s must hold %d contiguous values" % (name, n))


def _current(torch, x, *others):
    """The raw handle of the current stream of the device that all tensors are
    on, which has to be the current one."""
    d = x.get_device()
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError("tensors on different devices: cuda:%d and %s" % (d, t.device))
    current = torch._C._cuda_getDevice()
    if d != current:
        raise ValueError("tensors on cuda:%d, but the current device is cuda:%d" % (d, current))
    return torch._C._cuda_getCurrentRawStream(d)


_units = {}


def _compute_units(torch, d):
    if d not in _units:
        _units[d] = torch.cuda.get_device_properties(d).multi_processor_count
    return _units[d]


def _on_stream(stream, tensors, call):
    """``call`` with ``stream`` as the current stream, for which it then
    allocates; the tensors it reads are marked as used there."""
    import torch

    for t in tensors:
        if t is not None and t.is_cuda:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return call()


def _done(rc, name):
    if rc != GEMM_OK:
        raise GemmError(rc, name)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def gemm_fp8(A, scale_a, B, scale_b, *, out_dtype=None, out=None, exact=False, stream=None):
    """C = (A * scale_a) @ (B * scale_b).T for 8-bit A (M, K) and B (N, K).

    ``scale_a`` is (ceil(K / 128), M); ``scale_b`` is (ceil(K / 128), N) for a
    B quantised row by row or (ceil(K / 128), ceil(N / 128)) for one quantised
    in blocks.  Returns ``out`` (allocated if None) in ``out_dtype``, bfloat16
    (the default) or float32.

    A float32 result, one with K <= 256 and one with ``exact`` has fp32's sums.
    Other bfloat16 results take the 8-bit matrix instruction, up to 2.4 times as
    fast, which adds each run of 8 products along k on a grid of 2^-13 of the
    largest: 1.5e-5 of the result's norm on random operands, but all of a small
    product between large ones that cancel."""
    import torch

    if stream is not None:
        return _on_stream(stream, (A, scale_a, B, scale_b, out),
                          lambda: gemm_fp8(A, scale_a, B, scale_b, out_dtype=out_dtype, out=out, exact=exact))
    f8, f32, bf16 = torch.float8_e4m3fn, torch.float32, torch.bfloat16
    lda, ldb = _matrix("A", A, f8), _matrix("B", B, f8)
    (M, K), (N, KB) = A.shape, B.shape
    if KB != K:
        raise ValueError("inner dimensions differ: %d vs %d" % (K, KB))
    ldsa, ldsb = _matrix("scale_a", scale_a, f32), _matrix("scale_b", scale_b, f32)
    kb = _blocks(K)
    _shaped("scale_a", scale_a, kb, M)
    rows = 1 if scale_b.shape[1] == N else BLOCK
    _shaped("scale_b", scale_b, kb, N if rows == 1 else _blocks(N))
    if out_dtype is None:
        out_dtype = bf16 if out is None else out.dtype
    if out_dtype is not bf16 and out_dtype is not f32:
        raise TypeError("out_dtype must be bfloat16 or float32")
    s = _current(torch, A, B, scale_a, scale_b, out)
    if out is None:
        out, ldc = torch.empty(M, N, dtype=out_dtype, device=A.device), N
    else:
        ldc = _matrix("out", out, out_dtype)
        _shaped("out", out, M, N)
    _done(library().gemm_fp8_bt(M, N, K, A.data_ptr(), lda, scale_a.data_ptr(), ldsa, B.data_ptr(), ldb,
                                scale_b.data_ptr(), ldsb, rows, out.data_ptr(), ldc,
                                (TYPE_BF16 if out_dtype is bf16 else TYPE_FP32) + (FP8_EXACT if exact else 0), s),
          "gemm_fp8_bt")
    return out


def quantize_fp8(x, *, block_rows=1, transposed=False, stream=None):
    """(q, scale) of a bfloat16 matrix: e4m3 values with a scale for each row
    and block of 128 columns (``block_rows`` 1) or each 128 x 128 block (128),
    of x or, with ``transposed``, of its transpose."""
    import torch

    if stream is not None:
        return _on_stream(stream, (x,), lambda: quantize_fp8(x, block_rows=block_rows, transposed=transposed))
    ldx = _matrix("x", x, torch.bfloat16)
    M, K = x.shape
    if block_rows not in (1, BLOCK):
        raise ValueError("block_rows must be 1 or %d" % BLOCK)
    R, L = (K, M) if transposed else (M, K)
    cols, dev, s = R if block_rows == 1 else _blocks(R), x.device, _current(torch, x)
    q = torch.empty(R, L, dtype=torch.float8_e4m3fn, device=dev)
    scale = torch.empty(_blocks(L), cols, dtype=torch.float32, device=dev)
    _done(library().gemm_quantize_fp8(M, K, x.data_ptr(), ldx, q.data_ptr(), L, scale.data_ptr(), cols, block_rows,
                                      1 if transposed else 0, s), "gemm_quantize_fp8")
    return q, scale


def rms_norm(x, weight, *, residual=None, eps=1e-6, quantize=False, return_rstd=False, stream=None):
    """Root-mean-square norm of h = x + residual (h = x without one) times
    ``weight``, as an ``RmsNorm``: y in bfloat16 or, with ``quantize``, 8 bits
    and its row scales; h where there is a residual; 1 / rms of each row with
    ``return_rstd`` (the backward pass needs it)."""
    import torch

    if stream is not None:
        return _on_stream(stream, (x, weight, residual),
                          lambda: rms_norm(x, weight, residual=residual, eps=eps, quantize=quantize,
                                           return_rstd=return_rstd))
    bf16, f32 = torch.bfloat16, torch.float32
    ldx = _matrix("x", x, bf16)
    M, D = x.shape
    _vector("weight", weight, bf16, D)
    h, rstd, scale, ldr, dev = None, None, None, 0, x.device
    if residual is not None:
        ldr = _matrix("residual", residual, bf16)
        _shaped("residual", residual, M, D)
    s = _current(torch, x, weight, residual)
    if residual is not None:
        h = torch.empty(M, D, dtype=bf16, device=dev)
    if return_rstd:
        rstd = torch.empty(M, dtype=f32, device=dev)
    if quantize:
        y = torch.empty(M, D, dtype=torch.float8_e4m3fn, device=dev)
        scale = torch.empty(_blocks(D), M, dtype=f32, device=dev)
    else:
        y = torch.empty(M, D, dtype=bf16, device=dev)
    _done(library().gemm_rms_norm(M, D, x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr,
                                  weight.data_ptr(), eps, None if h is None else h.data_ptr(), D, y.data_ptr(), D,
                                  TYPE_FP8 if quantize else TYPE_BF16, None if scale is None else scale.data_ptr(), M,
                                  None if rstd is None else rstd.data_ptr(), s), "gemm_rms_norm")
    return RmsNorm(y, scale, h, rstd)


def rms_norm_backward(dy, h, weight, rstd, *, dresidual=None, stream=None):
    """(dx, dweight) of ``rms_norm`` for the gradient ``dy`` of y and, where h
    is used further on, the gradient ``dresidual`` that reaches it there.  h is
    the forward pass's h (its x without a residual) and rstd its result; dx
    (bfloat16) is the gradient of x and residual alike, dweight is float32."""
    import torch

    if stream is not None:
        return _on_stream(stream, (dy, h, weight, rstd, dresidual),
                          lambda: rms_norm_backward(dy, h, weight, rstd, dresidual=dresidual))
    bf16 = torch.bfloat16
    lddy, ldh = _matrix("dy", dy, bf16), _matrix("h", h, bf16)
    M, D = dy.shape
    _shaped("h", h, M, D)
    _vector("weight", weight, bf16, D)
    _vector("rstd", rstd, torch.float32, M)
    lddr, dev = 0, dy.device
    if dresidual is not None:
        lddr = _matrix("dresidual", dresidual, bf16)
        _shaped("dresidual", dresidual, M, D)
    s = _current(torch, dy, h, weight, rstd, dresidual)
    dx, dweight = torch.empty(M, D, dtype=bf16, device=dev), torch.empty(D, dtype=torch.float32, device=dev)
    args = (M, D, dy.data_ptr(), lddy, h.data_ptr(), ldh, weight.data_ptr(), rstd.data_ptr(),
            None if dresidual is None else dresidual.data_ptr(), lddr, dx.data_ptr(), D, dweight.data_ptr())
    rc = library().gemm_rms_norm_bwd_given(*args, None, 0, s)
    if rc == GEMM_ERR_SCRATCH:   # a capturing stream: see _linear_call
        n = gemm_rms_norm_bwd_scratch_cus(M, D, _compute_units(torch, dy.get_device()))
        w = torch.empty(n, dtype=torch.uint8, device=dev)
        rc = library().gemm_rms_norm_bwd_given(*args, w.data_ptr(), n, s)
    _done(rc, "gemm_rms_norm_bwd")
    return dx, dweight


def _gated(gu):
    M, F2 = gu.shape
    if F2 % 2:
        raise ValueError("gu must have an even number of columns")
    return M, F2 // 2


def swiglu(gu, *, quantize=False, stream=None):
    """silu(g) * u for gu = [g, u] side by side (M, 2F): y (M, F) in bfloat16
    or, with ``quantize``, the pair of 8-bit y and its row scales."""
    import torch

    if stream is not None:
        return _on_stream(stream, (gu,), lambda: swiglu(gu, quantize=quantize))
    ldgu, dev = _matrix("gu", gu, torch.bfloat16), gu.device
    M, F = _gated(gu)
    s = _current(torch, gu)
    if not quantize:
        y = torch.empty(M, F, dtype=torch.bfloat16, device=dev)
        _done(library().gemm_swiglu(M, F, gu.data_ptr(), ldgu, y.data_ptr(), F, TYPE_BF16, None, 0, s), "gemm_swiglu")
        return y
    q = torch.empty(M, F, dtype=torch.float8_e4m3fn, device=dev)
    scale = torch.empty(_blocks(F), M, dtype=torch.float32, device=dev)
    _done(library().gemm_swiglu(M, F, gu.data_ptr(), ldgu, q.data_ptr(), F, TYPE_FP8, scale.data_ptr(), M, s),
          "gemm_swiglu")
    return q, scale


def swiglu_backward(dy, gu, *, stream=None):
    """The gradient of gu = [g, u] (bfloat16, (M, 2F)) for the gradient dy (M, F) of ``swiglu``."""
    import torch

    if stream is not None:
        return _on_stream(stream, (dy, gu), lambda: swiglu_backward(dy, gu))
    ldgu, lddy = _matrix("gu", gu, torch.bfloat16), _matrix("dy", dy, torch.bfloat16)
    M, F = _gated(gu)
    _shaped("dy", dy, M, F)
    s = _current(torch, dy, gu)
    dgu = torch.empty(M, 2 * F, dtype=torch.bfloat16, device=gu.device)
    _done(library().gemm_swiglu_bwd(M, F, dy.data_ptr(), lddy, gu.data_ptr(), ldgu, dgu.data_ptr(), 2 * F, s),
          "gemm_swiglu_bwd")
    return dgu


# -- linear layers on bf16 operands -------------------------------------------------
# A weight has one row per output: (N, K), for x (M, K).  An activation is None,
# "relu", "gelu", "gelu_tanh" or "silu".  Streams and devices as above.
def _activation(name):
    if name not in ACTIVATIONS:
        raise ValueError("activation must be one of %s" % [a for a in ACTIVATIONS])
    return ACTIVATIONS[name]


def _optional(name, x, dtype, rows, cols):
    """(pointer, leading dimension) of an operand that may be None."""
    if x is None:
        return None, 0
    ld = _matrix(name, x, dtype)
    _shaped(name, x, rows, cols)
    return x.data_ptr(), ld


def _linear_call(torch, f, args, s, product, M, N, K, a, lda, b, ldb):
    """One entry point's call.  Where it needs temporary memory and the stream is
    capturing, again with some from torch, whose graphs keep theirs apart."""
    rc = f(*args, None, 0, s)
    if rc == GEMM_ERR_SCRATCH:
        even = lambda x, ld: x.data_ptr() % 16 == 0 and (x.shape[0] <= 1 or (ld % 8 == 0 and ld <= 1 << 22))  # noqa: E731
        plan = gemm_linear_plan_cus(M, N, K, product, even(a, lda), even(b, ldb),
                                    _compute_units(torch, a.get_device()))
        n = plan["scratch_bytes"]
        w = torch.empty(n, dtype=torch.uint8, device=a.device)
        rc = f(*args, w.data_ptr(), n, s)
        if rc == GEMM_ERR_SCRATCH:   # rows out of the tiles' reach
            n += plan["tiles"] * plan["rows"] * plan["cols"] * (8 if product == "gated_linear" else 4)
            w = torch.empty(n, dtype=torch.uint8, device=a.device)
            rc = f(*args, w.data_ptr(), n, s)
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_" + product)


def linear(x, weight, *, bias=None, activation=None, residual=None, return_preactivation=False, stream=None):
    """act(z) + residual with z = x @ weight.T + bias for x (M, K) and weight (N,
    K), the whole of it in the product's epilogue; with ``return_preactivation``
    the pair of it and z, which ``linear_backward_input`` reads.  All bfloat16."""
    import torch

    if stream is not None:
        return _on_stream(stream, (x, weight, bias, residual),
                          lambda: linear(x, weight, bias=bias, activation=activation, residual=residual,
                                         return_preactivation=return_preactivation))
    bf16, act = torch.bfloat16, _activation(activation)
    ldx, ldw = _matrix("x", x, bf16), _matrix("weight", weight, bf16)
    (M, K), (N, KW) = x.shape, weight.shape
    if KW != K:
        raise ValueError("inner dimensions differ: %d vs %d" % (K, KW))
    if bias is not None:
        _vector("bias", bias, bf16, N)
    r, ldr = _optional("residual", residual, bf16, M, N)
    s, dev = _current(torch, x, weight, bias, residual), x.device
    y = torch.empty(M, N, dtype=bf16, device=dev)
    z = torch.empty(M, N, dtype=bf16, device=dev) if return_preactivation else None
    _linear_call(torch, library().gemm_linear,
                 (M, N, K, x.data_ptr(), ldx, weight.data_ptr(), ldw, None if bias is None else bias.data_ptr(), act,
                  r, ldr, None if z is None else z.data_ptr(), N, y.data_ptr(), N), s, "linear", M, N, K, x, ldx,
                  weight, ldw)
    return (y, z) if return_preactivation else y


def linear_backward_input(dy, weight, *, preactivation=None, activation=None, dresidual=None, stream=None):
    """The gradient of ``linear``'s x (M, K) for the gradient dy (M, N) of its y,
    plus ``dresidual``, the gradient that reaches x in other ways; with an
    activation, x being act(preactivation), the gradient of preactivation:
    (dy @ weight + dresidual) * act'(preactivation).  bfloat16."""
    import torch

    if stream is not None:
        return _on_stream(stream, (dy, weight, preactivation, dresidual),
                          lambda: linear_backward_input(dy, weight, preactivation=preactivation, activation=activation,
                                                        dresidual=dresidual))
    bf16, act = torch.bfloat16, _activation(activation)
    lddy, ldw = _matrix("dy", dy, bf16), _matrix("weight", weight, bf16)
    (M, N), (NW, K) = dy.shape, weight.shape
    if NW != N:
        raise ValueError("dy has %d columns, weight %d rows" % (N, NW))
    if activation is None:
        preactivation = None      # its slope is 1 everywhere
    elif preactivation is None:
        raise ValueError("the gradient through an activation needs its preactivation")
    z, ldz = _optional("preactivation", preactivation, bf16, M, K)
    r, ldr = _optional("dresidual", dresidual, bf16, M, K)
    s = _current(torch, dy, weight, preactivation, dresidual)
    dx = torch.empty(M, K, dtype=bf16, device=dy.device)
    _linear_call(torch, library().gemm_linear_bwd_input,
                 (M, N, K, dy.data_ptr(), lddy, weight.data_ptr(), ldw, act, z, ldz, r, ldr, dx.data_ptr(), K), s,
                  "linear_bwd_input", M, N, K, dy, lddy, weight, ldw)
    return dx


def linear_backward_weight(dy, x, *, bias=False, out_dtype=None, stream=None):
    """The gradient dy.T @ x (N, K) of ``linear``'s weight for the gradient dy (M,
    N) of its z and its x (M, K), in ``out_dtype``, float32 (the default) or
    bfloat16; with ``bias`` the pair of it and the bias's, float32 (N,)."""
    import torch

    if stream is not None:
        return _on_stream(stream, (dy, x), lambda: linear_backward_weight(dy, x, bias=bias, out_dtype=out_dtype))
    bf16, f32 = torch.bfloat16, torch.float32
    if out_dtype is None:
        out_dtype = f32
    if out_dtype is not bf16 and out_dtype is not f32:
        raise TypeError("out_dtype must be bfloat16 or float32")
    lddy, ldx = _matrix("dy", dy, bf16), _matrix("x", x, bf16)
    (M, N), (MX, K) = dy.shape, x.shape
    if MX != M:
        raise ValueError("dy has %d rows, x %d" % (M, MX))
    s, dev = _current(torch, dy, x), dy.device
    dw = torch.empty(N, K, dtype=out_dtype, device=dev)
    db = torch.empty(N, dtype=f32, device=dev) if bias else None
    _linear_call(torch, library().gemm_linear_bwd_weight,
                 (M, N, K, dy.data_ptr(), lddy, x.data_ptr(), ldx, dw.data_ptr(), K,
                  TYPE_FP32 if out_dtype is f32 else TYPE_BF16, None if db is None else db.data_ptr()), s, "linear_bwd_weight", M, N, K, dy, lddy, x,
                  ldx)
    return (dw, db) if bias else dw


def gated_linear(x, weight, *, bias=None, activation="silu", return_gu=False, stream=None):
    """act(g) * u with [g, u] = x @ weight.T + bias for x (M, K) and weight (2F, K),
    the F rows of g and then the F rows of u: both projections and the gate in one
    kernel.  y (M, F); with ``return_gu`` the pair of it and [g, u] side by side (M,
    2F), which ``gated_linear_backward_input`` reads.  All bfloat16."""
    import torch

    if stream is not None:
        return _on_stream(stream, (x, weight, bias),
                          lambda: gated_linear(x, weight, bias=bias, activation=activation, return_gu=return_gu))
    bf16, act = torch.bfloat16, _activation(activation)
    ldx, ldw = _matrix("x", x, bf16), _matrix("weight", weight, bf16)
    (M, K), (F2, KW) = x.shape, weight.shape
    if KW != K:
        raise ValueError("inner dimensions differ: %d vs %d" % (K, KW))
    if F2 % 2:
        raise ValueError("weight must have an even number of rows")
    if bias is not None:
        _vector("bias", bias, bf16, F2)
    s, dev, F = _current(torch, x, weight, bias), x.device, F2 // 2
    y = torch.empty(M, F, dtype=bf16, device=dev)
    gu = torch.empty(M, F2, dtype=bf16, device=dev) if return_gu else None
    _linear_call(torch, library().gemm_gated_linear,
                 (M, F, K, x.data_ptr(), ldx, weight.data_ptr(), ldw, None if bias is None else bias.data_ptr(), act,
                  None if gu is None else gu.data_ptr(), F2, y.data_ptr(), F), s, "gated_linear", M, F, K, x, ldx,
                  weight, ldw)
    return (y, gu) if return_gu else y


def gated_linear_backward_input(dy, weight, gu, *, activation="silu", return_y=False, stream=None):
    """The gradient of gu = [g, u] (M, 2F) through the layer that reads ``gated_linear``'s
    y: dy (M, N) is the gradient of that layer's output and weight (N, F) its weight.
    With t = dy @ weight it is [t * u * act'(g), t * act(g)]; with ``return_y`` the
    pair of it and y again, which that weight's gradient reads.  bfloat16."""
    import torch

    if stream is not None:
        return _on_stream(stream, (dy, weight, gu),
                          lambda: gated_linear_backward_input(dy, weight, gu, activation=activation, return_y=return_y))
    bf16, act = torch.bfloat16, _activation(activation)
    lddy, ldw, ldgu = _matrix("dy", dy, bf16), _matrix("weight", weight, bf16), _matrix("gu", gu, bf16)
    (M, N), (NW, F) = dy.shape, weight.shape
    if NW != N:
        raise ValueError("dy has %d columns, weight %d rows" % (N, NW))
    _shaped("gu", gu, M, 2 * F)
    s, dev = _current(torch, dy, weight, gu), dy.device
    dgu = torch.empty(M, 2 * F, dtype=bf16, device=dev)
    y = torch.empty(M, F, dtype=bf16, device=dev) if return_y else None
    _linear_call(torch, library().gemm_gated_linear_bwd_input,
                 (M, F, N, dy.data_ptr(), lddy, weight.data_ptr(), ldw, act, gu.data_ptr(), ldgu, dgu.data_ptr(),
                  2 * F, None if y is None else y.data_ptr(), F), s, "gated_linear_bwd_input", M, F, N, dy, lddy, weight,
                  ldw)
    return (dgu, y) if return_y else dgu
