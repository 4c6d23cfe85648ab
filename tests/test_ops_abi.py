"""The 8-bit operators' entry points without a GPU: what they refuse, before
any device is touched, what they let through, and the formulas the GPU tests
compare with, checked in 64 bits against differences and against each other."""
import pytest
import torch

import ops_reference as ref
from pipelined_tiled_dense_amd import binding as bd

A0 = 1 << 30          # fake, aligned addresses 1 GiB apart: never dereferenced by these calls
X, Y, Z, W, V, U = (A0 * (i + 1) for i in range(6))
OK, BAD, MIS, SHAPE, DEVICE, ALIAS = (bd.GEMM_OK, bd.GEMM_ERR_INVALID_VALUE, bd.GEMM_ERR_MISALIGNED,
                                      bd.GEMM_ERR_UNSUPPORTED_SHAPE, bd.GEMM_ERR_DEVICE, bd.GEMM_ERR_ALIAS)


def gemm(M=64, N=256, K=512, A=X, lda=512, SA=Y, ldsa=64, B=Z, ldb=512, SB=W, ldsb=2, rows=128, C=V, ldc=256,
         ctype=bd.TYPE_BF16):
    return bd.gemm_fp8_bt(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, rows, C, ldc, ctype, None)


def quantize(M=64, K=512, x=X, ldx=512, q=Y, ldq=512, s=Z, lds=64, rows=1, t=0):
    return bd.gemm_quantize_fp8(M, K, x, ldx, q, ldq, s, lds, rows, t, None)


def norm(M=64, D=512, x=X, ldx=512, r=Y, ldr=512, w=Z, eps=1e-6, h=W, ldh=512, y=V, ldy=512, yt=bd.TYPE_BF16, s=None,
         lds=0, rstd=None):
    return bd.gemm_rms_norm(M, D, x, ldx, r, ldr, w, eps, h, ldh, y, ldy, yt, s, lds, rstd, None)


def norm_bwd(M=64, D=512, dy=X, lddy=512, h=Y, ldh=512, w=Z, rstd=W, s=None, lds=512, dx=V, lddx=512, dw=U):
    return bd.gemm_rms_norm_bwd(M, D, dy, lddy, h, ldh, w, rstd, s, lds, dx, lddx, dw, None)


def swiglu(M=64, F=512, gu=X, ldgu=1024, y=Y, ldy=512, yt=bd.TYPE_FP8, s=Z, lds=64):
    return bd.gemm_swiglu(M, F, gu, ldgu, y, ldy, yt, s, lds, None)


def swiglu_bwd(M=64, F=512, dy=X, lddy=512, gu=Y, ldgu=1024, d=Z, ldd=1024):
    return bd.gemm_swiglu_bwd(M, F, dy, lddy, gu, ldgu, d, ldd, None)


REFUSED = [
    # sizes, types, block sizes
    (gemm, {"M": -1}, BAD), (gemm, {"K": -1}, BAD), (gemm, {"rows": 64}, BAD), (gemm, {"ctype": bd.TYPE_FP8}, BAD),
    (gemm, {"ctype": 9}, BAD), (gemm, {"N": (1 << 22) + 1}, SHAPE), (gemm, {"K": (1 << 22) + 1}, SHAPE),
    (gemm, {"M": 1 << 31}, SHAPE), (quantize, {"rows": 2}, BAD), (quantize, {"M": -1}, BAD),
    (quantize, {"K": 1 << 31}, SHAPE), (norm, {"D": 0}, BAD), (norm, {"D": bd.NORM_MAX_WIDTH + 1}, SHAPE),
    (norm, {"yt": bd.TYPE_FP32}, BAD), (norm, {"eps": -1.0}, BAD), (norm, {"eps": float("nan")}, BAD),
    (norm, {"eps": float("inf")}, BAD), (norm_bwd, {"D": 0}, BAD), (norm_bwd, {"M": -2}, BAD),
    (norm_bwd, {"D": bd.NORM_MAX_WIDTH + 1}, SHAPE), (swiglu, {"F": -1}, BAD), (swiglu, {"yt": bd.TYPE_FP32}, BAD),
    (swiglu, {"F": 1 << 30}, SHAPE), (swiglu_bwd, {"M": -1}, BAD),
    # null pointers
    (gemm, {"A": None}, BAD), (gemm, {"SA": None}, BAD), (gemm, {"SB": None}, BAD), (gemm, {"C": None}, BAD),
    (quantize, {"q": None}, BAD), (quantize, {"s": None}, BAD), (norm, {"x": None}, BAD), (norm, {"w": None}, BAD),
    (norm, {"h": None}, BAD), (norm, {"y": None}, BAD), (norm, {"yt": bd.TYPE_FP8}, BAD), (norm_bwd, {"dw": None}, BAD),
    (norm_bwd, {"rstd": None}, BAD), (norm_bwd, {"dx": None}, BAD), (swiglu, {"s": None}, BAD),
    (swiglu_bwd, {"d": None}, BAD),
    # leading dimensions
    (gemm, {"lda": 511}, BAD), (gemm, {"ldb": 500}, BAD), (gemm, {"ldc": 255}, BAD), (gemm, {"ldsa": 63}, BAD),
    (gemm, {"ldsb": 1}, BAD), (gemm, {"rows": 1, "ldsb": 255}, BAD), (gemm, {"lda": 1 << 32}, BAD),
    (quantize, {"ldq": 511}, BAD), (quantize, {"lds": 63}, BAD), (quantize, {"t": 1, "ldq": 63, "lds": 512}, BAD),
    (quantize, {"t": 1, "ldq": 512, "M": 300, "lds": 511}, BAD), (norm, {"ldx": 100}, BAD), (norm, {"ldh": 511}, BAD),
    (norm, {"yt": bd.TYPE_FP8, "s": U, "lds": 63}, BAD), (norm_bwd, {"ldh": 0}, BAD), (swiglu, {"ldgu": 1023}, BAD),
    (swiglu_bwd, {"ldd": 1000}, BAD),
    # alignment
    (gemm, {"SA": Y + 2}, MIS), (gemm, {"C": V + 1}, MIS), (gemm, {"C": V + 2, "ctype": bd.TYPE_FP32}, MIS),
    (quantize, {"x": X + 1}, MIS), (quantize, {"s": Z + 2}, MIS), (norm, {"w": Z + 1}, MIS),
    (norm, {"rstd": U + 2}, MIS), (norm_bwd, {"dw": U + 1}, MIS), (swiglu, {"gu": X + 1}, MIS),
    # outputs over inputs or over each other
    (gemm, {"C": X + 64}, ALIAS), (gemm, {"C": W}, ALIAS), (quantize, {"q": X}, ALIAS), (quantize, {"s": Y}, ALIAS),
    (norm, {"h": X + 16}, ALIAS), (norm, {"h": X, "ldh": 520}, ALIAS), (norm, {"y": W}, ALIAS), (norm, {"y": Y}, ALIAS),
    (norm, {"h": X, "y": X}, ALIAS), (norm, {"y": Z}, ALIAS), (norm, {"yt": bd.TYPE_FP8, "y": X, "s": U, "lds": 64}, ALIAS),
    (norm, {"rstd": V}, ALIAS), (norm_bwd, {"dx": Y}, ALIAS), (norm_bwd, {"dx": X, "lddx": 640}, ALIAS),
    (norm_bwd, {"dw": Z}, ALIAS), (norm_bwd, {"dw": V}, ALIAS), (swiglu, {"y": X + 1024}, ALIAS), (swiglu, {"s": X}, ALIAS),
    (swiglu_bwd, {"d": X}, ALIAS), (swiglu_bwd, {"d": Y + 16}, ALIAS),
]


@pytest.mark.parametrize("fn,kw,want", REFUSED, ids=lambda v: getattr(v, "__name__", None) or str(v)[:60])
def test_refused(fn, kw, want):
    assert fn(**kw) == want


def test_nothing_to_do():
    assert gemm(M=0, A=None, SA=None, C=None) == OK and gemm(N=0, B=None, C=None) == OK
    assert quantize(M=0, x=None) == OK and quantize(K=0, q=None) == OK
    assert norm(M=0, x=None, y=None) == OK
    assert swiglu(M=0, gu=None) == OK and swiglu(F=0, y=None) == OK and swiglu_bwd(F=0, d=None) == OK


ACCEPTED = [
    (gemm, {}), (gemm, {"K": 511}), (gemm, {"A": X + 1, "B": Z + 3}), (gemm, {"K": 0, "A": None, "SA": None, "B": None}),
    (gemm, {"M": 1, "lda": 0, "ldc": 0}), (gemm, {"rows": 1, "ldsb": 256}), (gemm, {"ctype": bd.TYPE_FP32}),
    (quantize, {}), (quantize, {"t": 1, "ldq": 64, "lds": 512}), (quantize, {"rows": 128, "lds": 1}),
    (quantize, {"rows": 128, "t": 1, "ldq": 64, "lds": 4}), (norm, {}), (norm, {"h": X}), (norm, {"h": Y}),
    (norm, {"y": X}), (norm, {"r": None, "h": None}), (norm, {"r": None, "h": None, "y": X}), (norm, {"rstd": U}),
    (norm, {"yt": bd.TYPE_FP8, "s": U, "lds": 64}), (norm, {"x": X + 2, "eps": 0.0}), (norm_bwd, {}),
    (norm_bwd, {"dx": X}), (norm_bwd, {"s": 7 * A0}), (norm_bwd, {"s": 7 * A0, "dx": 7 * A0}),
    (norm_bwd, {"M": 0, "dy": None}), (swiglu, {}), (swiglu, {"yt": bd.TYPE_BF16, "s": None}), (swiglu_bwd, {}),
    (swiglu_bwd, {"d": Y}),
]


@pytest.mark.parametrize("fn,kw", ACCEPTED, ids=lambda v: getattr(v, "__name__", None) or str(v)[:60])
def test_accepted_calls_reach_the_device_query(fn, kw):
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible; these calls would launch on fake addresses")
    assert fn(**kw) == DEVICE


def test_constants_match_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gemm_bf16.h")).read()
    value = lambda n: int(re.search(r"\b%s = (\d+)" % n, text).group(1))  # noqa: E731
    assert (value("GEMM_TYPE_BF16"), value("GEMM_TYPE_FP8"), value("GEMM_TYPE_FP32")) == (
        bd.TYPE_BF16, bd.TYPE_FP8, bd.TYPE_FP32)
    assert value("GEMM_NORM_MAX_WIDTH") == bd.NORM_MAX_WIDTH


def test_tensor_functions_refuse_what_they_cannot_take():
    """Host tensors, types, ranks: refused by the binding before any call."""
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.ones(256, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 256).to(torch.float8_e4m3fn), torch.ones(2, 4)
    for call in (lambda: bd.rms_norm(x, w), lambda: bd.rms_norm_backward(x, x, w, torch.ones(4)), lambda: bd.swiglu(x),
                 lambda: bd.swiglu_backward(x[:, :128], x), lambda: bd.quantize_fp8(x),
                 lambda: bd.gemm_fp8(q, s, q, s)):
        with pytest.raises(TypeError):
            call()


# -- the formulas -------------------------------------------------------------------
def change(f, x, v, step=1e-5):
    return float((f(x + step * v) - f(x - step * v)).sum() / (2 * step))


def test_reference_gradients_against_differences():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    h, w, dy, e = r(5, 70), r(70), r(5, 70), r(5, 70)
    rstd = ref.rms_norm(h, None, w, 1e-5)[1]
    dx, dw = ref.rms_norm_bwd(dy, h, w, rstd, e)
    for _ in range(3):
        v, u = r(5, 70), r(70)
        assert change(lambda t: ref.rms_norm(t, None, w, 1e-5)[2] * dy + t * e, h, v) == pytest.approx(
            float((dx * v).sum()), rel=1e-6, abs=1e-8)
        assert change(lambda t: ref.rms_norm(h, None, t, 1e-5)[2] * dy, w, u) == pytest.approx(
            float((dw * u).sum()), rel=1e-6, abs=1e-8)
    gu, d = r(5, 140), r(5, 70)
    for _ in range(3):
        v = r(5, 140)
        assert change(lambda t: ref.swiglu(t) * d, gu, v) == pytest.approx(
            float((ref.swiglu_bwd(d, gu) * v).sum()), rel=1e-6, abs=1e-8)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantized_check_accepts_the_nearest_values_and_nothing_else(block_rows):
    """The check the GPU results go through: it takes e4m3 values nearest to
    y / scale, and rejects a value one step off, a scale a step off, and scales
    of the wrong block."""
    g = torch.Generator().manual_seed(1)
    y = torch.randn(200, 300, generator=g, dtype=torch.float64)
    scale = ref.quantized_scale(y, block_rows).float()
    q = (y / ref.spread(scale.double(), block_rows, y.shape)).float().to(torch.float8_e4m3fn)
    ref.check_quantized(q, scale, y, block_rows, 0.0)
    bad = q.clone()
    bad.view(torch.uint8)[7, 9] += 2
    with pytest.raises(AssertionError):
        ref.check_quantized(bad, scale, y, block_rows, 0.0)
    with pytest.raises(AssertionError):
        ref.check_quantized(q, scale * 1.001, y, block_rows, 0.0)
    with pytest.raises(AssertionError):
        ref.check_quantized(q, scale.flip(0), y, block_rows, 0.0)


def test_exact_sums_are_a_flag_of_the_product_alone():
    """GEMM_FP8_EXACT goes with both of the product's types and with nothing else."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gemm_bf16.h")).read()
    assert int(re.search(r"GEMM_FP8_EXACT = (\d+)", text).group(1)) == bd.FP8_EXACT
    assert gemm(ctype=bd.TYPE_FP8 | bd.FP8_EXACT) == BAD and gemm(ctype=bd.FP8_EXACT * 2) == BAD
    assert norm(yt=bd.TYPE_BF16 | bd.FP8_EXACT) == BAD and swiglu(yt=bd.TYPE_FP8 | bd.FP8_EXACT) == BAD
    if not torch.cuda.is_available():
        assert gemm(ctype=bd.TYPE_BF16 | bd.FP8_EXACT) == DEVICE and gemm(ctype=bd.TYPE_FP32 | bd.FP8_EXACT) == DEVICE


def test_overlap_of_the_largest_strides():
    """An output whose rows span more bytes than 63 bits count still meets what lies
    behind it."""
    m = (1 << 31) - 1
    assert gemm(M=m, ldsa=m, C=A0 // 2, ldc=m, ctype=bd.TYPE_FP32) == ALIAS
    assert gemm(M=m, ldsa=m, C=A0 // 2, ldc=m) == ALIAS
    assert quantize(M=m, x=A0 // 2, ldx=m, lds=m) == ALIAS
