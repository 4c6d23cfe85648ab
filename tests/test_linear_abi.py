"""The linear layers' entry points without a GPU: what they refuse before any device
is touched, what they let through, the plans, and the formulas the GPU tests
compare with, checked against differences."""
import pytest
import torch

import linear_reference as ref
from pipelined_tiled_dense_amd import binding as bd

A0 = 1 << 30          # fake, aligned addresses 1 GiB apart: never dereferenced by these calls
X, W, B, R, Z, Y, V = (A0 * (i + 1) for i in range(7))
OK, BAD, MIS, SHAPE, DEVICE, ALIAS = (bd.GEMM_OK, bd.GEMM_ERR_INVALID_VALUE, bd.GEMM_ERR_MISALIGNED,
                                      bd.GEMM_ERR_UNSUPPORTED_SHAPE, bd.GEMM_ERR_DEVICE, bd.GEMM_ERR_ALIAS)
NONE, RELU, GELU, TANH, SILU = (bd.ACTIVATIONS[a] for a in ref.ACTS)


def linear(M=64, N=256, K=512, x=X, ldx=512, w=W, ldw=512, b=B, act=GELU, r=R, ldr=256, z=Z, ldz=256, y=Y, ldy=256):
    return bd.gemm_linear(M, N, K, x, ldx, w, ldw, b, act, r, ldr, z, ldz, y, ldy, None)


def dinput(M=64, N=256, K=512, dy=X, lddy=256, w=W, ldw=512, act=GELU, z=Z, ldz=512, r=R, ldr=512, dx=Y, lddx=512):
    return bd.gemm_linear_bwd_input(M, N, K, dy, lddy, w, ldw, act, z, ldz, r, ldr, dx, lddx, None)


def dweight(M=64, N=256, K=512, dy=X, lddy=256, x=W, ldx=512, dw=Y, lddw=512, t=bd.TYPE_FP32, db=V):
    return bd.gemm_linear_bwd_weight(M, N, K, dy, lddy, x, ldx, dw, lddw, t, db, None)


def gated(M=64, F=256, K=512, x=X, ldx=512, w=W, ldw=512, b=B, act=SILU, gu=Z, ldgu=512, y=Y, ldy=256):
    return bd.gemm_gated_linear(M, F, K, x, ldx, w, ldw, b, act, gu, ldgu, y, ldy, None)


def dgated(M=64, F=256, N=512, dy=X, lddy=512, w=W, ldw=256, act=SILU, gu=Z, ldgu=512, d=V, ldd=512, y=Y, ldy=256):
    return bd.gemm_gated_linear_bwd_input(M, F, N, dy, lddy, w, ldw, act, gu, ldgu, d, ldd, y, ldy, None)


BIG = (1 << 22) + 1
NARROW = (1 << 28) + 1
REFUSED = [
    # sizes, activations, types
    *((f, {k: -1}, BAD) for f in (linear, dinput, dweight) for k in "MNK"), (gated, {"F": -1}, BAD), (dgated, {"F": -1}, BAD),
    *((f, {"M": 1 << 31}, SHAPE) for f in (linear, dinput, dweight, gated, dgated)),
    *((f, {k: BIG}, SHAPE) for f in (linear, dinput, dweight) for k in "NK"), (gated, {"F": BIG}, SHAPE),
    (gated, {"K": BIG}, SHAPE), (dgated, {"F": BIG}, SHAPE), (dgated, {"N": BIG}, SHAPE),
    (linear, {"M": NARROW, "N": 7}, SHAPE), (dinput, {"M": NARROW, "K": 7}, SHAPE), (gated, {"M": NARROW, "F": 7}, SHAPE),
    (dgated, {"M": NARROW, "F": 1}, SHAPE),
    *((f, {"act": a}, BAD) for f in (linear, dinput, gated, dgated) for a in (-1, 5)),
    (dweight, {"t": bd.TYPE_FP8}, BAD), (dweight, {"t": 3}, BAD),
    # null pointers
    (linear, {"x": None}, BAD), (linear, {"w": None}, BAD), (linear, {"y": None}, BAD), (dinput, {"dy": None}, BAD),
    (dinput, {"w": None}, BAD), (dinput, {"z": None}, BAD), (dinput, {"dx": None}, BAD), (dweight, {"dy": None}, BAD),
    (dweight, {"x": None}, BAD), (dweight, {"dw": None}, BAD), (gated, {"x": None}, BAD), (gated, {"w": None}, BAD),
    (gated, {"y": None}, BAD), (dgated, {"dy": None}, BAD), (dgated, {"w": None}, BAD), (dgated, {"gu": None}, BAD),
    (dgated, {"d": None}, BAD), (linear, {"K": 0, "x": None, "w": None, "y": None}, BAD),
    # leading dimensions
    *((linear, {k: v}, BAD) for k, v in (("ldx", 511), ("ldw", 511), ("ldr", 255), ("ldz", 255), ("ldy", 255))),
    *((dinput, {k: v}, BAD) for k, v in (("lddy", 255), ("ldw", 511), ("ldz", 511), ("ldr", 511), ("lddx", 511))),
    *((dweight, {k: v}, BAD) for k, v in (("lddy", 255), ("ldx", 511), ("lddw", 511))),
    *((gated, {k: v}, BAD) for k, v in (("ldx", 511), ("ldw", 0), ("ldgu", 511), ("ldy", 255))),
    *((dgated, {k: v}, BAD) for k, v in (("lddy", 511), ("ldw", 255), ("ldgu", 511), ("ldd", 511), ("ldy", 255))),
    (linear, {"ldx": 1 << 31}, BAD), (dgated, {"ldd": 1 << 40}, BAD),
    # alignment
    *((linear, {k: a + 1}, MIS) for k, a in (("x", X), ("w", W), ("b", B), ("r", R), ("z", Z), ("y", Y))),
    *((dinput, {k: a + 1}, MIS) for k, a in (("dy", X), ("w", W), ("z", Z), ("r", R), ("dx", Y))),
    (dweight, {"dy": X + 1}, MIS), (dweight, {"x": W + 1}, MIS), (dweight, {"dw": Y + 2}, MIS), (dweight, {"db": V + 2}, MIS),
    (dweight, {"dw": Y + 1, "t": bd.TYPE_BF16}, MIS), (gated, {"gu": Z + 1}, MIS), (gated, {"b": B + 1}, MIS),
    (dgated, {"gu": Z + 1}, MIS), (dgated, {"d": V + 1}, MIS), (dgated, {"y": Y + 1}, MIS),
    # outputs over inputs or over each other
    *((linear, {"y": a}, ALIAS) for a in (X, W, B + 64, R + 2, Z)), *((linear, {"z": a}, ALIAS) for a in (X, W, B, R, Y + 512)),
    (linear, {"y": R, "ldy": 264}, ALIAS), (linear, {"x": R, "y": R, "N": 512, "ldr": 512, "ldy": 512, "ldz": 512}, ALIAS),
    *((dinput, {"dx": a}, ALIAS) for a in (X, W, Z + 2, R + 2)), (dinput, {"dx": Z, "lddx": 520}, ALIAS),
    (dinput, {"dx": Z, "r": Z + 1024}, ALIAS),
    (dweight, {"dw": X}, ALIAS), (dweight, {"dw": W + 4}, ALIAS), (dweight, {"db": X}, ALIAS), (dweight, {"db": W}, ALIAS),
    (dweight, {"db": Y + 1024}, ALIAS), *((gated, {"y": a}, ALIAS) for a in (X, W, B, Z)),
    *((gated, {"gu": a}, ALIAS) for a in (X, W, B)), *((dgated, {"d": a}, ALIAS) for a in (X, W, Z + 2, Y)),
    (dgated, {"d": Z, "ldd": 520}, ALIAS), *((dgated, {"y": a}, ALIAS) for a in (X, W, Z)),
]


@pytest.mark.parametrize("fn,kw,want", REFUSED, ids=lambda v: getattr(v, "__name__", None) or str(v)[:60])
def test_refused(fn, kw, want):
    assert fn(**kw) == want


def test_workspace_refused():
    """A workspace off the 256-byte grid, of negative size, or over an operand."""
    from pipelined_tiled_dense_amd.binding import gemm_linear as call
    args = (64, 256, 512, X, 512, W, 512, B, GELU, R, 256, Z, 256, Y, 256, None)
    assert call(*args, V + 16, 4096) == MIS and call(*args, V, -1) == BAD
    for a in (X, W, B, R, Z, Y):
        assert call(*args, a - 256, 4096) == ALIAS
    assert bd.gemm_linear_bwd_weight(64, 256, 512, X, 256, W, 512, Y, 512, bd.TYPE_FP32, V, None, V - 256, 4096) == ALIAS
    if not torch.cuda.is_available():
        assert call(*args, V, 4096) == DEVICE and call(*args, V, 0) == DEVICE


def test_nothing_to_do():
    assert linear(M=0, x=None, y=None) == OK and linear(N=0, w=None, y=None) == OK
    assert dinput(M=0, dy=None, dx=None) == OK and dinput(K=0, w=None, dx=None) == OK
    assert dweight(N=0, dy=None, dw=None) == OK and dweight(K=0, x=None, dw=None, db=None) == OK
    assert gated(M=0, y=None) == OK and gated(F=0, w=None, y=None) == OK
    assert dgated(M=0, d=None) == OK and dgated(F=0, gu=None, d=None) == OK


ACCEPTED = [
    (linear, {}), (linear, {"b": None, "r": None, "z": None, "act": NONE}), (linear, {"y": R}), (linear, {"x": X + 2, "K": 511}),
    (linear, {"K": 0, "x": None, "w": None}), (linear, {"M": 1, "ldx": 0, "ldy": 0, "ldr": 0, "ldz": 0}),
    (linear, {"r": None, "ldr": -5}), (linear, {"r": X, "N": 512, "ldr": 512, "ldy": 512, "ldz": 512}),
    (dinput, {}), (dinput, {"act": NONE, "z": None}), (dinput, {"dx": Z}), (dinput, {"dx": R}), (dinput, {"dx": Z, "r": Z}),
    (dinput, {"act": NONE, "z": Y}), (dinput, {"N": 0, "dy": None, "w": None}), (dinput, {"r": None}),
    (dweight, {}), (dweight, {"db": None}), (dweight, {"t": bd.TYPE_BF16, "dw": Y + 2}), (dweight, {"M": 0, "dy": None, "x": None}),
    (dweight, {"K": 0, "x": None, "dw": None}), (dweight, {"x": X, "N": 512, "lddy": 512}),
    (gated, {}), (gated, {"b": None, "gu": None, "act": NONE}), (gated, {"K": 0, "x": None, "w": None}),
    (dgated, {}), (dgated, {"y": None}), (dgated, {"d": Z}), (dgated, {"N": 0, "dy": None, "w": None}),
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
    for name, code in bd.ACTIVATIONS.items():
        assert value("GEMM_ACT_%s" % (name or "none").upper()) == code
    for name, code in bd.LINEAR_PRODUCTS.items():
        assert value("GEMM_%s" % name.upper()) == code


def test_tensor_functions_refuse_what_they_cannot_take():
    """Host tensors, types and ranks, and names of activations: refused by the binding
    before any call."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: bd.linear(x, x), lambda: bd.linear_backward_input(x, x), lambda: bd.linear_backward_weight(x, x),
                 lambda: bd.gated_linear(x, x), lambda: bd.gated_linear_backward_input(x, x, x),
                 lambda: bd.linear_backward_weight(x, x, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        bd.linear(x, x, activation="swish")


# -- plans ---------------------------------------------------------------------------
def plan(M, N, K, product, a=True, b=True, cus=256):
    return bd.gemm_linear_plan_cus(M, N, K, product, a, b, cus)


@pytest.mark.parametrize("product", list(bd.LINEAR_PRODUCTS))
@pytest.mark.parametrize("M", [1, 5, 17, 40, 65, 300, 2047, 9000])
@pytest.mark.parametrize("cus", [1, 64, 256])
def test_plans_cover_the_product(product, M, cus):
    """Every output and every term in some workgroup's part, nothing in two; the sums'
    memory as large as the launches take it to be."""
    for N, K in ((1, 8), (7, 3), (8, 8), (64, 4096), (1000, 520), (4100, 65), (33, 20000)):
        p = plan(M, N, K, product, cus=cus)
        rows, cols, terms = {"linear": (M, N, K), "linear_bwd_input": (M, K, N), "linear_bwd_weight": (N, K, M),
                             "gated_linear": (M, N, K), "gated_linear_bwd_input": (M, N, K)}[product]
        assert p["tiles"] == -(-rows // p["rows"]) * -(-cols // p["cols"])
        assert p["k_splits"] == -(-terms // p["k_chunk"]) and (p["k_splits"] == 1 or p["k_chunk"] % 64 == 0)
        factors = 2 if product == "gated_linear" else 1
        want = p["tiles"] * p["k_splits"] * p["rows"] * p["cols"] * factors * 4 if p["k_splits"] > 1 else 0
        assert p["workspace_bytes"] == want
        assert p["scratch_bytes"] >= want + p["pad_bytes"]
        if p["waves_share_k"]:
            assert p["grid"] >= p["tiles"] * p["k_splits"] and p["pad_bytes"] == 0
        else:
            assert 1 <= p["grid"] <= max(cus, 1) and cols >= 8
            if product == "linear":
                assert (p["pad_bytes"] > 0) == (K % 8 != 0)
                assert plan(M, N, K, product, a=False, b=False, cus=cus)["pad_bytes"] >= 2 * (M + N) * K or \
                    plan(M, N, K, product, a=False, b=False, cus=cus)["waves_share_k"]


def test_plan_kinds_and_refusals():
    assert plan(1, 4096, 8192, "linear")["waves_share_k"] == 1
    assert plan(8192, 8192, 8192, "linear")["rows"] == 256
    assert plan(2048, 2048, 2048, "linear")["rows"] == 128
    assert plan(32768, 1024, 1024, "linear_bwd_weight")["k_splits"] > 1
    p = plan(20000, 100, 5, "linear_bwd_weight")
    assert p["scratch_bytes"] >= p["workspace_bytes"] + 100 * 4 * 2
    assert all(v == 0 for v in plan(0, 5, 5, "linear").values()) and all(v == 0 for v in plan(5, 5, 0, "linear").values())
    for args in ((1, 1, 1, 5), (1, 1, 1, -1)):
        with pytest.raises(bd.GemmError):
            bd.gemm_linear_plan_cus(*args, 1, 1, 256)
    with pytest.raises(bd.GemmError):
        plan(1, 1, 1, "linear", cus=0)
    assert bd.library().gemm_linear_plan_cus(1, 1, 1, 0, 1, 1, 256, None) == BAD


# -- the formulas -------------------------------------------------------------------
def change(f, x, v, step=1e-5):
    return float((f(x + step * v) - f(x - step * v)).sum() / (2 * step))


@pytest.mark.parametrize("act", ref.ACTS)
def test_reference_gradients_against_differences(act):
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    z0, w, dy, res = r(5, 7), r(9, 7) / 3, r(5, 9), r(5, 7)
    value = lambda z: ref.activation(z, act)[0]  # noqa: E731
    dz = ref.linear_backward_input(dy, w, z0, act, res)[0]
    for _ in range(3):
        v = r(5, 7)
        # y = act(z) w^T, and res what reaches act(z) otherwise.
        assert change(lambda z: (value(z) @ w.t() * dy).sum() + (value(z) * res).sum(), z0, v) == pytest.approx(
            float((dz * v).sum()), rel=1e-6, abs=1e-8)
    gu = r(5, 14)
    dgu = ref.gated_backward_input(dy, w, gu, act)["dgu"][0]
    for _ in range(3):
        v = r(5, 14)
        assert change(lambda t: (value(t[:, :7]) * t[:, 7:]) @ w.t() * dy, gu, v) == pytest.approx(
            float((dgu * v).sum()), rel=1e-6, abs=1e-8)
    x, dw = r(5, 7), r(9, 7)
    grad = ref.product(dy.t(), x)[0]
    assert change(lambda t: (x @ t.t()) * dy, w, dw) == pytest.approx(float((grad * dw).sum()), rel=1e-6)


def test_reference_activations():
    """Against torch's own functions, in 64 bits."""
    z = torch.linspace(-12, 12, 400, dtype=torch.float64)
    f = torch.nn.functional
    for act, want in ((None, z), ("relu", z.relu()), ("gelu", f.gelu(z)), ("gelu_tanh", f.gelu(z, approximate="tanh")),
                      ("silu", f.silu(z))):
        assert torch.allclose(ref.activation(z, act)[0], want, rtol=1e-9, atol=1e-14)
        assert float(ref.activation(z, act)[1].abs().max()) < ref.STEEPEST


def test_check_rejects_a_step():
    """The check takes the nearest bf16 value and rejects the one beyond it."""
    g = torch.Generator().manual_seed(1)
    y = torch.randn(50, 60, generator=g, dtype=torch.float64)
    b = ref.rounded(y, torch.zeros_like(y))
    q = y.to(torch.bfloat16)
    ref.check(q, y, b)
    bad = q.clone()
    bad.view(torch.int16)[7, 9] += 2
    with pytest.raises(AssertionError):
        ref.check(bad, y, b)
    bad = q.clone()
    bad[3, 3] = float("nan")
    with pytest.raises(AssertionError):
        ref.check(bad, y, b)


@pytest.mark.parametrize("product", list(bd.LINEAR_PRODUCTS))
@pytest.mark.parametrize("cols", [1, 7, 8, 100])
@pytest.mark.parametrize("even", [0, 1])
def test_launches_stay_below_their_limit(product, cols, even):
    """A launch holds fewer than 2^32 threads, at the most rows that are taken."""
    rows = 1 << 22 if product == "linear_bwd_weight" else 1 << 28 if cols < 8 else (1 << 31) - 1
    for inner in (1, 64, 1000):
        sizes = {"linear_bwd_input": (rows, inner, cols), "linear_bwd_weight": (inner, rows, cols)}.get(product, (rows, cols, inner))
        p = plan(*sizes, product, even, even)
        assert p["grid"] * p["threads"] < 1 << 32, p
    if product != "linear_bwd_weight" and cols < 8:
        more = {"linear_bwd_input": (NARROW, 64, cols)}.get(product, (NARROW, cols, 64))
        with pytest.raises(bd.GemmError):
            plan(*more, product, even, even)
