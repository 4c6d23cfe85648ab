"""Which kernel an 8-bit product takes, without a GPU (gemm_fp8_plan_cus): that the
sizes the GPU tests run reach the kernels they are there for, and that every plan
is one that can be launched."""
import random

import pytest

from gemm_fp8_cases import CASES
from pipelined_tiled_dense_amd import binding as bd

CUS = 256   # MI355X


def plan(M, N, K, b_rows=128, exact=False, a=True, b=True, fp32=False, cus=CUS):
    c_type = (bd.TYPE_FP32 if fp32 else bd.TYPE_BF16) | (bd.FP8_EXACT if exact else 0)
    return bd.gemm_fp8_plan_cus(M, N, K, b_rows, c_type, a, b, cus)


def cdiv(a, b):
    return -(-a // b)


@pytest.mark.parametrize("case,want", CASES, ids=lambda v: "-".join(str(int(x)) for x in v))
def test_sizes_reach_their_kernels(case, want):
    M, N, K, b_rows, exact, a, b = case
    p = plan(M, N, K, b_rows, exact, a, b)
    places = CUS * (1 if p["rows"] == 256 or p["few_rows"] else 2)
    many = not p["few_rows"] and p["tiles"] * p["k_splits"] > places
    assert (bool(p["few_rows"]), p["rows"], p["cols"], p["k_splits"] > 1, many) == want
    assert p["exact"] == exact


def test_the_cases_cover_every_kernel():
    """Each kernel with both kinds of B's scales somewhere, and each form of tiles
    with a padded copy of A, of B, of both for their alignment and for K."""
    seen, padded = set(), set()
    for (M, N, K, b_rows, exact, a, b), (few, rows, cols, chunks, _) in CASES:
        seen.add((few, rows, cols, exact, b_rows))
        if not few:
            padded.add((rows, exact, "k" if K % 16 else (a, b)))
    shapes = [(True, 16, 16), (True, 16, 32), (True, 32, 32), (True, 64, 32), (False, 128, 128)]
    for s in shapes:
        assert {s + (e, r) for e in (False, True) for r in (1, 128)} <= seen, s
    assert {(False, 256, 256, False, r) for r in (1, 128)} | {(True, 64, 64, False, 128)} <= seen
    for rows, exact in ((128, False), (128, True), (256, False)):
        assert {(rows, exact, "k"), (rows, exact, (False, True)), (rows, exact, (True, False))} <= padded


def random_size(rng):
    """Sizes that a card's memory holds, up to 2^27 rows."""
    while True:
        M, N, K = (int(2 ** rng.uniform(0, hi)) for hi in (27, 20, 20))
        if N * K <= 1 << 36 and M * K <= 1 << 38 and M * N <= 1 << 38:
            return M, N, K


def test_plans_are_sound():
    """Random sizes: the workgroups cover C, the chunks cover k with none empty, and
    what needs memory says how much."""
    rng = random.Random(3)
    for _ in range(20000):
        M, N, K = random_size(rng)
        a, b, b_rows = rng.random() < 0.5, rng.random() < 0.5, rng.choice((1, 128))
        p = plan(M, N, K, b_rows, rng.random() < 0.3, a, b, rng.random() < 0.3, rng.choice((1, 64, 256, 304)))
        kb = cdiv(K, 128)
        assert p["tiles"] == cdiv(M, p["rows"]) * cdiv(N, p["cols"])
        assert (p["k_splits"] - 1) * p["k_blocks"] < kb <= p["k_splits"] * p["k_blocks"] and p["k_splits"] <= 16
        assert p["grid"] >= 1
        fits = (a and b) and K % 16 == 0
        assert (p["pad_bytes"] > 0) == (not p["few_rows"] and not fits)
        assert not p["few_rows"] or fits or K >= 16
        if p["k_splits"] == 1:
            assert p["workspace_bytes"] == 0
        else:
            c = M * N if p["few_rows"] else p["tiles"] * p["rows"] * p["cols"]
            assert p["workspace_bytes"] == p["k_splits"] * c * 4
            assert p["few_rows"] or p["grid"] == p["tiles"] * p["k_splits"]
        assert p["exact"] or kb > 2


def test_launches_fit():
    """A launch's threads are a 32-bit number, also for the most rows and for few
    columns, whose tiles the few-rows kernel rounds up to a multiple of 8."""
    rng = random.Random(5)
    sizes = [random_size(rng) for _ in range(20000)]
    sizes += [(int(2 ** rng.uniform(20, 31)) - 1, rng.randint(1, 300), int(2 ** rng.uniform(0, 12))) for _ in range(20000)]
    for M, N, K in sizes:
        p = plan(M, N, K, rng.choice((1, 128)), rng.random() < 0.5, rng.random() < 0.5, True)
        assert p["grid"] * p["threads"] < 1 << 32, (M, N, K, p)


def test_plan_refuses_what_the_product_refuses():
    for kw, code in (({"M": -1}, bd.GEMM_ERR_INVALID_VALUE), ({"b_rows": 2}, bd.GEMM_ERR_INVALID_VALUE),
                     ({"cus": 0}, bd.GEMM_ERR_INVALID_VALUE), ({"N": (1 << 22) + 1}, bd.GEMM_ERR_UNSUPPORTED_SHAPE)):
        with pytest.raises(bd.GemmError) as e:
            plan(**{"M": 64, "N": 64, "K": 64, **kw})
        assert e.value.code == code
    assert plan(0, 5, 128)["grid"] == 0 == plan(5, 5, 0)["grid"]
    assert bd.library().gemm_fp8_plan_cus(1, 1, 1, 1, 0, 1, 1, 256, None) == bd.GEMM_ERR_INVALID_VALUE
