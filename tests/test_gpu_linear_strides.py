"""The linear layers' leading dimensions at their ends: those that do not count, a single
row's and an absent operand's, and those past what a tile's own offsets reach."""
import pytest
import torch

import linear_reference as ref
from pipelined_tiled_dense_amd import binding as bd

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    bd.library()
    yield
    torch.cuda.empty_cache()


@pytest.fixture(autouse=True)
def named(request):
    print("  %s" % request.node.name, flush=True)
    yield
    torch.cuda.synchronize()


def rand(g, *shape, size=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * size).to(BF16)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def stream():
    return torch.cuda.current_stream().cuda_stream


def units():
    return torch.cuda.get_device_properties(0).multi_processor_count


# -- leading dimensions that do not count ------------------------------------------------
ANY = [0, 7, -3, 1 << 40]


@pytest.mark.parametrize("ld", ANY)
@pytest.mark.parametrize("M,K,kind", [(8, 65536, 0), (64, 65536, 0), (1000, 65536, 0), (100000, 4096, 0), (8, 4096, 1)])
def test_weight_of_one_row(M, K, kind, ld):
    """One output feature: dW is a single row, in tiles of 128 and 256, in k chunks and in waves."""
    plan = bd.gemm_linear_plan_cus(M, 1, K, "linear_bwd_weight", 0, 1, units())
    assert plan["waves_share_k"] == kind
    g = gen(M)
    dy, x = rand(g, M, 1), rand(g, M, K)
    want, err = ref.product(dy.double().t(), x.double())
    for dtype, code in ((BF16, bd.TYPE_BF16), (F32, bd.TYPE_FP32)):
        dw = torch.full((K + 16,), 7.0, dtype=dtype, device="cuda")
        assert bd.gemm_linear_bwd_weight(M, 1, K, dy.data_ptr(), 1, x.data_ptr(), K, dw.data_ptr(), ld, code, None,
                                         stream()) == bd.GEMM_OK
        ref.check(dw[:K], want[0], err[0] if dtype is F32 else ref.rounded(want, err)[0], "ld %d" % ld)
        assert (dw[K:] == 7.0).all()
        assert torch.equal(dw[:K], bd.linear_backward_weight(dy, x, out_dtype=dtype)[0])


@pytest.mark.parametrize("ld", ANY)
@pytest.mark.parametrize("N,K", [(40, 64), (4096, 512), (65536, 72)])
def test_single_rows(N, K, ld):
    """One row: none of its leading dimensions count."""
    g = gen(N)
    x, w, wt, r, z, gu = rand(g, 1, K), rand(g, N, K), rand(g, K, N), rand(g, 1, N), rand(g, 1, N), rand(g, 1, 2 * N)
    w2, st = rand(g, 2 * N, K), stream()
    out = [torch.zeros(1, N, dtype=BF16, device="cuda") for _ in range(4)] + [torch.zeros(1, 2 * N, dtype=BF16, device="cuda") for _ in range(2)]
    y, kept, dx, yg, gg, dgu = out
    assert bd.gemm_linear(1, N, K, x.data_ptr(), ld, w.data_ptr(), K, None, 4, r.data_ptr(), ld, kept.data_ptr(), ld, y.data_ptr(), ld, st) == 0
    want = bd.linear(x, w, activation="silu", residual=r, return_preactivation=True)
    assert torch.equal(y, want[0]) and torch.equal(kept, want[1])
    assert bd.gemm_linear_bwd_input(1, K, N, x.data_ptr(), ld, wt.data_ptr(), N, 4, z.data_ptr(), ld, r.data_ptr(), ld, dx.data_ptr(), ld, st) == 0
    assert torch.equal(dx, bd.linear_backward_input(x, wt, preactivation=z, activation="silu", dresidual=r))
    assert bd.gemm_gated_linear(1, N, K, x.data_ptr(), ld, w2.data_ptr(), K, None, 4, gg.data_ptr(), ld, yg.data_ptr(), ld, st) == 0
    want = bd.gated_linear(x, w2, return_gu=True)
    assert torch.equal(yg, want[0]) and torch.equal(gg, want[1])
    assert bd.gemm_gated_linear_bwd_input(1, N, K, x.data_ptr(), ld, wt.data_ptr(), N, 4, gu.data_ptr(), ld, dgu.data_ptr(), ld,
                                          y.data_ptr(), ld, st) == 0
    want = bd.gated_linear_backward_input(x, wt, gu, return_y=True)
    assert torch.equal(dgu, want[0]) and torch.equal(y, want[1])


@pytest.mark.parametrize("M,N,K", [(1936, 1024, 1216), (4200, 4096, 136)])
def test_absent_operands_need_no_memory(M, N, K):
    """The leading dimension of an operand that is absent changes neither the way a call takes
    nor the temporary memory it asks for: a workspace of the planned bytes is enough."""
    g, st = gen(M), stream()
    x, w, wt, w2, gu = rand(g, M, K), rand(g, N, K), rand(g, K, N), rand(g, 2 * N, K), rand(g, M, 2 * N)
    y, dx, yg, dgu = (torch.empty(M, n, dtype=BF16, device="cuda") for n in (N, N, N, 2 * N))
    calls = [
        ("linear", lambda ld, m, n: bd.gemm_linear(M, N, K, x.data_ptr(), K, w.data_ptr(), K, None, 4, None, ld, None, ld,
                                                   y.data_ptr(), N, st, m, n), y, lambda: bd.linear(x, w, activation="silu")),
        ("linear_bwd_input", lambda ld, m, n: bd.gemm_linear_bwd_input(M, K, N, x.data_ptr(), K, wt.data_ptr(), N, 0, None, ld, None,
                                                                       ld, dx.data_ptr(), N, st, m, n), dx,
         lambda: bd.linear_backward_input(x, wt)),
        ("gated_linear", lambda ld, m, n: bd.gemm_gated_linear(M, N, K, x.data_ptr(), K, w2.data_ptr(), K, None, 4, None, ld,
                                                               yg.data_ptr(), N, st, m, n), yg, lambda: bd.gated_linear(x, w2)),
        ("gated_linear_bwd_input", lambda ld, m, n: bd.gemm_gated_linear_bwd_input(
            M, N, K, x.data_ptr(), K, wt.data_ptr(), N, 4, gu.data_ptr(), 2 * N, dgu.data_ptr(), 2 * N, None, ld, st, m, n), dgu,
         lambda: bd.gated_linear_backward_input(x, wt, gu)),
    ]
    tiles = 0
    for name, call, out, plain in calls:
        plan = bd.gemm_linear_plan_cus(*((M, K, N) if name == "linear_bwd_input" else (M, N, K)), name, 1, 1, units())
        tiles += not plan["waves_share_k"]
        n = plan["scratch_bytes"]
        ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
        for ld in ANY:
            out.fill_(0.0)
            assert call(ld, ws.data_ptr(), n) == bd.GEMM_OK, (name, ld)
            assert torch.equal(out, plain()), (name, ld)
    assert tiles >= 3


# -- rows further apart than a tile's offsets reach -----------------------------------------
FAR = (1 << 27) + 8


def far(x, ld=FAR):
    """A view of x's values in rows that far apart; what lies between is not written."""
    view = torch.empty((x.shape[0] - 1) * ld + x.shape[1], dtype=x.dtype, device="cuda").as_strided(x.shape, (ld, 1))
    view.copy_(x)
    return view


def planned(product, M, N, K):
    """The plan, and the temporary memory of a call whose epilogue is out of the tiles' reach: of
    one chunk, the sums of every tile beside what the plan says."""
    p = bd.gemm_linear_plan_cus(*((M, K, N) if product == "linear_bwd_input" else (M, N, K)), product, 1, 1, units())
    assert not p["waves_share_k"]
    sums = p["tiles"] * p["rows"] * p["cols"] * 4 * (2 if product == "gated_linear" else 1)
    return p, p["scratch_bytes"] + (sums if p["k_splits"] == 1 else 0)


def run(call, need):
    """The call in a workspace of exactly `need` bytes, which less is refused for."""
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    assert call(ws.data_ptr(), need - 256) == bd.GEMM_ERR_SCRATCH
    assert call(ws.data_ptr(), need) == bd.GEMM_OK
    torch.cuda.synchronize()
    assert (ws[need:] == 0xA5).all()


# 33 rows (a far one takes 9 GB) of 128- and 192-row tiles (256 where paired), one chunk; and k chunks.
WIDE = [(33, 32768, 64), (33, 65536, 64), (33, 8192, 8192)]


@pytest.mark.parametrize("which", ["residual", "z", "y", "y over residual"])
@pytest.mark.parametrize("M,N,K", WIDE)
def test_far_linear(M, N, K, which):
    plan, need = planned("linear", M, N, K)
    g = gen(N)
    x, w, r = rand(g, M, K), rand(g, N, K, size=K ** -0.5), rand(g, M, N)
    want = ref.linear(x.double(), w.double(), None, "silu", r.double())
    at = lambda name, t: far(t) if name in which else t  # noqa: E731
    res, z, y = at("residual", r), at("z", torch.zeros_like(r)), None
    y = res if "over" in which else at("y", torch.zeros_like(r))
    run(lambda m, n: bd.gemm_linear(M, N, K, x.data_ptr(), K, w.data_ptr(), K, None, 4, res.data_ptr(), res.stride(0), z.data_ptr(),
                                    z.stride(0), y.data_ptr(), y.stride(0), stream(), m, n), need)
    ref.check(y, *want["y"], "y")
    ref.check(z, *want["z"], "z")


@pytest.mark.parametrize("which", ["z", "dres", "dx", "dx over z"])
@pytest.mark.parametrize("M,N,K", WIDE)
def test_far_linear_backward_input(M, N, K, which):
    plan, need = planned("linear_bwd_input", M, N, K)
    g = gen(N + 1)
    dy, w, z, r = rand(g, M, K), rand(g, K, N, size=K ** -0.5), rand(g, M, N), rand(g, M, N)
    want = ref.linear_backward_input(dy.double(), w.double(), z.double(), "gelu", r.double())
    zs = far(z) if which in ("z", "dx over z") else z
    rs = far(r) if which == "dres" else r
    dx = zs if "over" in which else far(torch.zeros_like(z)) if which == "dx" else torch.zeros_like(z)
    run(lambda m, n: bd.gemm_linear_bwd_input(M, K, N, dy.data_ptr(), K, w.data_ptr(), N, bd.ACTIVATIONS["gelu"], zs.data_ptr(),
                                              zs.stride(0), rs.data_ptr(), rs.stride(0), dx.data_ptr(), dx.stride(0), stream(), m, n), need)
    ref.check(dx, *want, "dx")


@pytest.mark.parametrize("which", ["gu", "y"])
@pytest.mark.parametrize("M,F,K", [(33, 14336, 64), (33, 32768, 64), (33, 4096, 8192)])
def test_far_gated_linear(M, F, K, which):
    plan, need = planned("gated_linear", M, F, K)
    g = gen(F + 2)
    x, w = rand(g, M, K), rand(g, 2 * F, K, size=K ** -0.5)
    want = ref.gated(x.double(), w.double(), None, "silu")
    y, gu = torch.zeros(M, F, dtype=BF16, device="cuda"), torch.zeros(M, 2 * F, dtype=BF16, device="cuda")
    y, gu = (far(y), gu) if which == "y" else (y, far(gu))
    run(lambda m, n: bd.gemm_gated_linear(M, F, K, x.data_ptr(), K, w.data_ptr(), K, None, 4, gu.data_ptr(), gu.stride(0), y.data_ptr(),
                                          y.stride(0), stream(), m, n), need)
    ref.check(y, *want["y"], "y")
    ref.check(gu, *want["gu"], "gu")


@pytest.mark.parametrize("which", ["gu", "dgu", "dgu over gu", "y"])
@pytest.mark.parametrize("M,F,N", WIDE)
def test_far_gated_linear_backward_input(M, F, N, which):
    plan, need = planned("gated_linear_bwd_input", M, F, N)
    g = gen(F + 3)
    dy, w, gu = rand(g, M, N), rand(g, N, F, size=N ** -0.5), rand(g, M, 2 * F)
    want = ref.gated_backward_input(dy.double(), w.double(), gu.double(), "silu")
    gs = far(gu) if which in ("gu", "dgu over gu") else gu
    d = gs if "over" in which else far(torch.zeros_like(gu)) if which == "dgu" else torch.zeros_like(gu)
    y = torch.zeros(M, F, dtype=BF16, device="cuda")
    y = far(y) if which == "y" else y
    run(lambda m, n: bd.gemm_gated_linear_bwd_input(M, F, N, dy.data_ptr(), N, w.data_ptr(), F, 4, gs.data_ptr(), gs.stride(0),
                                                    d.data_ptr(), d.stride(0), y.data_ptr(), y.stride(0), stream(), m, n), need)
    ref.check(d, *want["dgu"], "dgu")
    ref.check(y, *want["y"], "y")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(64, 3, 32768), (64, 2, 65536), (8192, 4, 8192)])
def test_far_weight(M, N, K, dtype):
    p = bd.gemm_linear_plan_cus(M, N, K, "linear_bwd_weight", 0, 1, units())
    assert not p["waves_share_k"]
    sums = p["tiles"] * p["rows"] * p["cols"] * 4
    need = p["scratch_bytes"] + (sums if p["k_splits"] == 1 else 0)
    g = gen(K + 4)
    dy, x = rand(g, M, N), rand(g, M, K)
    want, err = ref.product(dy.double().t(), x.double())
    dw = far(torch.zeros(N, K, dtype=dtype, device="cuda"))
    code = bd.TYPE_FP32 if dtype is F32 else bd.TYPE_BF16
    db = torch.empty(N, device="cuda")
    run(lambda m, n: bd.gemm_linear_bwd_weight(M, N, K, dy.data_ptr(), N, x.data_ptr(), K, dw.data_ptr(), FAR, code, db.data_ptr(),
                                               stream(), m, n), need)
    ref.check(dw, want, err if dtype is F32 else ref.rounded(want, err), "dw")
    ref.check(db, dy.double().sum(0), (M + 4) * ref.U32 * dy.double().abs().sum(0), "dbias")


@pytest.mark.parametrize("M,N,K", WIDE)
def test_far_rows_under_capture(M, N, K):
    """A captured call whose residual, preactivation or [g, u] is that far apart: torch's memory is
    as much as it takes, and every replay gives the eager result."""
    g = gen(N + 5)
    x, w, wt = rand(g, M, K), rand(g, N, K, size=K ** -0.5), rand(g, K, N, size=K ** -0.5)
    r, gu = far(rand(g, M, N)), far(rand(g, M, 2 * N))
    calls = lambda: [bd.linear(x, w, activation="silu", residual=r), bd.linear_backward_input(x, wt, preactivation=r, activation="gelu"),  # noqa: E731
                     bd.gated_linear_backward_input(x, wt, gu)]
    want = [t.clone() for t in calls()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = calls()
    for _ in range(3):
        for t in out:
            t.fill_(0.0)
        for a, b in zip(calls(), want):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
