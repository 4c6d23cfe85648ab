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
