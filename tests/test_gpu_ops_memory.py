"""The 8-bit operators on rows whose offsets pass 32 bits, and the product's
temporary memory under graph capture in the forms that take it."""
import pytest
import torch

import ops_reference as ref
from pipelined_tiled_dense_amd import binding as bd

pytestmark = pytest.mark.gpu

BF16, FP8, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32
LD = 1_200_000_005      # elements between rows: the third row starts past 2^31 elements and 2^32 bytes


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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def far(x):
    """x's rows LD apart."""
    buf = torch.empty((x.shape[0] - 1) * LD + x.shape[1], dtype=x.dtype, device="cuda")
    view = buf.as_strided(x.shape, (LD, 1))
    view.copy_(x)
    return view


def bits(x):
    return x.view(torch.uint8) if x.dtype is FP8 else x


@pytest.mark.parametrize("D", [640, 1001])
def test_rows_far_apart(D):
    """Inputs in rows that far apart give what the same rows give side by side."""
    g = gen(D)
    x, r, dy = (torch.randn(3, D, generator=g, device="cuda").to(BF16) for _ in range(3))
    w = torch.randn(D, generator=g, device="cuda").to(BF16)
    gu = torch.randn(3, 2 * D, generator=g, device="cuda").to(BF16)
    calls = [
        (lambda x: bd.rms_norm(x, w, quantize=True)[:2], (x,)), (lambda x: bd.rms_norm(x, w, residual=r)[::2], (x,)),
        (lambda r: bd.rms_norm(x, w, residual=r)[::2], (r,)),
        (lambda dy: bd.rms_norm_backward(dy, x, w, torch.ones(3, device="cuda"), dresidual=r), (dy,)),
        (lambda x: bd.rms_norm_backward(dy, x, w, torch.ones(3, device="cuda")), (x,)),
        (lambda gu: bd.swiglu(gu, quantize=True), (gu,)), (lambda gu: (bd.swiglu_backward(dy, gu),), (gu,)),
        (bd.quantize_fp8, (x,)), (lambda x: bd.quantize_fp8(x, block_rows=128, transposed=True), (x,)),
        (lambda x: bd.quantize_fp8(x, block_rows=128), (x,)), (lambda x: bd.quantize_fp8(x, transposed=True), (x,)),
    ]
    for f, args in calls:
        want, got = f(*args), f(*(far(a) for a in args))
        for a, b in zip(want, got):
            assert torch.equal(bits(a), bits(b))


def test_product_of_rows_far_apart():
    g = gen(1)
    q, s = bd.quantize_fp8(torch.randn(3, 1040, generator=g, device="cuda").to(BF16))
    b, sb = bd.quantize_fp8(torch.randn(70, 1040, generator=g, device="cuda").to(BF16))
    assert torch.equal(bd.gemm_fp8(far(q.view(torch.uint8)).view(FP8), s, b, sb), bd.gemm_fp8(q, s, b, sb))
    out = far(torch.zeros(3, 70, dtype=BF16, device="cuda"))
    assert torch.equal(bd.gemm_fp8(q, s, b, sb, out=out), bd.gemm_fp8(q, s, b, sb))
    assert torch.equal(bd.gemm_fp8(b, sb, far(q.view(torch.uint8)).view(FP8), s), bd.gemm_fp8(b, sb, q, s))


# (M, N, K, pad, exact): few rows with k chunks, padded copies before tiles, both k
# splits and padded copies, exact tiles with k splits.
@pytest.mark.parametrize("M,N,K,pad,exact", [(6, 60, 16640, 0, False), (2000, 900, 272, 5, False),
                                             (75, 1641, 16985, 0, False), (401, 707, 16000, 0, True)])
def test_graph_replay(M, N, K, pad, exact):
    """Every replay, with eager calls and synchronisations in between, gives the
    eager result."""
    g = gen(M)
    def rows(n):
        buf = (torch.randn(n, K + pad, generator=g, device="cuda") * 20).to(FP8)
        return buf[:, :K], torch.rand(ref.nblocks(K), n, generator=g, device="cuda") + 0.5
    a, sa = rows(M)
    b, sb = rows(N)
    p = bd.gemm_fp8_plan_cus(M, N, K, 1, bd.FP8_EXACT if exact else 0, (K + pad) % 16 == 0, (K + pad) % 16 == 0, 256)
    assert p["workspace_bytes"] or p["pad_bytes"]
    want = bd.gemm_fp8(a, sa, b, sb, exact=exact)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = bd.gemm_fp8(a, sa, b, sb, exact=exact)
    for _ in range(4):
        out.fill_(0.0)
        assert torch.equal(bd.gemm_fp8(a, sa, b, sb, exact=exact), want)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
