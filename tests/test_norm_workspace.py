"""The norm's gradients with the caller's temporary memory: its size and refusals without a
GPU; on one, exactly that memory, graphs that hold none of their own, and the bf16
feed-forward block's whole step captured."""
import ctypes

import pytest
import torch

from pipelined_tiled_dense_amd import binding as bd
from pipelined_tiled_dense_amd import mlp

A0 = 1 << 30          # fake, aligned addresses 1 GiB apart: never dereferenced by these calls
DY, H, W, RSTD, S, DX, DW, T = (A0 * (i + 1) for i in range(8))
BF16 = torch.bfloat16


def call(M=64, D=512, ws=T, n=1 << 20, dy=DY, lddy=512, dw=DW):
    return bd.gemm_rms_norm_bwd_given(M, D, dy, lddy, H, 512, W, RSTD, S, 512, DX, 512, dw, None, ws, n)


def test_refused():
    assert call(ws=T + 16) == bd.GEMM_ERR_MISALIGNED and call(n=-1) == bd.GEMM_ERR_INVALID_VALUE
    for a in (DY, H, W, RSTD, S, DX, DW):
        assert call(ws=a - 256) == bd.GEMM_ERR_ALIAS
    # What gemm_rms_norm_bwd refuses.
    assert call(D=0) == bd.GEMM_ERR_INVALID_VALUE and call(D=bd.NORM_MAX_WIDTH + 1) == bd.GEMM_ERR_UNSUPPORTED_SHAPE
    assert call(dy=None) == bd.GEMM_ERR_INVALID_VALUE and call(lddy=511) == bd.GEMM_ERR_INVALID_VALUE
    assert call(dy=DY + 1) == bd.GEMM_ERR_MISALIGNED and call(dw=H) == bd.GEMM_ERR_ALIAS
    if not torch.cuda.is_available():
        assert call() == bd.GEMM_ERR_DEVICE and call(ws=None, n=0) == bd.GEMM_ERR_DEVICE


def test_scratch():
    size = bd.gemm_rms_norm_bwd_scratch_cus
    assert [size(m, 4096, 256) for m in (0, 1, 4)] == [0, 0, 0]
    assert size(5, 4096, 256) == 3 * 4096 * 4 and size(9, 100, 256) == 2048          # 5 shares of 400 bytes, on the 256-byte grid
    for m in (1000, 100000):
        for d in (1, 512, 4096, 32768):
            assert 0 < size(m, d, 256) <= 256 * 8 * d * 4 + 256
    for args in ((-1, 8, 256), (8, 0, 256), (8, bd.NORM_MAX_WIDTH + 1, 256), (8, 8, 0)):
        with pytest.raises(bd.GemmError):
            size(*args)


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    yield
    torch.cuda.synchronize()


def rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(BF16)


@pytest.mark.gpu
@pytest.mark.parametrize("M,D", [(3, 4096), (5, 256), (37, 1001), (2047, 4096), (600, 16384), (4000, 96)])
def test_workspace(gpu, M, D):
    """Exactly the stated memory between guards gives what the call gives without; less is refused
    with nothing written."""
    g = torch.Generator(device="cuda").manual_seed(M)
    dy, h, w, r = rand(g, M, D), rand(g, M, D), rand(g, D), rand(g, M, D)
    rstd = torch.rand(M, generator=g, device="cuda") + 0.5
    want = bd.rms_norm_backward(dy, h, w, rstd, dresidual=r)
    n = bd.gemm_rms_norm_bwd_scratch_cus(M, D, torch.cuda.get_device_properties(0).multi_processor_count)
    guard = 1 << 16
    buf = torch.full((n + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
    dx, dw = torch.full((M, D), 7.0, dtype=BF16, device="cuda"), torch.full((D,), 7.0, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    go = lambda bytes: bd.gemm_rms_norm_bwd_given(M, D, dy.data_ptr(), D, h.data_ptr(), D, w.data_ptr(), rstd.data_ptr(),  # noqa: E731
                                                  r.data_ptr(), D, dx.data_ptr(), D, dw.data_ptr(), st, buf.data_ptr() + guard, bytes)
    if n:
        assert go(n - 256) == bd.GEMM_ERR_SCRATCH
        torch.cuda.synchronize()
        assert (dx == 7.0).all() and (dw == 7.0).all() and (buf == 0xA5).all()
    assert go(n) == bd.GEMM_OK
    torch.cuda.synchronize()
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    assert (buf[:guard] == 0xA5).all() and (buf[guard + n:] == 0xA5).all()


def capture(step, **kw):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph(**kw)
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = step()
    return graph, out


def node_types(graph):
    """The types of a kept graph's nodes, from the runtime that is loaded."""
    path = next(line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line)
    hip = ctypes.CDLL(path)
    g, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t()
    assert hip.hipGraphGetNodes(g, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert hip.hipGraphGetNodes(g, nodes, ctypes.byref(n)) == 0
    kinds = []
    for node in nodes:
        kind = ctypes.c_int()
        assert hip.hipGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        kinds.append(kind.value)
    return kinds


@pytest.mark.gpu
@pytest.mark.parametrize("M,D,F", [(1, 256, 640), (7, 256, 1001), (300, 512, 1280), (1000, 1024, 2056)])
def test_block_step_captured(gpu, M, D, F):
    """The bf16 block's forward and backward pass captured: kernels alone, no memory that the
    graph allocates; every replay, with the eager step and synchronisations in between,
    gives the eager results."""
    g = torch.Generator(device="cuda").manual_seed(M)
    block = mlp.FeedForwardBF16(1 + 0.1 * rand(g, D), rand(g, 2 * F, D) * D ** -0.5, rand(g, D, F) * F ** -0.5)
    x, r, dout, dh = (rand(g, M, D) for _ in range(4))

    def step():
        out, h, saved = block.forward(x, r)
        return [out, h, *block.backward(saved, dout, dh)]

    want = [t.clone() for t in step()]
    kept, _ = capture(step, keep_graph=True)
    assert set(node_types(kept)) == {0}          # hipGraphNodeTypeKernel
    graph, out = capture(step)
    for _ in range(4):
        for t in out:
            t.fill_(0.0)
        for a, b in zip(step(), want):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_capture_without_a_workspace_is_refused(gpu):
    g = torch.Generator(device="cuda").manual_seed(1)
    dy, h, w = rand(g, 64, 512), rand(g, 64, 512), rand(g, 512)
    rstd = torch.ones(64, device="cuda")
    dx, dw, x = torch.full((64, 512), 7.0, dtype=BF16, device="cuda"), torch.full((512,), 7.0, device="cuda"), torch.zeros(4, device="cuda")
    codes = []

    def step():
        x.add_(1)
        codes.append(bd.gemm_rms_norm_bwd_given(64, 512, dy.data_ptr(), 512, h.data_ptr(), 512, w.data_ptr(), rstd.data_ptr(), None, 0,
                                                dx.data_ptr(), 512, dw.data_ptr(), torch.cuda.current_stream().cuda_stream))

    graph, _ = capture(step)
    assert codes == [bd.GEMM_ERR_SCRATCH]
    graph.replay()
    torch.cuda.synchronize()
    assert (x == 1).all() and (dx == 7.0).all() and (dw == 7.0).all()
