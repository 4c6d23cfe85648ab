"""Results that the host reads right behind a call whose last kernel is also the completion of
the library's temporary memory: products in k chunks and on padded copies, the norm's
gradients and the linear layers, in each way that a user waits for them."""
import pytest
import torch

from pipelined_tiled_dense_amd import binding as bd

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def named(request):
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    print("  %s" % request.node.name, flush=True)
    yield
    torch.cuda.synchronize()


def rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(BF16)


def calls():
    """(name, call(input), three inputs)."""
    g = torch.Generator(device="cuda").manual_seed(7)
    w1, w2, w3 = rand(g, 1032, 8192), rand(g, 45, 4100), rand(g, 601, 1000)
    q, qs = bd.quantize_fp8(rand(g, 512, 16000), block_rows=128)
    p, ps = bd.quantize_fp8(rand(g, 300, 272), block_rows=128)
    weight, rstd = rand(g, 4096), torch.rand(700, generator=g, device="cuda") + 0.5
    h, gu = rand(g, 700, 4096), rand(g, 300, 1202)
    three = lambda *s: [rand(g, *s) for _ in range(3)]  # noqa: E731
    assert bd.gemm_bf16_plan(1000, 1032, 8192, True, 0, 0)["k_splits"] > 1
    fp8 = lambda b, s: lambda x: bd.gemm_fp8(*bd.quantize_fp8(x), b, s)  # noqa: E731
    return [
        ("product in chunks", lambda x: bd.gemm(x, w1, b_transposed=True), three(1000, 8192)),
        ("padded product", lambda x: bd.gemm(x, w2, b_transposed=True), three(37, 4100)),
        ("8-bit product in chunks", fp8(q, qs), three(6, 16000)),
        ("8-bit product", fp8(p, ps), three(2000, 272)),
        ("norm's gradients", lambda x: torch.cat([t.float().reshape(-1) for t in bd.rms_norm_backward(x, h, weight, rstd)]), three(700, 4096)),
        ("norm's weight gradient", lambda x: bd.rms_norm_backward(x, h, weight, rstd)[1], three(700, 4096)),
        ("layer in chunks", lambda x: bd.linear(x, w1, activation="silu"), three(70, 8192)),
        ("padded layer", lambda x: bd.linear(x, w3), three(300, 1000)),
        ("padded gradient", lambda x: bd.gated_linear_backward_input(x, w3.t().contiguous(), gu), three(300, 1000)),
        ("weight's gradient", lambda x: bd.linear_backward_weight(x, h, bias=True)[0], three(700, 130)),
        ("bias's gradient", lambda x: bd.linear_backward_weight(x, h, bias=True)[1], three(700, 130)),
    ]


def test_results_on_the_host():
    for name, call, xs in calls():
        print("  %s" % name, flush=True)
        want = []
        for x in xs:
            y = call(x)
            torch.cuda.synchronize()
            want.append(y.clone().cpu())
        assert not torch.equal(want[0], want[1])
        pinned = torch.empty(want[0].shape, dtype=want[0].dtype, pin_memory=True)
        here, other, done = torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Event()
        for i in range(9):
            w = want[i % 3]
            assert torch.equal(call(xs[i % 3]).cpu(), w), name                    # pageable
            pinned.copy_(call(xs[i % 3]), non_blocking=True)                      # pinned, by an event
            done.record()
            done.synchronize()
            assert torch.equal(pinned, w), name
            pinned.zero_()
            y = call(xs[i % 3])                                                   # behind a synchronised stream
            here.synchronize()
            with torch.cuda.stream(other):
                pinned.copy_(y, non_blocking=True)
            other.synchronize()
            assert torch.equal(pinned, w), name
            pinned.zero_()
            y = call(xs[i % 3])                                                   # on another stream, by an event
            done.record(here)
            other.wait_event(done)
            with torch.cuda.stream(other):
                pinned.copy_(y, non_blocking=True)
                y.record_stream(other)
            while not other.query():
                pass
            assert torch.equal(pinned, w), name


def test_blocks_pass_between_operators_and_streams():
    """Calls of all of them in turn on two streams, with no synchronisation: the kept blocks that
    one leaves and another takes spoil no result."""
    cs = calls()
    want = [call(xs[0]).clone() for _, call, xs in cs]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(4):
        for k, (_, call, xs) in enumerate(cs):
            with torch.cuda.stream(streams[(i + k) % 2]):
                outs.append((k, call(xs[0])))
    torch.cuda.synchronize()
    for k, y in outs:
        assert torch.equal(y, want[k]), cs[k][0]
    assert bd.gemm_bf16_workspace_info()["busy"] == 0
