"""The feed-forward block on bf16 operands: its output and gradients against the
block's formulas in 64 bits, single tokens against the batch, and the command."""
import pytest
import torch

import linear_reference as lin
import ops_reference as ref
from pipelined_tiled_dense_amd import mlp

pytestmark = pytest.mark.gpu

# Every stored intermediate is off by at most U16 of itself: n, gu, y, dgu, dn and the
# weights' operands.  The longest chain, to x's gradient, passes n, gu, dgu and dn and
# the slopes' change with gu (at most as large again), and its errors are independent of
# each other over the sums: 8 U16 of a result's norm covers them added up.
BOUND = 8 * ref.U16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")


def block(D, F, seed=0, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w = [x.to(torch.bfloat16) for x in ((1 + 0.1 * rand(D)), rand(2 * F, D) * D ** -0.5, rand(D, F) * F ** -0.5)]
    return mlp.FeedForwardBF16(*w, **kw), [x.double() for x in w], rand


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,D,F", [(1, 256, 512), (7, 384, 1001), (300, 512, 1280), (1000, 1024, 2048)])
def test_forward_and_gradients(M, D, F, act):
    b, (wn, wgu, wd), rand = block(D, F, seed=M, activation=act)
    x, r, dout, dh = (rand(M, D).to(torch.bfloat16) for _ in range(4))
    out, h, saved = b.forward(x, r)
    y, h2 = b(x, r)
    assert torch.equal(out, y) and torch.equal(h, h2)

    hd, rstd, n = ref.rms_norm(x.double(), r.double(), wn, b.eps)
    gu = torch.mm(n, wgu.t().contiguous())
    gate, up = gu.chunk(2, 1)
    value, slope, _, _ = lin.activation(gate, act)
    a = value * up
    assert off(h, hd) < 2 * ref.U16 and off(out, torch.mm(a, wd.t().contiguous())) < BOUND

    grads = b.backward(saved, dout, dh)
    d = dout.double()
    t = torch.mm(d, wd)
    dgu = torch.cat([t * up * slope, t * value], 1)
    dx, dnorm = ref.rms_norm_bwd(torch.mm(dgu, wgu), hd, wn, rstd, dh.double())
    assert off(grads.x, dx) < BOUND and off(grads.norm, dnorm) < BOUND
    assert off(grads.down, torch.mm(d.t().contiguous(), a)) < BOUND
    assert off(grads.gate_up, torch.mm(dgu.t().contiguous(), n)) < BOUND


def test_single_tokens_match_the_batch():
    """Serving row by row takes other kernels than the batch; a row's result differs by
    the rounding of n, y and out only."""
    b, _, rand = block(512, 1280)
    x = rand(130, 512).to(torch.bfloat16)
    whole = b(x)[0].double()
    for i in (0, 64, 129):
        assert off(b(x[i:i + 1])[0], whole[i:i + 1]) < 3 * ref.U16


def test_command_runs(capsys):
    mlp.main(["--bf16"])
    assert "token 2" in capsys.readouterr().out
