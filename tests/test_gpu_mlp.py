"""The feed-forward block on the 8-bit operators: its output and gradients
against the block's formulas in 64 bits, single tokens against the batch, and
a few steps of gradient descent."""
import pytest
import torch

import ops_reference as ref
from pipelined_tiled_dense_amd import mlp

pytestmark = pytest.mark.gpu

# Rounding to e4m3 is off by at most 2^-4 of a value, and by 2^-4 / sqrt(3) =
# 3.6% in the root mean square at worst.  A product's operands both carry it
# (5.1%), and the block's longest chain, to the first weight's gradient, passes
# three products whose errors are independent: 5.1% * sqrt(3) = 8.9%.
BOUND = 0.09


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")


def block(D, F, seed=0, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w = [(1 + 0.1 * rand(D)), rand(2 * F, D) * D ** -0.5, rand(D, F) * F ** -0.5]
    return mlp.FeedForward(*(x.to(torch.bfloat16) for x in w), **kw), [x.to(torch.bfloat16).double() for x in w], rand


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("M,D,F", [(1, 256, 512), (7, 384, 1000), (300, 512, 1280), (1000, 1024, 2048)])
def test_forward_and_gradients(M, D, F):
    b, (wn, wgu, wd), rand = block(D, F, seed=M, training=True)
    x, r, dout, dh = (rand(M, D).to(torch.bfloat16) for _ in range(4))
    out, h, saved = b.forward(x, r)
    y, h2 = b(x, r)
    assert torch.equal(out, y) and torch.equal(h, h2)

    hd, rstd, n = ref.rms_norm(x.double(), r.double(), wn, b.eps)
    gu = n @ wgu.t()
    a = ref.swiglu(gu)
    assert off(h, hd) < 2 * ref.U16 and off(out, a @ wd.t()) < BOUND

    grads = b.backward(saved, dout, dh)
    d = dout.double()
    dgu = ref.swiglu_bwd(d @ wd, gu)
    dx, dnorm = ref.rms_norm_bwd(dgu @ wgu, hd, wn, rstd, dh.double())
    assert off(grads.x, dx) < BOUND and off(grads.norm, dnorm) < BOUND
    assert off(grads.down, d.t() @ a) < BOUND and off(grads.gate_up, dgu.t() @ n) < BOUND


def test_single_tokens_match_the_batch():
    """Serving row by row takes other kernels than the batch; each row's
    result differs by their rounding only."""
    b, _, rand = block(512, 1280)
    x = rand(130, 512).to(torch.bfloat16)
    whole = b(x)[0].double()
    for i in (0, 64, 129):
        # bf16's rounding at the two products, and 8-bit neighbours it can
        # turn over in between: a share of about U16 / 2^-4 of the values by
        # 2^-4 of themselves, 1.6% in the root mean square.
        assert off(b(x[i:i + 1])[0], whole[i:i + 1]) < 0.02


def test_gradient_descent_lowers_the_error():
    b, w, rand = block(256, 512, training=True)
    x, target = rand(512, 256).to(torch.bfloat16), rand(512, 256)
    w = [t.float() for t in w]
    errors = []
    for _ in range(8):
        out, _, saved = b.forward(x)
        e = out.float() - target
        errors.append(float(e.square().mean()))
        for t, dt in zip(w, b.backward(saved, (2.0 / 512 * e).to(torch.bfloat16))[1:]):
            t -= 0.2 * dt
        b.set_weights(*(t.to(torch.bfloat16) for t in w))
    assert all(b < a for a, b in zip(errors, errors[1:])), errors


def test_backward_needs_a_training_block():
    b, _, rand = block(256, 512)
    x = rand(3, 256).to(torch.bfloat16)
    with pytest.raises(ValueError):
        b.backward(b.forward(x)[2], x)
