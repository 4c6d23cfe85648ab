"""The linear layers' activations and their slopes at every finite bf16 value, through
the products' epilogues, against the formulas in 64 bits to fp32's rounding.

One term of every sum is not zero, so the products are exact and what is left is the
activation's own error and one rounding to bf16.

Bounds, in shares of U32 = 2^-24.  An exponential's instruction is right to an ulp, 2, a
reciprocal's too, the sum below it 1, four products 4: 9, of each of the terms that the
value or the slope is the sum of.  Gelu's tail adds its polynomial's 2 (7e-8), the roundings of
its steps, 5, and those of its argument, 3: 19, rounded up to 20.  Below -9, where the
exponential may be a third power, its 4 come three times: 28.  An exponential's argument v is
off by the share that its product with log2 e is rounded by, 1, and that constant, 1/3, of
itself: 2 |v|; gelu's a^2 / 2 by that and its square's rounding, 3 of itself: 2 a^2;
gelu_tanh's, a cubic, by 4 more: 6 |v|."""
import math

import pytest
import torch

from ops_reference import TINY16, U16, U32
from pipelined_tiled_dense_amd import binding as bd

BF16, F32 = torch.bfloat16, torch.float32
ACTS = ["gelu", "gelu_tanh", "silu", "relu", None]
ROWS, COLS = 256, 256      # 65536 values


def patterns():
    """Every finite bf16 value, in the place of the others 1."""
    z = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
    return torch.where(z.isfinite(), z, torch.ones_like(z)).view(ROWS, COLS)


def formula(z, act):
    """(value, slope, error of the value, error of the slope) in 64 bits."""
    z = z.double()
    zero = torch.zeros_like(z)
    shares = torch.where(z < -9, 28 * U32, 20 * U32)
    if act is None:
        return z, torch.ones_like(z), zero, zero
    if act == "relu":
        return z.clamp_min(0), (z > 0).double(), zero, zero
    if act == "gelu":
        a = z.abs()
        density = torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
        tail = torch.where(a < 5, 0.5 * torch.erfc(a / math.sqrt(2)), 0.5 * torch.exp(-a * a / 2) * torch.special.erfcx(a / math.sqrt(2)))
        cdf = torch.where(z > 0, 1 - tail, tail)
        value, slope = z * cdf, torch.where(z > 0, 1 - (tail - a * density), tail - a * density)
        share = shares + 2 * a * a * U32
        return value, slope, a * tail * share + 4 * U32 * value.abs(), (tail + a * density) * share + 4 * U32 * slope.abs()
    v, dv = z, torch.ones_like(z)
    per = 2
    if act == "gelu_tanh":
        k = 2 * math.sqrt(2 / math.pi)
        # Beyond 1e6 the logistic function is 0 or 1, and z^3 would overflow.
        c = z.clamp(-1e6, 1e6)
        v, dv = k * (c + 0.044715 * c ** 3), k * (1 + 3 * 0.044715 * c ** 2)
        per = 6
    p, q = torch.sigmoid(v), torch.sigmoid(-v)
    # exp(v) vanishes long before z dv overflows.
    turn = torch.where(p * q > 0, z * dv * p * q, zero)
    bend = per * v.abs() * U32                       # where p is near 1 the exponential hardly enters it
    return z * p, p + turn, (z * p).abs() * (shares + q * bend), p * (shares + q * bend) + turn.abs() * (shares + bend)


def within(got, want, err, what):
    bound = err + U16 * (want.abs() + err) + TINY16
    d = (got.double() - want).abs()
    bad = ~(d <= bound)
    assert not bad.any(), "%s: %d of %d, worst %g of its bound at %s" % (
        what, int(bad.sum()), bad.numel(), float((d / bound).nan_to_num(float("inf")).max()), tuple(torch.nonzero(bad)[0].tolist()))


def test_formulas_against_differences():
    """The slope is the value's derivative, and torch's own functions give the values."""
    z = torch.linspace(-9, 9, 2001, dtype=torch.float64)
    f = torch.nn.functional
    own = {"gelu": f.gelu, "gelu_tanh": lambda x: f.gelu(x, approximate="tanh"), "silu": f.silu, "relu": f.relu, None: lambda x: x}
    for act in ACTS:
        value, slope, _, _ = formula(z, act)
        assert torch.allclose(value, own[act](z), rtol=1e-9, atol=1e-15)
        step = 1e-6
        change = (formula(z + step, act)[0] - formula(z - step, act)[0]) / (2 * step)
        keep = z.abs() > 1e-3                        # relu's corner
        assert torch.allclose(slope[keep], change[keep], rtol=1e-6, atol=1e-8)


def test_the_bound_tells_a_coarse_tail():
    """A tail that is right to 1.6e-5 only, a fiftieth of bf16's half step, is out of
    gelu's slope bound where the slope's terms cancel."""
    z = patterns()
    _, slope, _, err = formula(z, "gelu")
    a = z.double().abs()
    tail = 0.5 * torch.erfc(a / math.sqrt(2))
    coarse = slope + torch.where(z > 0, -1.0, 1.0) * tail * 1.6e-5
    within(slope.to(BF16), slope, err, "slope")
    with pytest.raises(AssertionError):
        within(coarse.to(F32).to(BF16), slope, err, "coarse")


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    yield
    torch.cuda.synchronize()


# Rows of the product beside the 256 columns: waves that share k, and tiles.
@pytest.mark.gpu
@pytest.mark.parametrize("copies", [1, 8, 16])
@pytest.mark.parametrize("act", ACTS)
def test_slopes_at_every_value(gpu, act, copies):
    z = patterns()
    _, slope, _, err = formula(z, act)
    zg = z.cuda().repeat(copies, copies)
    M, K = zg.shape
    kind = bd.gemm_linear_plan_cus(M, 64, K, "linear_bwd_input", 1, 1, 256)["waves_share_k"]
    assert kind == (copies == 1)
    dy, w = torch.zeros(M, 64, dtype=BF16, device="cuda"), torch.zeros(64, K, dtype=BF16, device="cuda")
    dy[:, 5], w[5] = 1.0, 1.0
    dx = bd.linear_backward_input(dy, w, preactivation=zg if act else None, activation=act)
    within(dx.cpu()[:ROWS, :COLS], slope, err, "slope of %s" % act)
    assert torch.equal(dx, dx[:ROWS, :COLS].repeat(copies, copies))
    # The gated gradient of u = 1: the same slope, and t times the value.
    value, _, ev, _ = formula(z, act)
    gu = torch.cat([zg, torch.ones_like(zg)], 1)
    dgu, y = bd.gated_linear_backward_input(dy, w, gu, activation=act, return_y=True)
    within(dgu[:ROWS, :COLS].cpu(), slope, err + 4 * U32 * slope.abs(), "dg of %s" % act)
    within(dgu[:ROWS, K:K + COLS].cpu(), value, ev, "du of %s" % act)
    assert torch.equal(y, dgu[:, K:])


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 20, 300])
@pytest.mark.parametrize("act", ACTS)
def test_values_at_every_value(gpu, act, M):
    z = patterns().reshape(-1)
    value, _, err, _ = formula(z, act)
    x, w = torch.zeros(M, 64, dtype=BF16, device="cuda"), torch.zeros(65536, 64, dtype=BF16, device="cuda")
    x[:, 9], w[:, 9] = 1.0, z.cuda()
    y = bd.linear(x, w, activation=act)
    within(y[:1].cpu()[0], value, err, "value of %s" % act)
    assert torch.equal(y, y[:1].expand(M, -1))
    both = torch.cat([w, torch.zeros_like(w)])
    both[65536:, 9] = 1.0
    yg = bd.gated_linear(x, both, activation=act)
    within(yg[:1].cpu()[0], value, err, "gated value of %s" % act)
    assert torch.equal(yg, yg[:1].expand(M, -1))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 4096])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_largest_factors_beside_slopes_above_one(gpu, act, M):
    """dg = t u act'(g) with t or u at the type's largest and a slope of up to 1.13: the
    result is finite where the other factor is small, in whichever order."""
    big = float(torch.finfo(BF16).max)
    gates = torch.linspace(0.0, 6.0, 64).to(BF16).repeat(8)
    for t, u in ((0.1, big), (big, 0.1), (1e-30, -big), (-big, 1e-30), (0.85, 3.2e38), (3.2e38, 0.85), (2e-38, big), (1.0, -2.9e38)):
        F = gates.numel()
        gu = torch.cat([gates, torch.full((F,), u).to(BF16)]).cuda().expand(M, -1).contiguous()
        dy, w = torch.zeros(M, 64, dtype=BF16, device="cuda"), torch.zeros(64, F, dtype=BF16, device="cuda")
        dy[:, 3], w[3] = t, 1.0
        td, ud = dy[0, 3].double().cpu(), gu[0, F].double().cpu()
        _, slope, _, err = formula(gates, act)
        want = td * ud * slope
        keep = want.abs() < 3.38e38                    # above, a bf16 result may be infinite
        assert (keep | (slope > 1)).all() and keep.any()
        dgu = bd.gated_linear_backward_input(dy, w, gu, activation=act)
        got = dgu[0, :F].cpu()
        within(got[keep], want[keep], ((td * ud).abs() * err + 8 * U32 * want.abs())[keep], "%g %g" % (t, u))
        assert torch.equal(dgu, dgu[:1].expand(M, -1))


@pytest.mark.gpu
@pytest.mark.parametrize("M,F", [(3, 64), (4096, 4096)])
@pytest.mark.parametrize("act", ACTS)
def test_infinities_and_nan(gpu, act, M, F):
    """What the formulas give: z Phi(z) at minus infinity and z phi(z) at both have a product of
    zero and infinity, and so have the logistic ones.  Finite values next to them stay."""
    inf, nan, big = float("inf"), float("nan"), float(torch.finfo(BF16).max)
    at = torch.tensor([inf, -inf, nan, big, -big, 1e20, -1e20, 0.0])
    values = {None: [inf, -inf, nan], "relu": [inf, 0.0, nan]}.get(act, [inf, nan, nan])
    slopes = {None: [1.0] * 3, "relu": [1.0, 0.0, nan]}.get(act, [nan] * 3)
    half = 0.0 if act == "relu" else 0.5
    values += [big, -big, 1e20, -1e20, 0.0] if act is None else [big, 0.0, 1e20, 0.0, 0.0]
    slopes += [1.0] * 5 if act is None else [1.0, 0.0, 1.0, 0.0, half]
    same = lambda got, want, what: torch.testing.assert_close(  # noqa: E731
        got, torch.tensor(want).to(BF16).repeat(F // 8).cuda().expand(M, F), rtol=0, atol=0, equal_nan=True, msg=what)
    z = at.to(BF16).repeat(F // 8).cuda()
    dy, wd = torch.zeros(M, 64, dtype=BF16, device="cuda"), torch.zeros(64, F, dtype=BF16, device="cuda")
    dy[:, 3], wd[3] = 1.0, 1.0
    gu = torch.cat([z, torch.ones_like(z)]).expand(M, -1).contiguous()
    same(bd.linear_backward_input(dy, wd, preactivation=gu[:, :F] if act else None, activation=act), slopes, "slope")
    dgu, y = bd.gated_linear_backward_input(dy, wd, gu, activation=act, return_y=True)
    same(dgu[:, :F], slopes, "dg"), same(dgu[:, F:], values, "du"), same(y, values, "y again")
    # Forward: the sums themselves are infinite, through a bias.
    x, w = torch.zeros(M, 64, dtype=BF16, device="cuda"), torch.zeros(2 * F, 64, dtype=BF16, device="cuda")
    same(bd.linear(x, w[:F], bias=z, activation=act), values, "value")
    same(bd.gated_linear(x, w, bias=torch.cat([z, torch.ones_like(z)]), activation=act), values, "gated value")
