"""The 8-bit operators at the ends of their number ranges, against their 64-bit
formulas."""
import pytest
import torch

import ops_reference as ref
from pipelined_tiled_dense_amd import binding as bd

pytestmark = pytest.mark.gpu

BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn
BF16_MAX = float(torch.finfo(BF16).max)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")
    bd.library()
    yield


@pytest.fixture(autouse=True)
def named(request):
    print("  %s" % request.node.name, flush=True)
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# -- gated unit --------------------------------------------------------------------
GATES = [-3.3e38, -1e30, -1e20, -1000.0, -217.0, -216.0, -200.0, -190.0, -177.0, -150.0, -128.0, -104.0, -100.0, -95.0, -90.0,
         -89.0, -88.5, -88.0, -87.0, -20.0, -1.0, -1e-3, -1e-38, 0.0, 1e-38, 1.0, 20.0, 88.0, 150.0, 151.0, 1e30, 8e37, 1e38,
         3.3e38]


@pytest.mark.parametrize("size", [1.0, -1e-3, 1e-30, 1e18, 3e38])
def test_swiglu_over_the_whole_range_of_gates(size):
    """Every gate against many u of one magnitude.  The kernel's steps are three
    exponentials of an ulp and a correction each, and five products: 16 U32.
    What passes bf16's largest value becomes an infinity."""
    g = torch.tensor(GATES, device="cuda").to(BF16)[:, None].expand(-1, 200)
    u = ((torch.rand(len(GATES), 200, generator=gen(1), device="cuda") * 0.9 + 0.1) * size).to(BF16)
    gu = torch.cat([g, u], 1)
    want = ref.swiglu(gu.double())
    rel = 16 * ref.U32
    y = bd.swiglu(gu).double()
    big = want.abs() > BF16_MAX * (1 - ref.U16)
    assert ((y - want).abs() <= (ref.U16 + rel) * want.abs() + ref.TINY16)[~big].all()
    assert (y[big].abs() >= BF16_MAX * (1 - ref.U16)).all() and (y[big].sign() == want[big].sign()).all()
    # Rows whose products pass fp32's range have no 8-bit form.
    fine = (want.abs().amax(1) < float(torch.finfo(torch.float32).max))
    q, scale = bd.swiglu(gu[fine].contiguous(), quantize=True)
    ref.check_quantized(q, scale, want[fine], 1, rel)


def test_swiglu_nonfinite_gates():
    """The formula's own values: an infinite gate passes u's sign on, minus
    infinity and NaN are not numbers."""
    g = torch.tensor([float("inf"), float("-inf"), float("nan"), -300.0])
    y = bd.swiglu(torch.cat([g, torch.full_like(g, -2.0)]).to(BF16).cuda()[None])[0]
    assert y[0] == float("-inf") and y[1].isnan() and y[2].isnan() and y[3] == 0


def test_swiglu_one_low_gate_among_others():
    """A single gate below the exponential's range in a chunk, at each place of a
    row, leaves its neighbours as they are."""
    F = 150
    gu = torch.randn(F, 2 * F, generator=gen(2), device="cuda").to(BF16)
    low = gu.clone()
    i = torch.arange(F, device="cuda")
    low[i, i] = -100.0
    low[i, F + i] = 1e38
    a, b, want = bd.swiglu(gu), bd.swiglu(low), ref.swiglu(low.double())
    keep = ~torch.eye(F, dtype=torch.bool, device="cuda")
    assert torch.equal(a[keep], b[keep])
    assert ((b[i, i].double() - want[i, i]).abs() <= (ref.U16 + 16 * ref.U32) * want[i, i].abs()).all()


@pytest.mark.parametrize("dy_size", [1e-3, 1.0, 1e18, 1e30])
def test_swiglu_backward_over_the_whole_range_of_gates(dy_size):
    """The gradients by the same gates, under gradients and u of any magnitude
    whose formula stays inside bf16's range.  Bounds as for ordinary gates: 32
    U32 of the terms' magnitudes, and the rounding."""
    gates = [g for g in GATES if abs(g) < 1e36 or g < 0]
    g = torch.tensor(gates, device="cuda").to(BF16)[:, None].expand(-1, 200)
    rand = lambda seed: torch.rand(len(gates), 200, generator=gen(seed), device="cuda") * 0.9 + 0.1  # noqa: E731
    dy = (rand(3) * dy_size).to(BF16)
    for size in (1.0, -1e-3, 1e25):
        u = (rand(4) * size).to(BF16)
        want = ref.swiglu_bwd(dy.double(), torch.cat([g, u], 1).double())
        s = 1.0 / (1.0 + torch.exp(-g.double()))
        d = dy.double().abs()
        # t e^g with the exponential's argument bounded: no infinity times zero.
        dg_mag = d * u.double().abs() * s * (1.0 + (g.double().abs() * (1.0 - s)).clamp_max(1e300))
        mag = torch.cat([dg_mag, d * g.double().abs() * s], 1)
        got = bd.swiglu_backward(dy, torch.cat([g, u], 1)).double()
        fine = mag < float(torch.finfo(BF16).max) / 4
        assert ((got - want).abs() <= ref.U16 * want.abs() + 32 * ref.U32 * mag + ref.TINY16)[fine].all()


# -- norm ------------------------------------------------------------------------
def rows_of(sizes, D, seed):
    """A bf16 row of D normal values, limited to 4, for each size."""
    x = torch.randn(len(sizes), D, generator=gen(seed), device="cuda").clamp(-4, 4)
    return (x * torch.tensor(sizes, device="cuda")[:, None]).to(BF16)


@pytest.mark.parametrize("quantize", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("D", [1, 300, 2048, 5005, 9001, 16384, 32761])
def test_rms_norm_rows_of_any_magnitude(D, residual, quantize):
    """Rows whose squares leave fp32's range at either end, with ordinary rows
    between them: the same bounds as anywhere else."""
    sizes = [1e-36, 1.0, 1e-25, 1e-19, 1e18, 1e20, 3.0, 1e30, 2e37]
    eps = 0.0
    x, w = rows_of(sizes, D, D), rows_of([1.0], D, 5)[0].abs() + 0.5
    r = rows_of(sizes, D, D + 1) if residual else None
    out = bd.rms_norm(x, w, residual=r, eps=eps, quantize=quantize, return_rstd=True)
    h, rstd, y = ref.rms_norm(x.double(), None if r is None else r.double(), w.double(), eps)
    rel = (D / 2 + 8) * ref.U32
    # rstd itself is below fp32's normal range where a row's values are at its top: its steps there are 2^-149.
    assert ((out.rstd.double() - rstd).abs() <= rel * rstd + 2.0 ** -149).all()
    rel += 2.0 ** -149 / float(rstd.min())
    if quantize:
        ref.check_quantized(out.y, out.scale, y, 1, rel)
    else:
        assert ((out.y.double() - y).abs() <= (ref.U16 + rel) * y.abs() + ref.TINY16).all()
    # Mixed magnitudes within a row: the large values carry the sum.
    m = x[:3].repeat(1, 1)
    m[:, D // 2] = 1e38
    got, want = bd.rms_norm(m, w, eps=1e-6).y.double(), ref.rms_norm(m.double(), None, w.double(), 1e-6)[2]
    assert ((got - want).abs() <= (ref.U16 + rel) * want.abs() + ref.TINY16)[:, D // 2].all()
