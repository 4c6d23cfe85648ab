"""The linear layers' operators on the GPU against their 64-bit formulas: values and
gradients at sizes, strides and alignments of every kernel, streams and graphs."""
import itertools

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


@pytest.fixture(autouse=True)
def named(request):
    print("  %s" % request.node.name, flush=True)
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand16(g, rows, cols, pad=0, shift=0, size=1.0):
    """A bf16 (rows, cols) view whose rows are cols + pad apart and start
    `shift` elements into the allocation; what lies around it is NaN."""
    buf = torch.full((rows * (cols + pad) + shift,), float("nan"), dtype=BF16, device="cuda")
    x = buf[shift:].view(rows, cols + pad)[:, :cols]
    x.copy_(torch.randn(rows, cols, generator=g, device="cuda") * size)
    return x


def d(x):
    return None if x is None else x.double()


# (M, N, K): few rows of each kind, tiles of both sizes, split sums, ragged edges.
SHAPES = [(1, 1, 8), (1, 40, 64), (1, 33, 4096), (2, 300, 200), (16, 64, 6400), (17, 72, 136), (32, 256, 520),
          (33, 40, 72), (64, 130, 1024), (65, 64, 64), (65, 130, 200), (127, 255, 320), (128, 128, 4096), (130, 260, 72),
          (200, 1000, 1544), (300, 96, 8200), (513, 1032, 264), (1000, 2000, 640), (2100, 1100, 192), (4099, 4104, 72),
          (4096, 4352, 192), (4360, 4096, 328)]
# Off the 8-element grid, rows apart, rows that start anywhere.
ODD = [(1, 7, 9, 0, 0), (1, 50, 1001, 3, 1), (3, 129, 15, 1, 3), (20, 37, 515, 0, 1), (64, 100, 999, 8, 8), (65, 5, 3, 0, 0),
       (70, 90, 201, 16, 8), (131, 77, 1025, 1, 0), (257, 300, 1000, 1, 1), (600, 257, 513, 24, 8), (4100, 4100, 100, 4, 4)]
SIZES = [(*s, 0, 0) for s in SHAPES] + ODD


def each(n):
    """Activations and options in turn over the cases, all of them on the small ones."""
    return itertools.product(ref.ACTS, (False, True), (False, True)) if n < 200000 else [
        ("gelu", True, False), ("silu", False, True), (None, True, True)]


@pytest.mark.parametrize("M,N,K,pad,shift", SIZES)
def test_linear(M, N, K, pad, shift):
    g = gen(M * 3 + N * 5 + K)
    x, w = rand16(g, M, K, pad, shift), rand16(g, N, K, pad, shift, K ** -0.5)
    b, r = rand16(g, 1, N, 0, shift)[0], rand16(g, M, N, pad, shift, 2.0)
    for act, bias, residual in each(M * N * K):
        want = ref.linear(d(x), d(w), d(b) if bias else None, act, d(r) if residual else None)
        kw = {"bias": b if bias else None, "activation": act, "residual": r if residual else None}
        y, z = bd.linear(x, w, return_preactivation=True, **kw)
        ref.check(y, *want["y"], "y %s" % act)
        ref.check(z, *want["z"], "z")
        assert torch.equal(y, bd.linear(x, w, **kw))


@pytest.mark.parametrize("M,N,K,pad,shift", SIZES)
def test_linear_backward_input(M, N, K, pad, shift):
    M, N, K = M, K, N                # the wide side is the contraction's
    g = gen(M * 3 + N * 5 + K)
    dy, w = rand16(g, M, N, pad, shift), rand16(g, N, K, pad, shift, N ** -0.5)
    z, r = rand16(g, M, K, pad, shift, 2.0), rand16(g, M, K, pad, shift)
    for act, _, residual in each(M * N * K):
        want = ref.linear_backward_input(d(dy), d(w), d(z), act, d(r) if residual else None)
        kw = {"activation": act, "preactivation": z if act else None, "dresidual": r if residual else None}
        got = bd.linear_backward_input(dy, w, **kw)
        ref.check(got, *want, "dx %s" % act)
        assert torch.equal(got, bd.linear_backward_input(dy, w, **kw))


@pytest.mark.parametrize("M,N,K,pad,shift", [(k, m, n, p, s) for m, n, k, p, s in SIZES])
def test_linear_backward_weight(M, N, K, pad, shift):
    g = gen(M * 3 + N * 5 + K)
    dy, x = rand16(g, M, N, pad, shift), rand16(g, M, K, pad, shift)
    want, err = ref.product(d(dy).t(), d(x))
    db = d(dy).sum(0)
    dw, bias = bd.linear_backward_weight(dy, x, bias=True)
    assert dw.dtype == F32 and bias.dtype == F32
    ref.check(dw, want, err, "dw")
    ref.check(bias, db, (M + 4) * ref.U32 * d(dy).abs().sum(0), "dbias")
    dw16 = bd.linear_backward_weight(dy, x, out_dtype=BF16)
    assert dw16.dtype == BF16
    ref.check(dw16, want, ref.rounded(want, err), "dw bf16")
    again, bias2 = bd.linear_backward_weight(dy, x, bias=True)
    assert torch.equal(dw, again) and torch.equal(bias, bias2) and torch.equal(dw.to(BF16), dw16)


@pytest.mark.parametrize("M,F,K,pad,shift", [(m, max(1, n // 2), k, p, s) for m, n, k, p, s in SIZES])
def test_gated_linear(M, F, K, pad, shift):
    g = gen(M * 3 + F * 5 + K)
    x, w = rand16(g, M, K, pad, shift), rand16(g, 2 * F, K, pad, shift, K ** -0.5)
    b = rand16(g, 1, 2 * F, 0, shift)[0]
    for act, bias, _ in each(M * F * K):
        want = ref.gated(d(x), d(w), d(b) if bias else None, act)
        kw = {"bias": b if bias else None, "activation": act}
        y, gu = bd.gated_linear(x, w, return_gu=True, **kw)
        ref.check(gu, *want["gu"], "gu")
        ref.check(y, *want["y"], "y %s" % act)
        assert torch.equal(y, bd.gated_linear(x, w, **kw))


@pytest.mark.parametrize("M,F,N,pad,shift", SIZES)
def test_gated_linear_backward_input(M, F, N, pad, shift):
    g = gen(M * 3 + F * 5 + N)
    dy, w = rand16(g, M, N, pad, shift), rand16(g, N, F, pad, shift, N ** -0.5)
    gu = rand16(g, M, 2 * F, pad, shift, 2.0)
    for act, _, again in each(M * F * N):
        want = ref.gated_backward_input(d(dy), d(w), d(gu), act)
        if again:
            dgu, y = bd.gated_linear_backward_input(dy, w, gu, activation=act, return_y=True)
            ref.check(y, *want["y"], "y %s" % act)
        else:
            dgu = bd.gated_linear_backward_input(dy, w, gu, activation=act)
        ref.check(dgu, *want["dgu"], "dgu %s" % act)
