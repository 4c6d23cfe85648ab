"""The 8-bit operators on the GPU against their 64-bit formulas: values,
gradients, scales, layouts, masked and degenerate sizes, streams and graphs."""
import pytest
import torch

import ops_reference as ref
from pipelined_tiled_dense_amd import binding as bd

pytestmark = pytest.mark.gpu

BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn


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


# -- norm ------------------------------------------------------------------------
WIDTHS = [1, 7, 8, 127, 128, 129, 512, 520, 1000, 2048, 4096, 5005, 8192, 16384, 32768]


@pytest.mark.parametrize("quantize", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("D", WIDTHS)
def test_rms_norm(D, residual, quantize):
    for M, pad, shift in ((1, 0, 0), (5, 3, 1), (600, 8, 8)):
        g = gen(D + M)
        x = rand16(g, M, D, pad, shift)
        r = rand16(g, M, D, pad + 1, shift, 3.0) if residual else None
        w = rand16(g, 1, D, 0, shift)[0]
        out = bd.rms_norm(x, w, residual=r, eps=1e-5, quantize=quantize, return_rstd=True)
        h, rstd, y = ref.rms_norm(x.double(), None if r is None else r.double(), w.double(), 1e-5)
        rel = (D / 2 + 8) * ref.U32
        assert ((out.rstd.double() - rstd).abs() <= rel * rstd).all()
        if residual:
            assert torch.equal(out.h, (x.float() + r.float()).to(BF16))
        else:
            assert out.h is None
        # h itself rounds to fp32 where there is a residual: an error in
        # proportion to h, as every other step's.
        if quantize:
            ref.check_quantized(out.y, out.scale, y, 1, rel)
        else:
            assert ((out.y.double() - y).abs() <= (ref.U16 + rel) * y.abs() + ref.TINY16).all()


def test_rms_norm_in_place():
    """The residual stream updated where it lies, through the C entry point."""
    g = gen(3)
    for M, D in ((3, 640), (700, 4096), (2, 20000)):
        x, r, w = rand16(g, M, D), rand16(g, M, D), rand16(g, 1, D)[0]
        want = bd.rms_norm(x, w, residual=r)
        for target in ("x", "residual"):
            xs, rs = x.clone(), r.clone()
            h = xs if target == "x" else rs
            y = torch.empty_like(x)
            st = torch.cuda.current_stream().cuda_stream
            assert bd.gemm_rms_norm(M, D, xs.data_ptr(), D, rs.data_ptr(), D, w.data_ptr(), 1e-6, h.data_ptr(), D,
                                    y.data_ptr(), D, bd.TYPE_BF16, None, 0, None, st) == bd.GEMM_OK
            assert torch.equal(h, want.h) and torch.equal(y, want.y)


def test_rms_norm_zero_and_nonfinite_rows():
    """A row of zeros gives zeros (eps keeps rstd finite), a NaN or an infinity
    stays in its row, and values next to fp32's range do not overflow the sum."""
    x = torch.ones(5, 300, dtype=BF16, device="cuda")
    x[1] = 0.0
    x[2, 7] = float("nan")
    x[3, 150] = float("inf")
    x[4] = 1e-30
    w = torch.ones(300, dtype=BF16, device="cuda")
    y = bd.rms_norm(x, w, eps=1e-6).y
    assert torch.allclose(y[0].float(), torch.ones(300, device="cuda"), atol=1e-5)
    assert (y[1] == 0).all()
    assert y[2].isnan().all() and y[3, 150].isnan()
    assert y[4].isfinite().all()
    q = bd.rms_norm(x, w, eps=1e-6, quantize=True)
    v = q.y.float() * ref.spread(q.scale, 1, x.shape)
    assert (v[1] == 0).all() and q.scale.isfinite()[:, [0, 1, 4]].all()
    assert not v[2].isfinite().any()
    assert not v[3, 128:256].isfinite().any()


@pytest.mark.parametrize("dres", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("D", WIDTHS)
def test_rms_norm_backward(D, dres):
    for M, pad, shift in ((1, 0, 0), (5, 3, 1), (2100 if D <= 5005 else 530, 8, 8)):
        g = gen(D + M)
        dy, h = rand16(g, M, D, pad, shift), rand16(g, M, D, pad + 1, shift, 2.0)
        s = rand16(g, M, D, pad, shift) if dres else None
        w = rand16(g, 1, D)[0]
        rstd = (1.0 / torch.sqrt((h.double() ** 2).mean(1) + 1e-6)).float()
        dx, dw = bd.rms_norm_backward(dy, h, w, rstd, dresidual=s)
        a = [t.double() for t in (dy, h, w, rstd)]
        want_dx, want_dw = ref.rms_norm_bwd(*a, None if s is None else s.double())
        n = (a[1] * a[3][:, None]).abs()
        t = (a[0] * a[2]).abs()
        # Terms of dx: rstd * t, rstd * n * mean (a sum of D terms), dres.
        mag = a[3][:, None] * (t + n * (t * n).mean(1, keepdim=True)) + (0 if s is None else s.double().abs())
        assert ((dx.double() - want_dx).abs() <= ref.U16 * want_dx.abs() + (D + 8) * ref.U32 * mag + ref.TINY16).all()
        assert ((dw.double() - want_dw).abs() <= (M + 4) * ref.U32 * (a[0].abs() * n).sum(0)).all()
        again = bd.rms_norm_backward(dy, h, w, rstd, dresidual=s)
        assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def test_rms_norm_backward_against_differences():
    """The change of a 64-bit loss along random directions, by central
    differences, against the gradients the kernel returns."""
    g = gen(11)
    M, D, eps, step = 6, 384, 1e-5, 1e-4
    x, r, w = rand16(g, M, D), rand16(g, M, D), rand16(g, 1, D)[0]
    c, e = rand16(g, M, D), rand16(g, M, D)
    hx = (x.float() + r.float()).to(BF16)          # what the backward pass reads
    rstd = bd.rms_norm(hx, w, eps=eps, return_rstd=True).rstd
    dx, dw = bd.rms_norm_backward(c, hx, w, rstd, dresidual=e)

    def loss(h, weight):
        _, _, y = ref.rms_norm(h, None, weight, eps)
        return (y * c.double()).sum() + (h * e.double()).sum()

    for seed in range(4):
        v = torch.randn(M, D, generator=gen(seed), device="cuda").double()
        u = torch.randn(D, generator=gen(100 + seed), device="cuda").double()
        hd, wd = hx.double(), w.double()
        num = (loss(hd + step * v, wd + step * u) - loss(hd - step * v, wd - step * u)) / (2 * step)
        got = (dx.double() * v).sum() + (dw.double() * u).sum()
        bound = 2 * ref.U16 * (dx.double() * v).abs().sum() + 1e-5 * (dw.double() * u).abs().sum()
        assert abs(float(num - got)) <= float(bound) + 1e-6 * abs(float(num))


def test_rms_norm_backward_of_no_rows_writes_zeros():
    z = torch.empty(0, 300, dtype=BF16, device="cuda")
    w = torch.ones(300, dtype=BF16, device="cuda")
    dx, dw = bd.rms_norm_backward(z, z, w, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 300) and (dw == 0).all()
    assert bd.rms_norm(z, w).y.shape == (0, 300)


# -- gated unit --------------------------------------------------------------------
@pytest.mark.parametrize("F", [1, 7, 8, 127, 128, 129, 1000, 4096, 5005])
def test_swiglu(F):
    for M, pad, shift in ((1, 0, 0), (3, 5, 1), (333, 8, 8)):
        g = gen(F + M)
        gu = rand16(g, M, 2 * F, pad, shift, 4.0)
        y = ref.swiglu(gu.double())
        got = bd.swiglu(gu)
        rel = 16 * ref.U32
        assert ((got.double() - y).abs() <= (ref.U16 + rel) * y.abs() + ref.TINY16).all()
        q, scale = bd.swiglu(gu, quantize=True)
        ref.check_quantized(q, scale, y, 1, rel)
        dy = rand16(g, M, F, pad, shift)
        want, have = ref.swiglu_bwd(dy.double(), gu.double()), bd.swiglu_backward(dy, gu)
        # 1 + g (1 - s) cancels where the gradient of silu crosses zero: the
        # error goes with the magnitudes of its two terms.
        gd, ud = gu.double().chunk(2, 1)
        s = 1.0 / (1.0 + torch.exp(-gd))
        mag = torch.cat([(dy.double() * ud).abs() * s * (1.0 + gd.abs() * (1.0 - s)), (dy.double() * gd).abs() * s], 1)
        assert ((have.double() - want).abs() <= ref.U16 * want.abs() + 2 * rel * mag + ref.TINY16).all()


def test_swiglu_extremes():
    """Gates at the ends of the exponential's range, zeros, and what is not a
    number: silu(-large) is 0, silu(large) the gate itself."""
    g = torch.tensor([-3e38, -1000.0, -100.0, -88.0, -1.0, 0.0, 1.0, 88.0, 200.0, 1e30, float("inf"), float("nan")])
    gu = torch.cat([g, torch.ones_like(g)]).to(BF16).cuda()[None]
    y = bd.swiglu(gu)[0].double()
    want = ref.swiglu(gu.double())[0]
    fine = torch.arange(3, 10)
    assert ((y - want)[fine].abs() <= (ref.U16 + 16 * ref.U32) * want[fine].abs()).all()
    # Below -87 the true value is under 2^-118; the kernel's stays under 2^-110 of the gate.
    assert (y[:3].abs() <= 2.0 ** -110 * g[:3].abs().double().cuda()).all()
    assert y[10] == float("inf") and y[11].isnan()
    d = bd.swiglu_backward(torch.ones(1, 12, dtype=BF16, device="cuda"), gu)[0]
    assert d[:10].isfinite().all() and d[12:22].isfinite().all()


def test_swiglu_backward_against_differences():
    g = gen(5)
    gu, c = rand16(g, 4, 2 * 200, size=2.0), rand16(g, 4, 200)
    d = bd.swiglu_backward(c, gu).double()
    for seed in range(4):
        v = torch.randn(4, 400, generator=gen(seed), device="cuda").double()
        num = ((ref.swiglu(gu.double() + 1e-5 * v) - ref.swiglu(gu.double() - 1e-5 * v)) * c.double()).sum() / 2e-5
        assert abs(float((d * v).sum() - num)) <= 2 * ref.U16 * float((d * v).abs().sum())


def test_swiglu_backward_in_place():
    g = gen(6)
    gu, dy = rand16(g, 37, 2 * 1000), rand16(g, 37, 1000)
    want = bd.swiglu_backward(dy, gu)
    assert bd.gemm_swiglu_bwd(37, 1000, dy.data_ptr(), 1000, gu.data_ptr(), 2000, gu.data_ptr(), 2000,
                              torch.cuda.current_stream().cuda_stream) == bd.GEMM_OK
    assert torch.equal(gu, want)


# -- quantisation --------------------------------------------------------------------
@pytest.mark.parametrize("transposed", [False, True], ids=["straight", "transposed"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 300), (7, 8), (127, 129), (128, 128), (129, 127), (300, 1000),
                                 (1000, 2048), (2049, 136)])
def test_quantize(M, K, block_rows, transposed):
    for pad, shift in ((0, 0), (3, 1)):
        x = rand16(gen(M + K), M, K, pad, shift)
        q, scale = bd.quantize_fp8(x, block_rows=block_rows, transposed=transposed)
        y = (x.t() if transposed else x).double()
        ref.check_quantized(q, scale, y.contiguous(), block_rows, 0.0)


def test_quantize_exact_values():
    """Values that e4m3 holds, with a largest of 448 in every block, come back
    as they are under a scale of exactly 1; ties go to the even neighbour."""
    every = torch.arange(256, dtype=torch.uint8).view(FP8).float()
    every = every[every.isfinite()].repeat(2)[:384].cuda()
    x = every[torch.randperm(384, generator=gen(1), device="cuda").expand(256, 384)].to(BF16)
    x[:, ::128] = 448.0
    for kw in ({}, {"block_rows": 128}):
        q, scale = bd.quantize_fp8(x, **kw)
        assert (scale == 1.0).all() and torch.equal(q.float(), x.float())
    t = torch.tensor([448.0, 17.0, 19.0, 2.125, 2.375, 0.0009765625, 0.0029296875] + [0.0] * 121)
    q, _ = bd.quantize_fp8(t[None].to(BF16).cuda())
    assert q[0, :7].float().tolist() == [448.0, 16.0, 20.0, 2.0, 2.5, 0.0, 0.00390625]


def test_quantize_zero_tiny_and_nonfinite_blocks():
    x = torch.zeros(256, 512, dtype=BF16, device="cuda")
    x[0, 128:256] = 1e-39                # below the smallest scale times 448
    x[1, 256] = float("nan")
    x[2, 300] = float("-inf")
    x[3, 384:] = 3e38
    for kw in ({}, {"transposed": True}, {"block_rows": 128}, {"block_rows": 128, "transposed": True}):
        q, scale = bd.quantize_fp8(x, **kw)
        v = q.float() * ref.spread(scale, kw.get("block_rows", 1), q.shape)
        v = v.t() if kw.get("transposed") else v
        assert not v[1, 256].isfinite() and not v[2, 300].isfinite()
        fine = torch.ones_like(v, dtype=torch.bool)
        fine[:128, 256:384] = False      # the blocks that may share a scale with them
        assert v[fine].isfinite().all()
        assert (v[200:] == 0).all() and (v[3, 384:] - 3e38).abs().max() < 3e38 * 2.0 ** -4
        assert (scale[scale.isfinite()] >= ref.MIN_SCALE).all()


# -- product ---------------------------------------------------------------------------
def fp8_operand(g, rows, K, br, pad=0, shift=0):
    """Random e4m3 values and scales; rows K + pad apart, NaN bytes around."""
    buf = torch.full((rows * (K + pad) + shift,), 0x7F, dtype=torch.uint8, device="cuda")
    q = buf[shift:].view(rows, K + pad)[:, :K]
    q.copy_((torch.randn(rows, K, generator=g, device="cuda") * 20).to(FP8).view(torch.uint8))
    cols = -(-rows // br)
    sbuf = torch.full((ref.nblocks(K), cols + pad), float("nan"), device="cuda")
    scale = sbuf[:, :cols]
    scale.copy_(torch.rand(ref.nblocks(K), cols, generator=g, device="cuda") + 0.25)
    return q.view(FP8), scale


SHAPES = [(1, 1, 16), (1, 16, 128), (1, 1000, 1024), (1, 8, 2064), (3, 129, 272), (16, 256, 4096), (17, 100, 1040),
          (31, 4096, 512), (33, 130, 256), (64, 640, 8192), (65, 65, 128), (127, 255, 384), (128, 128, 2048),
          (129, 257, 400), (300, 1000, 4112), (513, 384, 1152), (1024, 1024, 16384), (4200, 4100, 640)]


@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_fp8(M, N, K, b_rows):
    g = gen(M * 3 + N * 5 + K)
    a, sa = fp8_operand(g, M, K, 1)
    b, sb = fp8_operand(g, N, K, b_rows)
    want, mag = ref.gemm(a, sa, b, sb, b_rows)
    slack = (K + ref.nblocks(K) + 4) * 2 * ref.U32 * mag
    c = bd.gemm_fp8(a, sa, b, sb, out_dtype=torch.float32)
    assert ((c.double() - want).abs() <= slack).all()
    c16 = bd.gemm_fp8(a, sa, b, sb)
    assert c16.dtype == BF16 and ((c16.double() - want).abs() <= ref.U16 * want.abs() + slack + ref.TINY16).all()
    assert torch.equal(c, bd.gemm_fp8(a, sa, b, sb, out_dtype=torch.float32))
    assert torch.equal(c16, bd.gemm_fp8(a, sa, b, sb))


@pytest.mark.parametrize("M,N,K,pad,shift", [(1, 33, 17, 0, 0), (3, 50, 129, 1, 1), (70, 90, 200, 16, 8), (40, 8, 2000, 7, 0),
                                             (200, 300, 1001, 0, 0), (513, 129, 127, 5, 3), (256, 256, 512, 16, 0),
                                             (20, 256, 512, 16, 0), (300, 260, 1000, 24, 16)])
def test_gemm_fp8_strides_and_alignment(M, N, K, pad, shift):
    """K off the 16-byte grid, strides, unaligned operands, padded scales, and an
    output in a wider buffer whose other columns stay as they are."""
    for b_rows in (128, 1):
        g = gen(M + N + K)
        a, sa = fp8_operand(g, M, K, 1, pad, shift)
        b, sb = fp8_operand(g, N, K, b_rows, pad, shift)
        want, mag = ref.gemm(a, sa, b, sb, b_rows)
        for dtype in (torch.float32, BF16):
            buf = torch.full((M, N + 5), 7.0, dtype=dtype, device="cuda")
            c = bd.gemm_fp8(a, sa, b, sb, out=buf[:, 1:N + 1])
            u = ref.U16 if dtype == BF16 else 0.0
            assert ((c.double() - want).abs() <= u * want.abs() + (K + 8) * 2 * ref.U32 * mag + ref.TINY16).all()
            assert (buf[:, 0] == 7.0).all() and (buf[:, N + 1:] == 7.0).all()


@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("M,N,K", [(1, 40, 2048), (5, 64, 1168), (20, 200, 2944), (50, 96, 640), (100, 130, 1296),
                                   (260, 520, 5000), (2100, 4400, 272), (1024, 1024, 4096)])
def test_gemm_fp8_exact(M, N, K, b_rows):
    """Whole numbers and scales that are powers of two: every partial sum fits
    fp32, so the product is exact, to the last element and k."""
    g = gen(K)
    a = torch.randint(-4, 5, (M, K), generator=g, device="cuda").float().to(FP8)
    b = torch.randint(-4, 5, (N, K), generator=g, device="cuda").float().to(FP8)
    cols = -(-N // b_rows)
    sa = 2.0 ** torch.randint(-2, 3, (ref.nblocks(K), M), generator=g, device="cuda").float()
    sb = 2.0 ** torch.randint(-2, 3, (ref.nblocks(K), cols), generator=g, device="cuda").float()
    want, _ = ref.gemm(a, sa, b, sb, b_rows)
    assert torch.equal(bd.gemm_fp8(a, sa, b, sb, out_dtype=torch.float32).double(), want)


@pytest.mark.parametrize("M,N,K,b_rows", [(5, 130, 13952, 128), (33, 99, 9001, 1), (1, 250, 20000, 128), (64, 32, 32768, 1),
                                          (250, 2600, 1040, 128)])
def test_gemm_fp8_few_rows_split_k(M, N, K, b_rows):
    """A long k against a few columns, whose k range several workgroups share, and
    a C of as many tiles as the device has compute units: whole numbers again, so
    every order of the sums gives the same; twice, for the kept memory."""
    g = gen(K + N)
    a = torch.randint(-4, 5, (M, K), generator=g, device="cuda").float().to(FP8)
    b = torch.randint(-4, 5, (N, K), generator=g, device="cuda").float().to(FP8)
    sa = 2.0 ** torch.randint(-1, 1, (ref.nblocks(K), M), generator=g, device="cuda").float()
    sb = 2.0 ** torch.randint(-1, 1, (ref.nblocks(K), -(-N // b_rows)), generator=g, device="cuda").float()
    want, _ = ref.gemm(a, sa, b, sb, b_rows)
    for _ in range(2):
        buf = torch.full((M, N + 3), 7.0, device="cuda")
        assert torch.equal(bd.gemm_fp8(a, sa, b, sb, out=buf[:, :N]).double(), want)
        assert (buf[:, N:] == 7.0).all()
        assert torch.equal(bd.gemm_fp8(a, sa, b, sb), want.float().to(BF16))


def test_gemm_fp8_nonfinite_operands_stay_in_their_rows():
    """NaN in one row of A and one of B, and an infinite scale: they reach the
    row and columns they belong to and nothing else."""
    for M, N, K in ((10, 200, 512), (150, 300, 512), (300, 260, 500)):
        g = gen(M)
        a, sa = fp8_operand(g, M, K, 1)
        b, sb = fp8_operand(g, N, K, 1)
        a.view(torch.uint8)[3, 17] = 0x7F
        b.view(torch.uint8)[100, 400] = 0x7F
        sa[1, 5] = float("inf")
        c = bd.gemm_fp8(a, sa, b, sb)
        assert c[3].isnan().all() and c[:, 100].isnan().all() and not c[5].isfinite().any()
        keep = torch.ones_like(c, dtype=torch.bool)
        keep[[3, 5]] = False
        keep[:, 100] = False
        assert c[keep].isfinite().all()


def test_gemm_fp8_empty_sizes():
    for M, N, K in ((0, 5, 128), (5, 0, 128), (0, 0, 0)):
        a, b = torch.empty(M, K, device="cuda").to(FP8), torch.empty(N, K, device="cuda").to(FP8)
        k = ref.nblocks(K)
        c = bd.gemm_fp8(a, torch.empty(k, M, device="cuda"), b, torch.empty(k, N, device="cuda"))
        assert c.shape == (M, N)
    for dtype in (BF16, torch.float32):
        out = torch.full((5, 9), 3.0, dtype=dtype, device="cuda")
        a, b = torch.empty(5, 0, device="cuda").to(FP8), torch.empty(9, 0, device="cuda").to(FP8)
        bd.gemm_fp8(a, torch.empty(0, 5, device="cuda"), b, torch.empty(0, 9, device="cuda"), out=out)
        assert (out == 0).all() and not out.signbit().any()


# -- streams and graphs --------------------------------------------------------------
def test_streams():
    """Calls on a stream of their own, with work queued ahead of them there,
    give what the calls on the current stream give."""
    g = gen(21)
    x, w = rand16(g, 500, 2048), rand16(g, 1, 2048)[0]
    wq, ws = bd.quantize_fp8(rand16(g, 1024, 2048), block_rows=128)
    n = bd.rms_norm(x, w, quantize=True)
    want = bd.gemm_fp8(n.y, n.scale, wq, ws)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    src = torch.zeros_like(x)
    with torch.cuda.stream(st):
        torch.cuda._sleep(2_000_000)
        src.copy_(x)
    m = bd.rms_norm(src, w, quantize=True, stream=st)
    got = bd.gemm_fp8(m.y, m.scale, wq, ws, stream=st)
    st.synchronize()
    assert torch.equal(got, want)


def test_graph_replay():
    """A norm, a split product and both gradients captured once: every replay,
    with eager calls and synchronisations in between, gives the eager result."""
    g = gen(22)
    M, D = 200, 8192
    x, r, w = rand16(g, M, D), rand16(g, M, D), rand16(g, 1, D)[0]
    wq, ws = bd.quantize_fp8(rand16(g, 512, D), block_rows=128)

    def step():
        n = bd.rms_norm(x, w, residual=r, quantize=True, return_rstd=True)
        c = bd.gemm_fp8(n.y, n.scale, wq, ws)
        y = bd.swiglu(c)
        return [n.h, c, y, bd.swiglu_backward(y, c), *bd.rms_norm_backward(x, n.h, w, n.rstd, dresidual=r)]

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = step()
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
