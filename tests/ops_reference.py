"""The 8-bit operators in 64 bits, from their formulas, and the bounds their
results are held to.  Nothing here uses the library.

Bounds.  U16 = 2^-8 is bf16's unit roundoff and U32 = 2^-24 fp32's: a value
rounded once is off by at most that share of itself.  A sum of n terms in fp32,
in any order, is off by at most n * U32 times the sum of the terms' magnitudes;
matrix instructions may cut instead of rounding, which doubles U32 there."""
import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24
FP8_MAX, MIN_SCALE, BLOCK = 448.0, 2.0 ** -126, 128
TINY16 = 2.0 ** -133     # bf16's smallest step


def nblocks(n):
    return -(-n // BLOCK)


def quantized_scale(y, block_rows):
    """(ceil(K / 128), ceil(R / block_rows)) scales of y (R, K)."""
    R, K = y.shape
    s = torch.empty(nblocks(K), -(-R // block_rows), dtype=y.dtype, device=y.device)
    for kb in range(s.shape[0]):
        part = y[:, kb * BLOCK:(kb + 1) * BLOCK].abs().amax(1)
        for rb in range(s.shape[1]) if block_rows > 1 else [slice(None)]:
            if block_rows > 1:
                s[kb, rb] = part[rb * block_rows:(rb + 1) * block_rows].max()
            else:
                s[kb] = part
    return (s / FP8_MAX).clamp_min(MIN_SCALE)


def spread(scale, block_rows, shape):
    """Scales over the (R, K) elements they cover."""
    s = scale.t().repeat_interleave(block_rows, 0)[: shape[0]]
    return s.repeat_interleave(BLOCK, 1)[:, : shape[1]]


def check_quantized(q, scale, y, block_rows, rel):
    """8-bit q and its scales against y in 64 bits, both computed from y with a
    relative error of at most `rel`: the scale carries that error and its own
    rounding, and the value is within half a step of e4m3 (a share of 2^-4, or
    2^-10 below the smallest normal value) of y / scale."""
    want = quantized_scale(y, block_rows)
    got = scale.double()
    assert got.shape == want.shape
    assert ((got - want).abs() <= (rel + 4 * U32) * want).all(), "scales"
    s = spread(got, block_rows, y.shape)
    v = y / s
    err = (q.double() - v).abs()
    bound = torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10) + (rel + 4 * U32) * v.abs()
    bad = err > bound
    assert not bad.any(), "values: %d of %d, worst %g" % (int(bad.sum()), bad.numel(), float((err / bound).max()))


def rms_norm(x, residual, weight, eps):
    h = x if residual is None else x + residual
    rstd = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h, rstd[:, 0], h * rstd * weight


def rms_norm_bwd(dy, h, weight, rstd, dres):
    n = h * rstd[:, None]
    t = dy * weight
    dx = rstd[:, None] * (t - n * (t * n).mean(1, keepdim=True))
    return (dx if dres is None else dx + dres), (dy * n).sum(0)


def swiglu(gu):
    g, u = gu.chunk(2, 1)
    return g / (1.0 + torch.exp(-g)) * u


def swiglu_bwd(dy, gu):
    g, u = gu.chunk(2, 1)
    s = 1.0 / (1.0 + torch.exp(-g))
    return torch.cat([dy * u * s * (1.0 + g * (1.0 - s)), dy * g * s], 1)


def gemm(q_a, scale_a, q_b, scale_b, b_rows):
    """(product, product of the magnitudes)."""
    a = q_a.double() * spread(scale_a.double(), 1, q_a.shape)
    b = q_b.double() * spread(scale_b.double(), b_rows, q_b.shape)
    return torch.mm(a, b.t().contiguous()), torch.mm(a.abs(), b.abs().t().contiguous())
