"""The linear layers' operators in 64 bits, from their formulas, and the bounds
their results are held to.  Nothing here uses the library.

Bounds, beside those of ops_reference.  A product of n terms a row is off by at most
(n + 4) * 2 * U32 times the sum of the terms' magnitudes.  An activation's slope is
below 1.13, so its argument's error enters a value times that; ``activation`` gives
what its own evaluation in fp32 may add:

  logistic   z p(v) with an exponential whose argument is right to 8 U32 |v| and 16
             roundings beside it: the share (16 + 8 |v| (1 - p)) U32, since where p
             is near 1 the exponential hardly enters;
  normal     the tail h exp(-a^2 / 2) from a polynomial right to 1.6e-5 = 269 U32, an
             argument right to 2 U32 a^2 and a few roundings: (300 + 2 a^2) U32 of
             the tail, beside roundings of the whole."""
import math

import torch

from ops_reference import TINY16, U16, U32

ACTS = [None, "relu", "gelu", "gelu_tanh", "silu"]
STEEPEST = 1.13


def activation(z, act):
    """(value, slope, error of the value, error of the slope) at z."""
    zero = torch.zeros_like(z)
    if act is None:
        return z, torch.ones_like(z), zero, zero
    if act == "relu":
        return z.clamp_min(0), (z > 0).to(z.dtype), zero, zero
    if act == "gelu":
        a = z.abs()
        phi = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        tail, cdf = 0.5 * torch.erfc(a / math.sqrt(2)), 0.5 * torch.erfc(-z / math.sqrt(2))
        share = (300 + 2 * a * a) * U32
        value, slope = z * cdf, cdf + z * phi
        return value, slope, a * tail * share + 4 * U32 * value.abs(), (tail + a * phi) * share + 4 * U32 * slope.abs()
    if act == "gelu_tanh":
        k = 2 * math.sqrt(2 / math.pi)
        v, dv = k * (z + 0.044715 * z ** 3), k * (1 + 3 * 0.044715 * z ** 2)
    else:
        v, dv = z, torch.ones_like(z)
    p, q = torch.sigmoid(v), torch.sigmoid(-v)
    share = (16 + 8 * v.abs() * q) * U32
    bend = p * q * (z * dv).abs()
    return z * p, p + z * dv * p * q, (z * p).abs() * share, p * share + bend * (32 + 16 * v.abs()) * U32


def product(a, b):
    """(a @ b, bound of its error) for 64-bit a and b."""
    return torch.mm(a, b.contiguous()), (a.shape[1] + 4) * 2 * U32 * torch.mm(a.abs(), b.abs().contiguous())


def rounded(want, err):
    """The bound of a bf16 result whose fp32 value is off by at most err."""
    return err + U16 * (want.abs() + err) + TINY16


def check(got, want, bound, what=""):
    d = (got.double() - want).abs()
    bad = ~(d <= bound)
    assert not bad.any(), "%s: %d of %d, worst %g at %s" % (
        what, int(bad.sum()), bad.numel(), float((d / bound).nan_to_num(float("inf")).max()),
        tuple(torch.nonzero(bad)[0].tolist()))


def linear(x, w, bias, act, residual):
    """{name: (value, bound)} of y and z."""
    z, err = product(x, w.t())
    if bias is not None:
        z = z + bias
        err = err + U32 * z.abs()
    y, _, own, _ = activation(z, act)
    e = STEEPEST * err + own
    if residual is not None:
        y = y + residual
        e = e + U32 * y.abs()
    return {"y": (y, rounded(y, e)), "z": (z, rounded(z, err))}


def linear_backward_input(dy, w, z, act, dres):
    t, err = product(dy, w)
    if dres is not None:
        t = t + dres
        err = err + U32 * t.abs()
    if act is None:
        return t, rounded(t, err)
    _, slope, _, own = activation(z, act)
    dx = t * slope
    return dx, rounded(dx, slope.abs() * err + (t.abs() + err) * own + 4 * U32 * dx.abs())


def gated(x, w, bias, act):
    gu, err = product(x, w.t())
    if bias is not None:
        gu = gu + bias
        err = err + U32 * gu.abs()
    (g, u), (eg, eu) = gu.chunk(2, 1), err.chunk(2, 1)
    value, _, own, _ = activation(g, act)
    eg = STEEPEST * eg + own
    y = value * u
    return {"y": (y, rounded(y, eg * (u.abs() + eu) + value.abs() * eu + 4 * U32 * y.abs())),
            "gu": (gu, rounded(gu, err))}


def gated_backward_input(dy, w, gu, act):
    t, err = product(dy, w)
    g, u = gu.chunk(2, 1)
    value, slope, ev, es = activation(g, act)
    tt = t.abs() + err
    dg, du, y = t * u * slope, t * value, value * u
    return {"dgu": (torch.cat([dg, du], 1),
                    torch.cat([rounded(dg, u.abs() * (slope.abs() * err + tt * es) + 4 * U32 * dg.abs()),
                               rounded(du, value.abs() * err + tt * ev + 4 * U32 * du.abs())], 1)),
            "y": (y, rounded(y, u.abs() * ev + 4 * U32 * y.abs()))}
