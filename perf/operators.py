"""Cases of the 8-bit operators around the matrix product, for measurement.

Operators: the root-mean-square norm with the residual's addition (bf16 output,
or 8 bits with a scale for each 128 values) and its gradient; the gated unit
silu(g) * u with the same outputs, and its gradient; the quantisation of
activations, gradients and weights; and the matrix product of 8-bit operands
with a scale for each block of 128.

Scales are stored with the block index along k first: ``scale_a[kb, m]`` scales
``A[m, 128 * kb : 128 * kb + 128]``, and ``scale_b[kb, nb]`` the rows
``128 * nb ..`` (or the single row ``nb``) of B over the same columns.

``run`` computes in plain torch while ``own`` is false, and calls the package
while it is true.
"""
import math

import torch
import torch.nn.functional as F

own = False

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
MIN_SCALE = 2.0 ** -126
EPS = 1e-6


# -- the cases -----------------------------------------------------------------
def listed():
    return [
        # The norm before a product while one sequence generates: a single
        # token, where the call's latency is all there is.
        {"name": "norm_fp8_token", "op": "norm", "rows": 1, "width": 4096, "fp8": True, "residual": True},
        # The same over a long prompt.
        {"name": "norm_fp8_prompt", "op": "norm", "rows": 8192, "width": 8192, "fp8": True, "residual": True},
        # The norm's gradients in a training step, a ragged batch.
        {"name": "norm_backward", "op": "norm_backward", "rows": 8191, "width": 4096, "residual": True},
        # The gated unit before the second product: a few sequences generating,
        # and a prompt.
        {"name": "swiglu_fp8_tokens", "op": "swiglu", "rows": 4, "width": 8192, "fp8": True},
        {"name": "swiglu_fp8_prompt", "op": "swiglu", "rows": 8192, "width": 8192, "fp8": True},
        # Its gradient in a training step, odd sizes off the vector grid.
        {"name": "swiglu_backward", "op": "swiglu_backward", "rows": 2047, "width": 5005},
        # The operands of a weight's gradient: activations quantised along the
        # tokens, transposed on the way.
        {"name": "quantize_transposed", "op": "quantize", "rows": 8192, "cols": 4096, "block_rows": 1,
         "transposed": True},
        # A weight quantised in blocks, odd sizes.
        {"name": "quantize_weight", "op": "quantize", "rows": 1000, "cols": 4040, "block_rows": 128,
         "transposed": False},
        # The product for a single token: the weight's bytes are the time.
        {"name": "gemm_token", "op": "gemm", "M": 1, "N": 8192, "K": 8192, "block_n": 128, "fp32": False},
        # A short ragged prompt, no size a multiple of the tile.
        {"name": "gemm_ragged", "op": "gemm", "M": 300, "N": 1000, "K": 4112, "block_n": 128, "fp32": False},
        # The framework's throughput shape.
        {"name": "gemm_8192", "op": "gemm", "M": 8192, "N": 8192, "K": 8192, "block_n": 128, "fp32": False},
        # A weight's gradient: few output tiles and a long k range, both
        # operands scaled row by row, the sums returned in 32 bits.
        {"name": "gemm_weight_gradient", "op": "gemm", "M": 1024, "N": 1024, "K": 32768, "block_n": 1, "fp32": True},
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // step * step if v >= step else v))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "swiglu", "swiglu_backward", "quantize", "gemm", "gemm", "gemm"])
    # Mostly whole blocks of 128, often a multiple of 16 only, sometimes odd.
    step = lambda: rng.choice([128, 128, 128, 16, 16, 1])  # noqa: E731
    if op == "gemm":
        while True:
            c = {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 128, 8192, step()),
                 "K": _log(rng, 128, 32768, step()), "block_n": rng.choice([128, 128, 1]),
                 "fp32": rng.random() < 0.3}
            if c["M"] * c["N"] * c["K"] <= 8192 ** 3 and (c["M"] + c["N"]) * c["K"] <= 2 * 8192 ** 2:
                return c
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 64, 16384, step()),
                "block_rows": rng.choice([1, 128]), "transposed": rng.random() < 0.5}
    while True:
        c = {"op": op, "rows": _log(rng, 1, 16384), "width": _log(rng, 64, 16384, step())}
        if c["rows"] * c["width"] <= 8192 ** 2:
            break
    if op in ("norm", "swiglu"):
        c["fp8"] = rng.random() < 0.7
    if op in ("norm", "norm_backward"):
        c["residual"] = rng.random() < 0.7
    return c


# -- inputs --------------------------------------------------------------------
def _activations(g, rows, cols, size=1.0):
    """Normal values whose channels differ in size, a few of them by much."""
    spread = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    return (torch.randn(rows, cols, generator=g, device="cuda") * (size * spread)).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, s = case["op"], {"case": case}
    if op == "gemm":
        # Operands as a quantiser leaves them; not timed.
        a = _activations(g, case["M"], case["K"])
        b = (torch.randn(case["N"], case["K"], generator=g, device="cuda") * case["K"] ** -0.5).to(torch.bfloat16)
        s["a"], s["scale_a"] = _quantize(a.float(), 1)
        s["b"], s["scale_b"] = _quantize(b.float(), case["block_n"])
        return s
    if op == "quantize":
        s["x"] = _activations(g, case["rows"], case["cols"])
        return s
    rows, width = case["rows"], case["width"]
    if op == "swiglu":
        s["gu"] = _activations(g, rows, 2 * width)
    elif op == "swiglu_backward":
        s["gu"] = _activations(g, rows, 2 * width)
        s["dy"] = _activations(g, rows, width, 1e-3)
    else:
        s["weight"] = (1.0 + 0.1 * torch.randn(width, generator=g, device="cuda")).to(torch.bfloat16)
        s["x"] = _activations(g, rows, width)
        if op == "norm":
            s["residual"] = _activations(g, rows, width, 4.0) if case["residual"] else None
        else:
            s["dy"] = _activations(g, rows, width, 1e-3)
            s["dresidual"] = _activations(g, rows, width, 1e-3) if case["residual"] else None
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
    return s


# -- the operators in plain torch ----------------------------------------------
def _blocks(x, br):
    """x padded with zeros to whole blocks of br x 128, as [rows/br, br, cols/128, 128]."""
    r, c = x.shape
    x = F.pad(x, (0, -c % 128, 0, -r % br))
    return x.view(x.shape[0] // br, br, x.shape[1] // 128, 128)


def _quantize(x, br):
    """(8-bit values, scales with the k block first) of a 32-bit x."""
    v = _blocks(x, br)
    scale = (v.abs().amax((1, 3), keepdim=True) / FP8_MAX).clamp_min(MIN_SCALE)
    q = (v / scale).clamp(-FP8_MAX, FP8_MAX).to(FP8)
    q = q.view(v.shape[0] * br, -1)[: x.shape[0], : x.shape[1]].contiguous()
    return q, scale[:, 0, :, 0].t().contiguous()


def _dequantize(q, scale, br, dtype):
    """The values that 8-bit q and its scales stand for."""
    s = scale.to(dtype).t().repeat_interleave(br, 0)[: q.shape[0]]
    return q.to(dtype) * s.repeat_interleave(128, 1)[:, : q.shape[1]]


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "gemm":
        c = _dequantize(s["a"], s["scale_a"], 1, torch.float32) @ \
            _dequantize(s["b"], s["scale_b"], case["block_n"], torch.float32).t()
        return {"c": c if case["fp32"] else c.to(torch.bfloat16)}
    if op == "quantize":
        x = s["x"].float()
        q, scale = _quantize(x.t() if case["transposed"] else x, case["block_rows"])
        return {"q": q, "scale": scale}
    if op == "norm":
        h = s["x"].float()
        out = {}
        if s["residual"] is not None:
            h = h + s["residual"].float()
            out["h"] = h.to(torch.bfloat16)
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
        if case["fp8"]:
            out["q"], out["scale"] = _quantize(y, 1)
        else:
            out["y"] = y.to(torch.bfloat16)
        return out
    if op == "norm_backward":
        dy, h, r = s["dy"].float(), s["x"].float(), s["rstd"][:, None]
        n = h * r
        dn = dy * s["weight"].float()
        dx = r * (dn - n * (dn * n).mean(1, keepdim=True))
        if s["dresidual"] is not None:
            dx = dx + s["dresidual"].float()
        return {"dx": dx.to(torch.bfloat16), "dweight": (dy * n).sum(0)}
    g, u = s["gu"].float().chunk(2, 1)
    if op == "swiglu":
        y = g / (1.0 + torch.exp(-g)) * u
        if case["fp8"]:
            q, scale = _quantize(y, 1)
            return {"q": q, "scale": scale}
        return {"y": y.to(torch.bfloat16)}
    dy, p = s["dy"].float(), 1.0 / (1.0 + torch.exp(-g))
    dg = dy * u * p * (1.0 + g * (1.0 - p))
    return {"dgu": torch.cat([dg, dy * g * p], 1).to(torch.bfloat16)}


# -- the framework's operators ---------------------------------------------------
def _own(s):
    from pipelined_tiled_dense_amd import binding

    case = s["case"]
    op = case["op"]
    if op == "gemm":
        return {"c": binding.gemm_fp8(s["a"], s["scale_a"], s["b"], s["scale_b"],
                                      out_dtype=torch.float32 if case["fp32"] else torch.bfloat16)}
    if op == "quantize":
        q, scale = binding.quantize_fp8(s["x"], block_rows=case["block_rows"], transposed=case["transposed"])
        return {"q": q, "scale": scale}
    if op == "norm":
        r = binding.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, quantize=case["fp8"])
        out = {"q": r.y, "scale": r.scale} if case["fp8"] else {"y": r.y}
        if s["residual"] is not None:
            out["h"] = r.h
        return out
    if op == "norm_backward":
        dx, dw = binding.rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], dresidual=s["dresidual"])
        return {"dx": dx, "dweight": dw}
    if op == "swiglu":
        if case["fp8"]:
            q, scale = binding.swiglu(s["gu"], quantize=True)
            return {"q": q, "scale": scale}
        return {"y": binding.swiglu(s["gu"])}
    return {"dgu": binding.swiglu_backward(s["dy"], s["gu"])}


def run(state):
    return _own(state) if own else _plain(state)


# -- what a pass cannot do without -----------------------------------------------
def work(case):
    op = case["op"]
    if op == "gemm":
        M, N, K, kb = case["M"], case["N"], case["K"], -(-case["K"] // 128)
        scales = 4 * kb * (M + -(-N // case["block_n"]))
        return {"bytes": M * K + N * K + scales + M * N * (4 if case["fp32"] else 2), "flops": 2 * M * N * K}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": 3 * n + 4 * n // (128 * case["block_rows"]), "flops": 3 * n}
    n, w = case["rows"] * case["width"], case["width"]
    fp8 = case.get("fp8", False)
    out = n + 4 * case["rows"] * -(-w // 128) if fp8 else 2 * n
    if op == "norm":
        return {"bytes": 2 * n + (4 * n if case["residual"] else 0) + 2 * w + out, "flops": 6 * n}
    if op == "norm_backward":
        return {"bytes": 6 * n + (2 * n if case["residual"] else 0) + 4 * case["rows"] + 6 * w, "flops": 9 * n}
    if op == "swiglu":
        return {"bytes": 4 * n + out, "flops": 8 * n}
    return {"bytes": 10 * n, "flops": 12 * n}


# -- the definition in 64 bits ---------------------------------------------------
def _exact_quantized(y, br):
    """Scales and nearest 8-bit values, block by block of the definition."""
    r, c = y.shape
    rb, cb = torch.arange(r, device=y.device) // br, torch.arange(c, device=y.device) // 128
    top = torch.zeros(int(rb[-1]) + 1, c, dtype=y.dtype, device=y.device)
    top = top.index_reduce(0, rb, y.abs(), "amax")
    big = torch.zeros(int(cb[-1]) + 1, top.shape[0], dtype=y.dtype, device=y.device)
    big = big.index_reduce(0, cb, top.t().contiguous(), "amax")
    scale = torch.maximum(big / FP8_MAX, torch.full_like(big, MIN_SCALE))
    v = y / scale.t()[rb][:, cb]
    # Three bits below the leading one, and a fixed grid of 2^-9 below 2^-6.
    _, e = torch.frexp(v)
    grid = torch.ldexp(torch.ones_like(v), (e - 4).clamp_min(-9))
    return torch.round(v / grid) * grid, scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if op == "gemm":
        def values(q, scale, br):
            m = torch.arange(q.shape[0], device=q.device) // br
            k = torch.arange(q.shape[1], device=q.device) // 128
            return q * scale[k][:, m].t()
        return {"c": torch.mm(values(d["a"], d["scale_a"], 1), values(d["b"], d["scale_b"], case["block_n"]).t())}
    if op == "quantize":
        q, scale = _exact_quantized(d["x"].t() if case["transposed"] else d["x"], case["block_rows"])
        return {"q": q, "scale": scale}
    if op == "norm":
        out = {}
        h = d["x"]
        if "residual" in d:
            h = out["h"] = h + d["residual"]
        y = d["weight"] * h / torch.sqrt((h * h).sum(1, keepdim=True) / h.shape[1] + EPS)
        if case["fp8"]:
            out["q"], out["scale"] = _exact_quantized(y, 1)
        else:
            out["y"] = y
        return out
    if op == "norm_backward":
        # With n = h * rstd: dL/dh = rstd * (w dy - n * <w dy, n> / width), dL/dw = sum over rows of dy n.
        n = d["x"] * d["rstd"].unsqueeze(1)
        t = d["weight"] * d["dy"]
        dx = d["rstd"].unsqueeze(1) * (t - n * ((t * n).sum(1, keepdim=True) / n.shape[1]))
        if "dresidual" in d:
            dx = dx + d["dresidual"]
        return {"dx": dx, "dweight": (d["dy"] * n).sum(0)}
    w = case["width"]
    g, u = d["gu"][:, :w], d["gu"][:, w:]
    p = torch.sigmoid(g)
    if op == "swiglu":
        if case["fp8"]:
            q, scale = _exact_quantized(g * p * u, 1)
            return {"q": q, "scale": scale}
        return {"y": g * p * u}
    # d silu(g) / dg = p + g p (1 - p).
    return {"dgu": torch.hstack([d["dy"] * u * (p + g * p * (1 - p)), d["dy"] * g * p])}
