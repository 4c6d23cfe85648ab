"""Cases of the bf16 linear layers around the matrix product, for measurement.

Operators: a linear layer act(x @ w.T + bias) + residual with the activation in
the product's epilogue; its backward pass, as the gradient of its input, taken
through the activation that made the input, and the gradients of weight and
bias; the gated unit act(x @ wg.T) * (x @ wu.T) with both projections in one
product; and its backward pass through the layer that reads it.

Weights are stored with one row per output, ``w[n, k]``; a gated unit's hold the
F rows of the gate and then the F rows of the other factor.  Matrices are
bfloat16, sums 32 bits.

``run`` computes in plain torch while ``own`` is false, and calls the package
while it is true.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
F32 = torch.float32


# -- the cases -----------------------------------------------------------------
def listed():
    return [
        # The second product of a feed-forward block while one sequence
        # generates, the residual stream added on the way: the weight's bytes
        # and the call's latency are the time.
        {"name": "linear_token", "op": "linear", "M": 1, "N": 4096, "K": 8192, "bias": False, "act": "none",
         "residual": True, "keep": False},
        # A short ragged prompt through a first layer, no size a multiple of a tile.
        {"name": "linear_ragged", "op": "linear", "M": 300, "N": 1000, "K": 4112, "bias": True, "act": "gelu",
         "residual": False, "keep": False},
        # The framework's throughput shape as a first layer in training, which
        # keeps what its activation read.
        {"name": "linear_8192", "op": "linear", "M": 8192, "N": 8192, "K": 8192, "bias": True, "act": "gelu_tanh",
         "residual": False, "keep": True},
        # A training step's gradient through the activation between two layers:
        # a ragged batch with an odd inner width.
        {"name": "linear_backward_input_odd", "op": "linear_backward_input", "M": 2047, "N": 1000, "K": 5005,
         "act": "gelu", "residual": False},
        # The same at full width.
        {"name": "linear_backward_input", "op": "linear_backward_input", "M": 8192, "N": 4096, "K": 8192,
         "act": "silu", "residual": False},
        # Weight and bias gradients over an odd number of tokens, odd widths.
        {"name": "linear_backward_weight_odd", "op": "linear_backward_weight", "M": 2047, "N": 1001, "K": 5005,
         "bias": True, "fp32": True},
        # Few output tiles under a long sum over the tokens.
        {"name": "linear_backward_weight", "op": "linear_backward_weight", "M": 32768, "N": 1024, "K": 1024,
         "bias": True, "fp32": True},
        # The first product of a gated block: one sequence generating, a small
        # batch of them, and a long prompt in training, which keeps both factors.
        {"name": "gated_token", "op": "gated", "M": 1, "F": 8192, "K": 4096, "bias": False, "act": "silu",
         "keep": False},
        {"name": "gated_tokens", "op": "gated", "M": 37, "F": 5005, "K": 2048, "bias": False, "act": "silu",
         "keep": False},
        {"name": "gated_prompt", "op": "gated", "M": 8192, "F": 8192, "K": 4096, "bias": False, "act": "silu",
         "keep": True},
        # The gradients of both factors: a ragged batch of an odd width, whose
        # product is wanted again for the weight's gradient, and full width.
        {"name": "gated_backward_input_odd", "op": "gated_backward_input", "M": 2047, "F": 5005, "N": 1000,
         "act": "silu", "again": True},
        {"name": "gated_backward_input", "op": "gated_backward_input", "M": 8192, "F": 8192, "N": 4096,
         "act": "silu", "again": False},
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // step * step if v >= step else v))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward_input", "linear_backward_weight", "gated", "gated",
                     "gated_backward_input"])
    # Mostly multiples of 64, often of 8 only, sometimes odd.
    step = lambda: rng.choice([64, 64, 64, 8, 8, 1])  # noqa: E731
    size = lambda hi=16384: _log(rng, 64, hi, step())  # noqa: E731
    act = rng.choice(["gelu", "gelu_tanh", "silu", "silu", "relu", "none"])
    while True:
        c = {"op": op, "M": _log(rng, 16, 32768) if op == "linear_backward_weight" else _log(rng, 1, 16384)}
        if op.startswith("gated"):
            c["F"] = size(14336)
            c["K" if op == "gated" else "N"] = size(8192)
        else:
            c["N"], c["K"] = size(), size()
        sizes = [c[k] for k in ("M", "N", "K", "F") if k in c]
        if math.prod(sizes) * (2 if op == "gated" else 1) <= 8192 ** 3 and max(
                a * b for a in sizes for b in sizes if a is not b) <= 8192 * 16384:
            break
    if op != "linear_backward_weight":
        c["act"] = act
    if op in ("linear", "linear_backward_weight", "gated"):
        c["bias"] = rng.random() < 0.5
    if op in ("linear", "linear_backward_input"):
        c["residual"] = rng.random() < 0.4
    if op in ("linear", "gated"):
        c["keep"] = rng.random() < 0.4
    if op == "linear_backward_weight":
        c["fp32"] = rng.random() < 0.6
    if op == "gated_backward_input":
        c["again"] = rng.random() < 0.5
    return c


# -- inputs --------------------------------------------------------------------
def _activations(g, rows, cols, size=1.0):
    """Normal values whose channels differ in size, a few of them by much."""
    spread = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    return (torch.randn(rows, cols, generator=g, device="cuda") * (size * spread)).to(BF16)


def _weight(g, rows, cols):
    return (torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5).to(BF16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, M, s = case["op"], case["M"], {"case": case}
    if op in ("linear", "gated"):
        rows = case["N"] if op == "linear" else 2 * case["F"]
        s["x"], s["w"] = _activations(g, M, case["K"]), _weight(g, rows, case["K"])
        s["bias"] = (0.1 * torch.randn(rows, generator=g, device="cuda")).to(BF16) if case["bias"] else None
        if op == "linear":
            s["residual"] = _activations(g, M, case["N"], 4.0) if case["residual"] else None
        return s
    s["dy"] = _activations(g, M, case["N"], 1e-3)
    if op == "linear_backward_weight":
        s["x"] = _activations(g, M, case["K"])
    elif op == "linear_backward_input":
        s["w"] = _weight(g, case["N"], case["K"])
        s["z"] = _activations(g, M, case["K"]) if case["act"] != "none" else None
        s["dresidual"] = _activations(g, M, case["K"], 1e-3) if case["residual"] else None
    else:
        s["w"], s["gu"] = _weight(g, case["N"], case["F"]), _activations(g, M, 2 * case["F"])
    return s


# -- the operators in plain torch ----------------------------------------------
_TANH1 = 2.0 * math.sqrt(2.0 / math.pi)
_TANH3 = 0.044715 * _TANH1


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return z / (1.0 + torch.exp(-(_TANH1 * z + _TANH3 * z * z * z)))
    return z / (1.0 + torch.exp(-z))


def _slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (0.5 / math.pi) ** 0.5
    if act == "gelu_tanh":
        p = 1.0 / (1.0 + torch.exp(-(_TANH1 * z + _TANH3 * z * z * z)))
        return p + z * p * (1.0 - p) * (_TANH1 + 3.0 * _TANH3 * z * z)
    p = 1.0 / (1.0 + torch.exp(-z))
    return p * (1.0 + z * (1.0 - p))


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op in ("linear", "gated"):
        z = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        out = {"kept": z.to(BF16)} if case["keep"] else {}
        if op == "linear":
            y = _act(z, case["act"])
            if s["residual"] is not None:
                y = y + s["residual"].float()
        else:
            gate, up = z.chunk(2, 1)
            y = _act(gate, case["act"]) * up
        out["y"] = y.to(BF16)
        return out
    dy = s["dy"].float()
    if op == "linear_backward_weight":
        dw = dy.t() @ s["x"].float()
        out = {"dw": dw if case["fp32"] else dw.to(BF16)}
        if case["bias"]:
            out["dbias"] = dy.sum(0)
        return out
    t = dy @ s["w"].float()
    if op == "linear_backward_input":
        if s["dresidual"] is not None:
            t = t + s["dresidual"].float()
        if s["z"] is not None:
            t = t * _slope(s["z"].float(), case["act"])
        return {"dx": t.to(BF16)}
    gate, up = s["gu"].float().chunk(2, 1)
    a = _act(gate, case["act"])
    out = {"dgu": torch.cat([t * up * _slope(gate, case["act"]), t * a], 1).to(BF16)}
    if case["again"]:
        out["y"] = (a * up).to(BF16)
    return out


# -- the framework's operators ---------------------------------------------------
def _own(s):
    from pipelined_tiled_dense_amd import binding

    case = s["case"]
    op = case["op"]
    act = None if case.get("act", "none") == "none" else case["act"]
    if op == "linear":
        r = binding.linear(s["x"], s["w"], bias=s["bias"], activation=act, residual=s["residual"],
                           return_preactivation=case["keep"])
        return {"kept": r[1], "y": r[0]} if case["keep"] else {"y": r}
    if op == "gated":
        r = binding.gated_linear(s["x"], s["w"], bias=s["bias"], activation=act, return_gu=case["keep"])
        return {"kept": r[1], "y": r[0]} if case["keep"] else {"y": r}
    if op == "linear_backward_weight":
        r = binding.linear_backward_weight(s["dy"], s["x"], bias=case["bias"],
                                           out_dtype=F32 if case["fp32"] else BF16)
        return {"dw": r[0], "dbias": r[1]} if case["bias"] else {"dw": r}
    if op == "linear_backward_input":
        return {"dx": binding.linear_backward_input(s["dy"], s["w"], preactivation=s["z"], activation=act,
                                                    dresidual=s["dresidual"])}
    r = binding.gated_linear_backward_input(s["dy"], s["w"], s["gu"], activation=act, return_y=case["again"])
    return {"dgu": r[0], "y": r[1]} if case["again"] else {"dgu": r}


def run(state):
    return _own(state) if own else _plain(state)


# -- what a pass cannot do without -----------------------------------------------
def work(case):
    op, M = case["op"], case["M"]
    if op == "linear":
        N, K = case["N"], case["K"]
        outs = 1 + case["keep"] + case["residual"]
        return {"bytes": 2 * (M * K + N * K + M * N * outs + N * case["bias"]), "flops": 2 * M * N * K}
    if op == "gated":
        F, K = case["F"], case["K"]
        return {"bytes": 2 * (M * K + 2 * F * K + M * F * (1 + 2 * case["keep"]) + 2 * F * case["bias"]),
                "flops": 4 * M * F * K}
    N = case["N"]
    if op == "linear_backward_weight":
        K = case["K"]
        return {"bytes": 2 * M * (N + K) + (4 if case["fp32"] else 2) * N * K + 4 * N * case["bias"],
                "flops": 2 * M * N * K}
    if op == "linear_backward_input":
        K = case["K"]
        ins = 1 + (case["act"] != "none") + case["residual"]
        return {"bytes": 2 * (M * N + N * K + M * K * ins), "flops": 2 * M * N * K}
    F = case["F"]
    return {"bytes": 2 * (M * N + N * F + M * F * (4 + case["again"])), "flops": 2 * M * N * F}


# -- the definition in 64 bits ---------------------------------------------------
def _exact_act(z, act):
    """(value, derivative) of the activation."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp_min(0), torch.heaviside(z, torch.zeros_like(z))
    if act == "gelu":
        # z times the normal distribution function, whose derivative is its density.
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        inner = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        # (1 + tanh a) / 2 is the logistic function of 2 a.
        p = torch.sigmoid(2 * inner)
        return z * p, p + 2 * z * p * torch.sigmoid(-2 * inner) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
    p = torch.sigmoid(z)
    return z * p, p + z * p * torch.sigmoid(-z)


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    op = case["op"]
    if op == "linear_backward_weight":
        out = {"dw": torch.mm(d["dy"].t().contiguous(), d["x"])}
        if case["bias"]:
            out["dbias"] = torch.mv(d["dy"].t().contiguous(), torch.ones_like(d["dy"][:, 0]))
        return out
    if op in ("linear", "gated"):
        z = torch.mm(d["x"], d["w"].t().contiguous())
        if "bias" in d:
            z += d["bias"]
        out = {"kept": z} if case["keep"] else {}
        if op == "linear":
            y = _exact_act(z, case["act"])[0]
            out["y"] = y + d["residual"] if "residual" in d else y
        else:
            out["y"] = z[:, case["F"]:] * _exact_act(z[:, : case["F"]], case["act"])[0]
        return out
    t = torch.mm(d["dy"], d["w"])
    if op == "linear_backward_input":
        if "dresidual" in d:
            t += d["dresidual"]
        return {"dx": _exact_act(d["z"], case["act"])[1] * t if "z" in d else t}
    value, slope = _exact_act(d["gu"][:, : case["F"]], case["act"])
    up = d["gu"][:, case["F"]:]
    out = {"dgu": torch.hstack([slope * up * t, value * t])}
    if case["again"]:
        out["y"] = value * up
    return out
