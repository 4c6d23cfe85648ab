"""A gated feed-forward block on the 8-bit operators, for serving and training:

    h = x + residual,  n = rms_norm(h) * w,  [g, u] = n @ Wgu.T,
    out = (silu(g) * u) @ Wd.T

Both products run on 8-bit operands: activations and gradients quantised in
blocks of 128 along the contraction as they are made, weights once, in blocks
of 128 x 128.  ``python -m pipelined_tiled_dense_amd.mlp`` fits a small block to
random data and then serves single tokens with it.
"""
from __future__ import annotations

from typing import NamedTuple

from . import binding


class Gradients(NamedTuple):
    x: object          # bfloat16 (M, D), of x and of residual alike
    norm: object       # float32 (D,)
    gate_up: object    # float32 (2F, D)
    down: object       # float32 (D, F)


class FeedForward:
    """The block with bfloat16 weights ``norm`` (D,), ``gate_up`` (2F, D) and
    ``down`` (D, F).  ``training`` also keeps the transposed weights that the
    gradients of the activations read; ``exact`` computes every product with
    fp32's sums (see ``binding.gemm_fp8``)."""

    def __init__(self, norm, gate_up, down, *, eps=1e-6, training=False, exact=False):
        self.eps, self.training, self.exact = eps, training, exact
        self.set_weights(norm, gate_up, down)

    def set_weights(self, norm, gate_up, down):
        """Lays the weights out: call it after every change of theirs."""
        quantize = binding.quantize_fp8
        self.norm = norm
        self.gate_up, self.down = quantize(gate_up, block_rows=128), quantize(down, block_rows=128)
        if self.training:
            self.gate_up_t = quantize(gate_up, block_rows=128, transposed=True)
            self.down_t = quantize(down, block_rows=128, transposed=True)

    def __call__(self, x, residual=None):
        """(out, h) for x (M, D), any M: the block's output and the residual
        stream it is to be added to (x itself without a residual)."""
        n = binding.rms_norm(x, self.norm, residual=residual, eps=self.eps, quantize=True)
        gu = binding.gemm_fp8(n.y, n.scale, *self.gate_up, exact=self.exact)
        out = binding.gemm_fp8(*binding.swiglu(gu, quantize=True), *self.down, exact=self.exact)
        return out, (x if residual is None else n.h)

    def forward(self, x, residual=None):
        """As the call, and what ``backward`` reads: (out, h, saved)."""
        n = binding.rms_norm(x, self.norm, residual=residual, eps=self.eps, quantize=True, return_rstd=True)
        gu = binding.gemm_fp8(n.y, n.scale, *self.gate_up, exact=self.exact)
        out = binding.gemm_fp8(*binding.swiglu(gu, quantize=True), *self.down, exact=self.exact)
        h = x if residual is None else n.h
        return out, h, (h, n.rstd, gu)

    def backward(self, saved, dout, dh=None):
        """The gradients for ``dout`` of out and, where h is used further on,
        ``dh`` of h.  The weights' products contract over the tokens, so their
        operands are quantised along those, transposed on the way."""
        if not self.training:
            raise ValueError("backward needs a block made with training=True")
        import torch

        quantize, product, f32 = binding.quantize_fp8, binding.gemm_fp8, torch.float32
        h, rstd, gu = saved
        ddown = product(*quantize(dout, transposed=True), *quantize(binding.swiglu(gu), transposed=True), out_dtype=f32)
        dgu = binding.swiglu_backward(product(*quantize(dout), *self.down_t, exact=self.exact), gu)
        n = binding.rms_norm(h, self.norm, eps=self.eps).y
        dgate_up = product(*quantize(dgu, transposed=True), *quantize(n, transposed=True), out_dtype=f32)
        dx, dnorm = binding.rms_norm_backward(product(*quantize(dgu), *self.gate_up_t, exact=self.exact), h, self.norm,
                                              rstd, dresidual=dh)
        return Gradients(dx, dnorm, dgate_up, ddown)


def main():
    import torch

    D, F, M, bf16 = 512, 1280, 2048, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    weights = [torch.ones(D, device="cuda"), rand(2 * F, D) * D ** -0.5, rand(D, F) * F ** -0.5]
    x, target = rand(M, D).to(bf16), rand(M, D)
    block = FeedForward(*(w.to(bf16) for w in weights), training=True)
    for step in range(30):
        out, _, saved = block.forward(x)
        error = out.float() - target
        grads = block.backward(saved, (2.0 / M * error).to(bf16))
        for w, dw in zip(weights, grads[1:]):
            w -= 0.1 * dw
        block.set_weights(*(w.to(bf16) for w in weights))
        if step % 5 == 0 or step == 29:
            print("step %2d  mean squared error %.4f" % (step, float(error.square().mean())))
    for i in range(3):
        y, _ = block(x[i:i + 1])
        print("token %d  error against the batch's row %.4f" % (
            i, float((y.float() - block(x)[0][i:i + 1].float()).norm() / y.float().norm())))


if __name__ == "__main__":
    main()
