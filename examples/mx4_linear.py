"""A linear layer in 4-bit floating point, trained and served.

Training: activations, weights and gradients are quantised each step, every
matrix along the axis that its product sums over, so each is needed along its
rows for one product and along its columns for another; mx4_quantize_both
makes both from one reading:

    Y  = X W^T      sums over features   X, W along rows
    dX = dY W       sums over outputs    dY along rows, W along columns
    dW = dY^T X     sums over tokens     dY and X along columns

Quantising counts as the identity in the gradients (the straight-through
estimate). Serving: the weights are quantised once; prompts run with 4-bit
activations (gemm_mx4), single tokens with BF16 ones (gemm_w4).

    python examples/mx4_linear.py [--fmt nvfp4] [--tokens 8192 --inner 4096 --outer 14336]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_matrix_multiplication_sm_gb300 as tg  # noqa: E402


class LinearMx4(torch.autograd.Function):
    """y = x w^T + b with both products' operands in 4 bits: x (tokens,
    inner) and w (outer, inner) BF16 or FP32, b (outer) FP32 or None. y and dx
    are BF16, dw is FP32 before it is cast to w's type."""

    @staticmethod
    def forward(ctx, x, w, b, fmt):
        xq, ctx.x_t = tg.mx4_quantize_both(x, fmt)
        wq, ctx.w_t = tg.mx4_quantize_both(w, fmt)
        ctx.fmt, ctx.types = fmt, (x.dtype, w.dtype)
        return tg.gemm_mx4(xq, wq, out_dtype=torch.bfloat16, bias=b)

    @staticmethod
    def backward(ctx, dy):
        q, t = tg.mx4_quantize_both(dy.contiguous(), ctx.fmt)
        dx = dw = db = None
        if ctx.needs_input_grad[0]:
            dx = tg.gemm_mx4(q, ctx.w_t, out_dtype=torch.bfloat16).to(ctx.types[0])
        if ctx.needs_input_grad[1]:
            dw = tg.gemm_mx4(t, ctx.x_t).to(ctx.types[1])
        if ctx.needs_input_grad[2]:
            db = dy.float().sum(0)
        return dx, dw, db, None


class ServedLinearMx4:
    """The same layer with weights quantised once."""

    def __init__(self, w, b=None, fmt="mxfp4"):
        self.w, self.b, self.fmt = tg.mx4_quantize(w, fmt), b, fmt

    def prompt(self, x):
        """Many tokens: 4-bit activations."""
        return tg.gemm_mx4(tg.mx4_quantize(x, self.fmt), self.w, out_dtype=torch.bfloat16, bias=self.b)

    def tokens(self, x):
        """Few tokens: BF16 activations."""
        return tg.gemm_w4(x, self.w, out_dtype=torch.bfloat16, bias=self.b)


def milliseconds(f, repeat=10):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(repeat):
        f()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / repeat


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--fmt", choices=("mxfp4", "nvfp4"), default="nvfp4")
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=1024)
    ap.add_argument("--outer", type=int, default=512)
    ap.add_argument("--steps", type=int, default=40)
    a = ap.parse_args(argv)
    torch.manual_seed(1)
    target = torch.randn(a.outer, a.inner, device="cuda") * a.inner ** -0.5
    w = torch.zeros_like(target).requires_grad_()
    b = torch.zeros(a.outer, device="cuda").requires_grad_()
    rate = 0.5 * a.tokens                                     # the loss is a mean over tokens
    first = last = None
    for _ in range(a.steps):
        x = torch.randn(a.tokens, a.inner, device="cuda").bfloat16()
        y = LinearMx4.apply(x, w, b, a.fmt)
        loss = ((y.float() - x.float() @ target.t()) ** 2).sum(1).mean()
        loss.backward()
        with torch.no_grad():
            for p in (w, b):
                p -= rate / (a.tokens + a.inner) * 0.5 * p.grad
                p.grad = None
        last = loss.item()
        first = last if first is None else first
    print(f"loss {first:.4f} -> {last:.4f} in {a.steps} steps ({a.fmt})")

    layer = ServedLinearMx4(w.detach().bfloat16(), b.detach(), a.fmt)
    x = torch.randn(a.tokens, a.inner, device="cuda").bfloat16()
    both = layer.prompt(x).float(), layer.tokens(x).float()
    exact = x.float() @ w.detach().t() + b.detach()
    for name, y in zip(("4-bit activations", "BF16 activations"), both):
        print(f"{name}: {((y - exact).norm() / exact.norm()).item():.4f} off the FP32 layer")
    dy = torch.randn(a.tokens, a.outer, device="cuda").bfloat16()

    def step():
        xq, x_t = tg.mx4_quantize_both(x, a.fmt)
        wq, w_t = tg.mx4_quantize_both(w.detach(), a.fmt)
        q, t = tg.mx4_quantize_both(dy, a.fmt)
        tg.gemm_mx4(xq, wq, out_dtype=torch.bfloat16)
        tg.gemm_mx4(q, w_t, out_dtype=torch.bfloat16)
        tg.gemm_mx4(t, x_t)

    print(f"step {milliseconds(step):.3f} ms, prompt {milliseconds(lambda: layer.prompt(x)):.3f} ms, "
          f"one token {milliseconds(lambda: layer.tokens(x[:1])):.3f} ms")
    assert tg.device_status() == 0
    return first, last


if __name__ == "__main__":
    main()
