"""A gated feed-forward layer and a head trained and served with the products that
compute what follows them in their epilogue.

    y = x + (act(x Wg^T + bg) * (x Wu^T + bu)) Wd^T + bd,   loss = cross entropy(y Wh^T, target)

The layer's forward pass is two products (gate, up and gating in one; down, bias
and residual in the other), its backward pass five; the head's logits are never
kept. Run: python examples/fused_ffn.py [--steps 50] [--tokens 2048] ...
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_matrix_multiplication_sm_gb300 as tg  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class GatedFFN(torch.autograd.Function):
    """x (T x D) through w_in (2 H x D: gate's rows, then up's), its bias, and w_out
    (D x H) with its bias, onto x. Matrices BF16, biases FP32."""

    @staticmethod
    def forward(ctx, x, w_in, b_in, w_out, b_out, act):
        h, z = tg.gemm_act(x, w_in, act, trans_b=True, gated=True, bias=b_in, keep_z=True)
        y = tg.gemm_act(h, w_out, trans_b=True, bias=b_out, residual=x)
        ctx.save_for_backward(x, w_in, w_out, h, z)
        ctx.act = act
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w_in, w_out, h, z = ctx.saved_tensors
        dy = dy.contiguous()
        dz, db_in = tg.gemm_act_grad(dy, w_out, z, ctx.act, gated=True)
        dw_out = tg.gemm_act(dy, h, trans_a=True)
        db_out = dy.float().sum(dim=0)
        dw_in = tg.gemm_act(dz, x, trans_a=True)
        dx = tg.gemm_act(dz, w_in, residual=dy)
        return dx, dw_in, db_in, dw_out, db_out, None


class HeadLoss(torch.autograd.Function):
    """Each token's cross entropy; tokens whose target is negative are left out."""

    @staticmethod
    def forward(ctx, x, w, target):
        loss, lse = tg.gemm_ce(x, w, target)
        ctx.save_for_backward(x, w, target, lse)
        return loss

    @staticmethod
    def backward(ctx, dloss):
        x, w, target, lse = ctx.saved_tensors
        dx, dw = tg.gemm_ce_grad(x, w, target, lse, dloss.float().contiguous(), x_grad=ctx.needs_input_grad[0],
                                 w_grad=ctx.needs_input_grad[1])
        return dx, dw, None


def main(argv=None):
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=50)
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--width", type=int, default=512)
    p.add_argument("--hidden", type=int, default=1024)
    p.add_argument("--vocabulary", type=int, default=8000)
    p.add_argument("--rate", type=float, default=0.5)
    args = p.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)

    def draw(*size, std):
        return (torch.randn(size, generator=g, device="cuda") * std).requires_grad_()

    T, D, H, V = args.tokens, args.width, args.hidden, args.vocabulary
    # FP32 weights, rounded to BF16 for a step's products.
    w_in, w_out, w_head = draw(2 * H, D, std=D ** -0.5), draw(D, H, std=H ** -0.5), draw(V, D, std=D ** -0.5)
    b_in, b_out = draw(2 * H, std=0.0), draw(D, std=0.0)
    weights = [w_in, w_out, w_head, b_in, b_out]
    # Tokens whose next one is a function of them; one in ten is padding.
    words = torch.randn(V, D, generator=g, device="cuda")
    token = torch.randint(0, V, (T,), generator=g, device="cuda")
    target = (token * 7 + 3) % V
    target[torch.rand(T, generator=g, device="cuda") < 0.1] = -100
    kept = (target >= 0).sum()
    x = words[token].to(BF16)
    first = last = None
    for step in range(args.steps):
        y = GatedFFN.apply(x, w_in.to(BF16), b_in, w_out.to(BF16), b_out, "silu")
        loss = HeadLoss.apply(y, w_head.to(BF16), target).sum() / kept
        loss.backward()
        with torch.no_grad():
            for w in weights:
                w -= args.rate * w.grad
                w.grad = None
        last = loss.item()
        first = last if first is None else first
        if step % 10 == 0 or step == args.steps - 1:
            print(f"step {step:3d}  loss {last:.4f}")
    # Serving: one token, its likelihood under the head.
    with torch.no_grad():
        h = tg.gemm_act(x[:1], w_in.to(BF16), "silu", trans_b=True, gated=True, bias=b_in.detach())
        y = tg.gemm_act(h, w_out.to(BF16), trans_b=True, bias=b_out.detach(), residual=x[:1])
        nll, _ = tg.gemm_ce(y, w_head.to(BF16), (token[:1] * 7 + 3) % V)
    print(f"one token: -log p = {nll.item():.4f}")
    assert tg.device_status() == 0
    return first, last


if __name__ == "__main__":
    main()
