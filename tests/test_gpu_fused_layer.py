"""examples/fused_ffn.py: the operators together, as a training step uses them,
against the formulas in 64 bits."""
import os
import sys

import pytest
import torch

import fused_reference as ref
from test_gpu_fused_act import BF16, generator

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import fused_ffn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D,H,V", [(40, 64, 96, 300), (129, 100, 130, 515), (1, 16, 24, 40), (700, 264, 520, 1000)])
def test_a_step_is_that_of_the_formulas(tgemm, T, D, H, V):
    """Every gradient against 64 bits. Between the products matrices are BF16 (h, z,
    y, dz, dy), so a gradient is off by a few roundings of 2^-8 in a row: y, dy, dz and
    itself, and h's or z's in the products that take them -- six of them, of the
    magnitudes |a| |b| of its products in turn."""
    g = generator(T, D, H, V)
    x = torch.randn(T, D, generator=g).to(BF16)
    w_in = (torch.randn(2 * H, D, generator=g) * D ** -0.5).to(BF16)
    w_out = (torch.randn(D, H, generator=g) * H ** -0.5).to(BF16)
    w_head = (torch.randn(V, D, generator=g) * D ** -0.5).to(BF16)
    b_in, b_out = torch.randn(2 * H, generator=g), torch.randn(D, generator=g)
    target = torch.randint(0, V, (T,), generator=g)
    target[::7] = -100
    target[0] = 1
    weight = torch.rand(T, generator=g)
    leaves = [t.cuda().requires_grad_() for t in (x, w_in, b_in, w_out, b_out, w_head)]
    X, Wi, bi, Wo, bo, Wh = leaves
    y = fused_ffn.GatedFFN.apply(X, Wi, bi, Wo, bo, "silu")
    loss = fused_ffn.HeadLoss.apply(y, Wh, target.cuda())
    (loss * weight.cuda()).sum().backward()

    d = [t.double().requires_grad_() for t in (x, w_in, b_in, w_out, b_out, w_head)]
    xd, wi, bi_, wo, bo_, wh = d
    z = xd @ wi.t() + bi_
    h = torch.nn.functional.silu(z[:, :H]) * z[:, H:]
    yd = xd + h @ wo.t() + bo_
    want = torch.nn.functional.cross_entropy(yd @ wh.t(), target, ignore_index=-100, reduction="none")
    (want * weight.double()).sum().backward()
    with torch.no_grad():
        # Magnitudes: |h| |wo| + |x| + |bo| of y; p + [target] of dlogits; and so back.
        hm = h.abs()
        ym = xd.abs() + hm @ wo.abs().t() + bo_.abs()
        ey = 3 * 2.0 ** -8 * ym
        ref.check(y, yd, ey, "y")
        ez = ey @ wh.abs().t()                                     # of the logits
        kept = target >= 0
        tol = ez.max(dim=1).values * 2 + 2.0 ** -16
        ref.check(loss, want, torch.where(kept, tol, torch.zeros_like(tol)), "loss")
        p = torch.softmax(yd @ wh.t(), dim=1)
        # A logit off by e changes p by p (e + the row's mean e) at most e^(2 e) times over.
        spread = 2 * ez.max(dim=1, keepdim=True).values
        onehot = torch.zeros_like(p)
        onehot[kept.nonzero()[:, 0], target[kept]] = 1
        w_ = torch.where(kept, weight.double(), torch.zeros_like(weight.double()))[:, None]
        dl, edl = w_ * (p - onehot), w_ * (p * torch.expm1(spread + 2.0 ** -16))
        edl = edl + 2.0 ** -8 * (dl.abs() + edl)
        dy, edy = dl @ wh, edl @ wh.abs() + 2.0 ** -8 * (dl.abs() @ wh.abs())
        ref.check(Wh.grad, wh.grad, (edl.t() @ ym + dl.abs().t() @ ey) + 2 * 2.0 ** -8 * (dl.abs().t() @ ym), "head")
        dh, edh = dy.abs() @ wo.abs(), edy @ wo.abs()
        # silu and its slope are at most |z| and 1.1, and move by 1.1 and 0.5 of z's change.
        ezz = 2.0 ** -8 * z.abs()
        gate, up = z[:, :H].abs(), z[:, H:].abs()
        slope, value = 1.1, gate
        dzm = torch.cat((dh * up * slope, dh * value), 1)
        edz = torch.cat((edh * up * slope + dh * (ezz[:, H:] * slope + up * 0.5 * ezz[:, :H]),
                         edh * value + dh * 1.1 * ezz[:, :H]), 1) + 2.0 ** -7 * dzm
        hh = gate * up
        eh = 2.0 ** -8 * hh
        ref.check(Wo.grad, wo.grad, edy.t() @ hh + dy.abs().t() @ eh + 2.0 ** -7 * (dy.abs().t() @ hh), "w_out")
        ref.check(bo.grad, bo_.grad, edy.sum(0) + 2.0 ** -8 * dy.abs().sum(0), "b_out")
        ref.check(Wi.grad, wi.grad, edz.t() @ xd.abs() + 2.0 ** -7 * (dzm.t() @ xd.abs()), "w_in")
        ref.check(bi.grad, bi_.grad, edz.sum(0), "b_in")
        ref.check(X.grad, xd.grad, edz @ wi.abs() + edy + 2.0 ** -7 * (dzm @ wi.abs() + dy.abs()), "x")


def test_a_step_in_a_graph_is_the_step(tgemm):
    """Forward, backward and the head captured together and replayed."""
    T, D, H, V = 129, 104, 130, 515
    g = generator("graph")
    x, w_in, w_out, w_head = ((torch.randn(s, generator=g) * 0.1).to(BF16).cuda() for s in ((T, D), (2 * H, D), (D, H), (V, D)))
    b_in, b_out = torch.randn(2 * H, generator=g).cuda(), torch.randn(D, generator=g).cuda()
    target = torch.randint(-1, V, (T,), generator=g).cuda()
    dloss = torch.rand(T, generator=g).cuda()

    def step():
        h, z = tgemm.gemm_act(x, w_in, "gelu", trans_b=True, gated=True, bias=b_in, keep_z=True)
        y = tgemm.gemm_act(h, w_out, trans_b=True, bias=b_out, residual=x)
        loss, lse = tgemm.gemm_ce(y, w_head, target)
        dy, dw_head = tgemm.gemm_ce_grad(y, w_head, target, lse, dloss)
        dz, db_in = tgemm.gemm_act_grad(dy, w_out, z, "gelu", gated=True)
        return (y, loss, lse, dy, dw_head, dz, db_in, tgemm.gemm_act(dy, h, trans_a=True), tgemm.gemm_act(dz, x, trans_a=True),
                tgemm.gemm_act(dz, w_in, residual=dy))

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert tgemm.device_status() == 0


def test_the_example_trains_and_serves(tgemm, capsys):
    first, last = fused_ffn.main(["--steps", "12", "--tokens", "300", "--width", "96", "--hidden", "128", "--vocabulary", "500"])
    assert first > 0 and last > 0
    assert "one token" in capsys.readouterr().out
