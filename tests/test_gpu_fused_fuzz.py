"""Random calls of the fused products on whole numbers, exactly, whatever kernel and
tiles they get; random heads within their bounds."""
import random

import pytest
import torch

import fused_reference as ref
from test_gpu_fused_act import BF16, F32, place, room, untouched

pytestmark = pytest.mark.gpu


def size(r, lo, hi):
    return int(round(lo * (hi / lo) ** r.random()))


@pytest.mark.parametrize("seed", range(120))
def test_products(tgemm, seed):
    r = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    M, N, K = size(r, 1, 3000), size(r, 1, 4000), size(r, 1, 3000)
    way, grad, gated = r.choice(["packed", "padded", "odd"]), r.random() < 0.4, r.random() < 0.4
    ta, tb = r.random() < 0.3, r.random() < 0.5
    wide = 2 * N if gated else N
    cols = N if grad else wide
    # Small enough for sums that FP32 holds exactly, and for the reference's own.
    a, b = (torch.randint(-1, 2, s, generator=g).float() for s in ((M, K), (K, cols)))
    A, B = place(a.t().contiguous() if ta else a, BF16, way), place(b.t().contiguous() if tb else b, BF16, way)
    d = (a.cuda() @ b.cuda()).double().cpu()
    if grad:
        z = torch.randint(-2, 3, (M, wide), generator=g).double()
        want = torch.cat((d * z[:, N:] * (z[:, :N] > 0), d * z[:, :N].clamp(min=0)), 1) if gated else d * (z > 0)
        dtype = BF16 if gated else r.choice([BF16, F32])
        out, around = room(M, wide, dtype, way)
        with_db = r.random() < 0.7
        got = tgemm.gemm_act_grad(A, B, place(z, BF16, way), "relu", trans_a=ta, trans_b=tb, gated=gated, bias_grad=with_db, out=out)
        if with_db:
            # Sums of whole numbers below 2^24 in all.
            assert want.abs().sum(0).max() < 2 ** 24 and torch.equal(got[1].double().cpu(), want.sum(0))
    else:
        bias = torch.randint(-3, 4, (wide,), generator=g).double() if r.random() < 0.5 else None
        z = d if bias is None else d + bias
        want = z[:, :N].clamp(min=0) * z[:, N:] if gated else z.clamp(min=0)
        dtype = BF16 if gated else r.choice([BF16, F32])
        R = None
        if r.random() < 0.5:
            res = torch.randint(-3, 4, (M, N), generator=g).double()
            R, want = place(res, r.choice([BF16, F32]), way), want + res
        out, around = room(M, N, dtype, way)
        keep = r.random() < 0.4
        got = tgemm.gemm_act(A, B, "relu", trans_a=ta, trans_b=tb, gated=gated, bias=None if bias is None else bias.float().cuda(),
                             residual=R, keep_z=keep, out=out)
        if keep:
            assert torch.equal(got[1].cpu(), z.bfloat16())
    assert torch.equal(out.cpu(), want.to(dtype))
    assert untouched(out, around)
    assert tgemm.device_status() == 0


@pytest.mark.parametrize("seed", range(40))
def test_heads(tgemm, seed):
    r = random.Random(1000 + seed)
    g = torch.Generator().manual_seed(seed)
    T, V, D = size(r, 1, 1200), size(r, 2, 6000), size(r, 8, 2500)
    way = r.choice(["packed", "padded", "odd"])
    alpha = r.choice([1.0, 1.0, 0.3, -1.5])
    w = (torch.randn(V, D, generator=g) / D ** 0.5).to(BF16)
    target = torch.randint(-1, V, (T,), generator=g)
    x = (torch.randn(T, D, generator=g) + 4 * w[target.clamp(min=0)].float()).to(BF16)
    X, W, t = place(x, BF16, way), place(w, BF16, way), target.cuda()
    loss, lse = tgemm.gemm_ce(X, W, t, alpha=alpha)
    want, want_lse, z, ez = ref.ce(x.double(), w.double(), target, alpha)
    e_lse, e_loss = ref.ce_bounds(z, ez, want_lse)
    ref.check(lse, want_lse, e_lse, "lse")
    ref.check(loss, want, e_loss, "loss")
    dloss = torch.rand(T, generator=g)
    out, around = room(V, D, r.choice([BF16, F32]), way)
    dx, _ = tgemm.gemm_ce_grad(X, W, t, lse, dloss.cuda(), alpha=alpha, dx_dtype=r.choice([BF16, F32]), dw_out=out)
    want_x, want_w, ex, ew = ref.ce_grad(x.double(), w.double(), target, lse.double().cpu(), dloss.double(), alpha)
    ref.check(dx, want_x, ref.rounded(want_x, ex, dx.dtype), "dX")
    ref.check(out, want_w, ref.rounded(want_w, ew, out.dtype), "dW")
    assert untouched(out, around)
    assert tgemm.device_status() == 0
