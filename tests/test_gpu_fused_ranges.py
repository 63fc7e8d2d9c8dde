"""The fused products at the ends of the numbers' range: what is finite by the formulas is finite."""
import pytest
import torch

import fused_reference as ref
from test_gpu_fused_act import BF16, F32, kernel  # noqa: F401

pytestmark = pytest.mark.gpu

FAR = [5.0, 40.0, 1e10, 1e19, 3e19, 5e19, 1e20, 1e30, 3e38]


@pytest.mark.parametrize("act", ref.ACTS)
def test_activations_and_slopes_far_out(tgemm, kernel, act):
    """z to both ends of BF16, times one: from 40 on act(z) is z or 0 to all bits, its slope 1 or 0."""
    z = torch.tensor(FAR + [-x for x in FAR])[:, None].to(BF16)
    one = torch.ones(1, 72, dtype=BF16)
    rows = torch.ones(len(z), 1, dtype=BF16, device="cuda")
    v, s = (x.expand(-1, 72) for x in ref.act(act, z.double()))
    ev, es = (2.0 ** -17 * (x.abs() + (z.abs() < 40)) for x in (v, s))
    for dtype in (BF16, F32):
        ref.check(tgemm.gemm_act(z.cuda(), one.cuda(), act, out_dtype=dtype), v, ref.rounded(v, ev, dtype), "value")
        got, db = tgemm.gemm_act_grad(rows, one.cuda(), z.expand(-1, 72).contiguous().cuda(), act, out_dtype=dtype)
        ref.check(got, s, ref.rounded(s, es, dtype), "slope")
        ref.check(db, s.sum(dim=0), es.sum(dim=0) + 2.0 ** -20 * s.abs().sum(dim=0), "db")
    both = torch.cat((z.expand(-1, 72), one.expand(len(z), -1)), dim=1).contiguous()
    got = tgemm.gemm_act_grad(rows, one.cuda(), both.cuda(), act, gated=True, bias_grad=False)
    want, e = torch.cat((s, v), dim=1), torch.cat((es, ev), dim=1)
    ref.check(got, want, ref.rounded(want, e, BF16), "gated")


def far_logits(V, other):
    """(X, W, z): rows all of whose logits, or whose largest and least, are near the ends of FP32's range; z in 64 bits."""
    x = torch.tensor([1.0, -1.0, 0.5, 2.0 ** -130, 0.0])[:, None] * 2.0 ** 64
    w = torch.full((V, 1), other * 2.0 ** 63)
    w[3] = w[V - 2] = 1.75 * 2.0 ** 63
    z = x.double() @ w.double().t()
    assert z.isfinite().all() and z[0].max() > 2.4e38 and z[1].max().abs() > 2.4e38
    return x.to(BF16), w.to(BF16), z


@pytest.mark.parametrize("V,other", [(40, 1.5), (300, 1.5), (40, -1.625), (300, -1.625)])
def test_losses_of_logits_far_out(tgemm, kernel, V, other):
    X, W, z = far_logits(V, other)
    # Each row's largest logit (one of two or more), and its least.
    target = torch.cat((z.argmax(dim=1), z.argmin(dim=1)))
    X, z = torch.cat((X, X)), torch.cat((z, z))
    top = z.max(dim=1).values
    more = torch.log(torch.exp(z - top[:, None]).sum(dim=1))
    # (From the maximum: lse itself has no bits left for log 2.) Losses past FP32's range are infinities.
    loss = (more + (top - z.gather(1, target[:, None])[:, 0])).float().double()
    got, lse = tgemm.gemm_ce(X.cuda(), W.cuda(), target.cuda())
    got, finite = got.double().cpu(), loss.isfinite()
    assert torch.equal(got[~finite], loss[~finite])
    ref.check(got[finite], loss[finite], 2.0 ** -18 + 2.0 ** -20 * loss[finite].abs(), "loss")
    ref.check(lse, top + more, 2.0 ** -18 + 2.0 ** -20 * top.abs(), "lse")
