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


@pytest.mark.parametrize("V,other", [(40, 1.5), (300, 1.5), (40, -1.625), (300, -1.625)])
def test_gradients_of_logits_far_out(tgemm, kernel, V, other):
    """lse in FP32 is the largest logit itself, exp(z - lse) 1 or 0: sums of whole multiples of W's numbers, exact."""
    X, W, z = far_logits(V, other)
    target = z.argmax(dim=1)
    lse = torch.logsumexp(z, dim=1).float()
    p = torch.exp(z - lse.double()[:, None])
    p[torch.arange(len(X)), target] -= 1
    dloss = torch.full((len(X),), 2.0 ** -6)
    dx, dw = tgemm.gemm_ce_grad(X.cuda(), W.cuda(), target.cuda(), lse.cuda(), dloss.cuda(), dx_dtype=F32, dw_dtype=F32)
    assert torch.equal(dx.double().cpu()[:3], ((p * 2.0 ** -6) @ W.double())[:3])
    assert dw.isfinite().all()


@pytest.mark.parametrize("T,V", [(7, 100), (300, 1000)])
@pytest.mark.parametrize("scale", [6, 12, 20, 28, 31, 34, 40, 80])
def test_large_logits(tgemm, kernel, scale, T, V):
    """Whole numbers times 2^scale: exact logits, and a loss of their exact differences and the logarithm of a small number."""
    g = torch.Generator().manual_seed(scale + V)
    x, w = torch.randint(-3, 4, (T, 8), generator=g).double(), torch.randint(-3, 4, (V, 8), generator=g).double()
    target = torch.randint(0, V, (T,), generator=g)
    z = x @ w.t() * 2.0 ** scale
    target[::2] = z.argmax(dim=1)[::2]
    X, W = (x * 2.0 ** scale).to(BF16), w.to(BF16)
    top = z.max(dim=1).values
    more = torch.log(torch.exp(z - top[:, None]).sum(dim=1))
    loss = more + (top - z.gather(1, target[:, None])[:, 0])
    got, lse = tgemm.gemm_ce(X.cuda(), W.cuda(), target.cuda())
    # Exponentials and their sums to 2^-19, additions to 2^-24 of their sum.
    ref.check(got, loss, 2.0 ** -18 + 2.0 ** -23 * loss, "loss")
    ref.check(lse, top + more, 2.0 ** -18 + 2.0 ** -23 * top.abs(), "lse")
    # Under the lse that FP32 holds: a difference rounded once, an exponential, and dz's rounding to BF16.
    lse = lse.double().cpu()
    p = torch.exp(z - lse[:, None])
    ep = p * torch.expm1(2.0 ** -23 * (z - lse[:, None]).abs().clamp(max=200) + 2.0 ** -18)
    if scale == 6:
        ep = ep + p * torch.expm1(2.0 ** -22 * (z.abs() + lse.abs()[:, None]))
    p[torch.arange(T), target] -= 1
    # (FP32's and BF16's normal numbers end at 2^-126: an exponential below is 0.)
    edz = ep + 2.0 ** -8 * (p.abs() + ep) + 2.0 ** -126
    dx, dw = tgemm.gemm_ce_grad(X.cuda(), W.cuda(), target.cuda(), lse.float().cuda(), torch.ones(T, device="cuda"),
                                dx_dtype=F32, dw_dtype=F32)
    for got, a, b, e in ((dx, p, w, edz), (dw, p.t(), x * 2.0 ** scale, edz.t())):
        want, tol = ref.sums(a, b)
        ref.check(got, want, tol + e @ b.abs(), "gradient")


@pytest.mark.parametrize("V", [40, 300])
def test_gradients_under_an_alpha_far_out(tgemm, kernel, V):
    """alpha past FP32's range over log2(e), logits of ordinary size."""
    alpha = 1.5 * 2.0 ** 127
    g = torch.Generator().manual_seed(V)
    X = torch.randint(-3, 4, (33, 8), generator=g) * 2.0 ** -64
    W = torch.randint(-3, 4, (V, 8), generator=g) * 2.0 ** -64
    X, W = X.to(BF16), W.to(BF16)
    target = torch.randint(0, V, (33,), generator=g)
    loss, lse, z, ez = ref.ce(X.double(), W.double(), target, alpha)
    assert z.abs().max() < 100
    got, got_lse = tgemm.gemm_ce(X.cuda(), W.cuda(), target.cuda(), alpha)
    e_lse, e_loss = ref.ce_bounds(z, ez, lse)
    ref.check(got, loss, e_loss, "loss")
    ref.check(got_lse, lse, e_lse, "lse")
    dloss = torch.full((33,), 2.0 ** -60)
    want_x, want_w, ex, ew = ref.ce_grad(X.double(), W.double(), target, got_lse.double().cpu(), dloss.double(), alpha)
    dx, dw = tgemm.gemm_ce_grad(X.cuda(), W.cuda(), target.cuda(), got_lse, dloss.cuda(), alpha, dx_dtype=F32, dw_dtype=F32)
    ref.check(dx, want_x, ref.rounded(want_x, ex, F32), "dX")
    ref.check(dw, want_w, ref.rounded(want_w, ew, F32), "dW")


@pytest.mark.parametrize("act", ref.ACTS[2:])
def test_tails_of_activations_keep_their_digits(tgemm, kernel, act):
    """The relative error alone, down to values of 2^-100. An exponential of y (in units of its exponent) is off by
    the rounding of y: 2^-24 y a rounding, of one product (silu: y = |z|), of the square and its product (gelu: z^2 / 2),
    of the cubic's four and the factor (gelu_tanh: 2 u), each with the 2^-26 of y that log2(e) is off by; beside it
    2^-22 of the exponential, 2^-22 of the reciprocal, their sum's 2^-24, gelu's fit (1.9e-7) and the roundings of
    its polynomial, of degree 7: 2^-19 holds them."""
    z = torch.cat([torch.linspace(-60, 12, 6001), torch.linspace(-8, 8, 4001), torch.linspace(-0.1, 0.1, 401)]).to(BF16).unique()
    zd = z.double()
    want = ref.act(act, zd)[0]
    z, zd, want = (x[want.abs() >= 2.0 ** -100] for x in (z, zd, want))
    y = {"silu": zd.abs(), "gelu": zd * zd / 2, "gelu_tanh": 2 * ref.R2PI * zd.abs() * (1 + 0.044715 * zd * zd)}[act]
    roundings = {"silu": 1, "gelu": 2, "gelu_tanh": 5}[act]
    got = tgemm.gemm_act(z[:, None].cuda(), torch.ones(1, 40, dtype=BF16, device="cuda"), act, out_dtype=F32)
    off = (got.double().cpu() - want[:, None]).abs() / want.abs()[:, None]
    # (Above zero the exponential is below one and goes into 1 + it, or 1 - it: what it is off by shrinks with it.)
    bound = 2.0 ** -19 + (roundings + 0.25) * 2.0 ** -24 * y * torch.where(zd > 0, torch.exp(-y), torch.ones_like(y))
    assert (off <= bound[:, None]).all(), (zd[(off > bound[:, None]).any(dim=1)], off.max())
