"""64-bit forms of the products with what follows them in their epilogue, and
bounds on the kernels' errors.

Sums: products of BF16 numbers are exact; a step of 16 columns of K is added to
an FP32 sum with low bits cut off, at most 2^-22 of the sum of magnitudes a
step with the step's own sum's; so |z' - z| <= (K / 16 + 4) 2^-22 |A||B| (the 4
for adding the bias, parts, and a factor).

Activations are made of exponentials and quotients with relative errors of
some 2^-21, where arguments up to 16 are rounded to 2^-24 of themselves before
an exponential or erfc takes them (erfc(x) changes by 2 x^2 of itself a relative
change of x: x up to 4): 2^-17 of the value holds them all.
"""
import math

import torch

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
R2PI = math.sqrt(2 / math.pi)


def act(name, z):
    """(act(z), act'(z)) in 64 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "gelu":
        phi = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        u, du = R2PI * (z + 0.044715 * z ** 3), R2PI * (1 + 3 * 0.044715 * z * z)
        # (1 + tanh u) / 2 as sigmoid(2 u), and (1 - tanh^2 u) / 2 as 2 s (1 - s): 1 + tanh u has lost all
        # of its 53 bits at u = -18 (z = -8).
        s = torch.sigmoid(2 * u)
        return z * s, s + 2 * z * s * torch.sigmoid(-2 * u) * du
    s = torch.sigmoid(z)
    return z * s, s + z * s * torch.sigmoid(-z)


def sums(a, b, bias=None):
    """(z, bound on its error) of a b + bias, both in 64 bits."""
    z, size = a @ b, a.abs() @ b.abs()
    if bias is not None:
        z, size = z + bias, size + bias.abs()
    return z, (a.shape[1] / 16 + 4) * 2.0 ** -22 * size


def rounded(value, tol, dtype):
    """The bound with the result's own rounding: half a step."""
    return tol + torch.finfo(dtype).eps / 2 * (value.abs() + tol)


def act_bound(name, z, ez):
    """act(z) and the bound on its error (slopes are at most 1.13)."""
    v, _ = act(name, z)
    return v, 1.13 * ez + 2.0 ** -17 * v.abs()


def grad_bound(name, z):
    """act'(z) and the bound on its error, z exact: its terms are s and z s (1 - s)
    times at most 1 + z^2."""
    _, d = act(name, z)
    return d, 2.0 ** -17 * (1 + z.abs()) * (1 + (0.14 * z * z if name == "gelu_tanh" else 0)) if name not in ("none", "relu") \
        else torch.zeros_like(z)


def check(got, want, tol, what=""):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0].tolist()}: " \
                          f"{got[bad][0].item()} for {want[bad][0].item()}, bound {tol.expand_as(want)[bad][0].item()}"


def ce(x, w, target, alpha):
    """(loss, lse, z, bound on z's error) in 64 bits."""
    z, ez = sums(x, w.t())
    z, ez = alpha * z, abs(alpha) * ez + 2.0 ** -23 * (alpha * z).abs()
    lse = torch.logsumexp(z, dim=1)
    kept = (target >= 0) & (target < w.shape[0])
    at = torch.where(kept, target, torch.zeros_like(target))
    picked = z.gather(1, at[:, None])[:, 0] if w.shape[0] else torch.zeros_like(lse)
    return torch.where(kept, lse - picked, torch.zeros_like(lse)), lse, z, ez


def ce_bounds(z, ez, lse):
    """Bounds on lse's and a loss's error: the largest of z's errors, exponentials
    to 2^-20, their sums and joins to 2^-19, the last additions to 2^-22."""
    e = ez.max(dim=1).values + 2.0 ** -18 + 2.0 ** -22 * (lse.abs() + z.abs().max(dim=1).values)
    return e, 2 * e


def ce_grad(x, w, target, lse, dloss, alpha):
    """(dX, dW, their bounds) in 64 bits: dz is rounded to BF16 (2^-8 of itself)
    after errors of z, of z - lse (2^-22 of both) and of an exponential."""
    z, ez = sums(x, w.t())
    z, ez = alpha * z, abs(alpha) * ez
    kept = (target >= 0) & (target < w.shape[0])
    p = torch.exp(z - lse[:, None])
    ep = p * (torch.expm1(ez + 2.0 ** -18 + 2.0 ** -22 * (z.abs() + lse.abs()[:, None])))
    p[kept.nonzero()[:, 0], target[kept]] -= 1
    g = torch.where(kept, alpha * dloss, torch.zeros_like(dloss))[:, None]
    dz = torch.where(kept[:, None], g * p, torch.zeros_like(p))
    edz = torch.where(kept[:, None], g.abs() * ep, torch.zeros_like(p))
    edz = edz + 2.0 ** -8 * (dz.abs() + edz)
    xk = torch.where(kept[:, None], x, torch.zeros_like(x))
    dx, ex = sums(dz, w)
    dw, ew = sums(dz.t(), xk)
    return dx, dw, ex + edz @ w.abs(), ew + edz.t() @ xk.abs()
