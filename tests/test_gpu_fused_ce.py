"""gemm_ce and gemm_ce_grad against 64-bit forms."""
import pytest
import torch

import fused_reference as ref
from test_gpu_fused_act import BF16, F32, generator, kernel, place, room, untouched  # noqa: F401

pytestmark = pytest.mark.gpu


def inputs(g, T, V, D, left_out=0.2, scale=1.0):
    w = (torch.randn(V, D, generator=g) / D ** 0.5).to(BF16)
    target = torch.randint(0, V, (T,), generator=g)
    x = (torch.randn(T, D, generator=g) * scale + 4 * w[target].float()).to(BF16)
    out = torch.rand(T, generator=g) < left_out
    marks = torch.tensor([-100, -1, V, V + 5, 2 ** 62, -2 ** 62])
    target = torch.where(out, marks[torch.randint(0, 6, (T,), generator=g)], target)
    return x, w, target


SIZES = [(1, 1, 1), (1, 300, 64), (5, 7, 9), (16, 1000, 72), (31, 33, 65), (130, 257, 40), (256, 256, 64), (300, 1037, 136),
         (600, 5000, 200), (64, 128, 1100), (270, 515, 2061), (1300, 4999, 72)]


@pytest.mark.parametrize("way", ["packed", "odd"])
@pytest.mark.parametrize("alpha", [1.0, -0.4])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_losses(tgemm, kernel, T, V, D, alpha, way):
    g = generator(T, V, D, alpha, way)
    x, w, target = inputs(g, T, V, D)
    loss, lse = tgemm.gemm_ce(place(x, BF16, way), place(w, BF16, way), target.cuda(), alpha=alpha)
    want, want_lse, z, ez = ref.ce(x.double(), w.double(), target, alpha)
    e_lse, e_loss = ref.ce_bounds(z, ez, want_lse)
    assert loss.dtype == F32 and lse.dtype == F32
    ref.check(lse, want_lse, e_lse, "lse")
    ref.check(loss, want, e_loss, "loss")
    assert (loss.cpu()[(target < 0) | (target >= V)] == 0).all()
    assert tgemm.device_status() == 0


@pytest.mark.parametrize("way", ["packed", "odd"])
@pytest.mark.parametrize("dx,dw", [(BF16, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_gradients(tgemm, kernel, T, V, D, dx, dw, way):
    alpha = 0.8
    g = generator(T, V, D, str(dx), str(dw), way)
    x, w, target = inputs(g, T, V, D)
    X, W, t = place(x, BF16, way), place(w, BF16, way), target.cuda()
    _, lse, _, _ = ref.ce(x.double(), w.double(), target, alpha)
    lse, dloss = lse.float(), torch.rand(T, generator=g) / T
    out, around = room(V, D, dw, way)
    got_x, got_w = tgemm.gemm_ce_grad(X, W, t, lse.cuda(), dloss.cuda(), alpha=alpha, dx_dtype=dx, dw_out=out)
    want_x, want_w, ex, ew = ref.ce_grad(x.double(), w.double(), target, lse.double(), dloss.double(), alpha)
    ref.check(got_x, want_x, ref.rounded(want_x, ex, dx), "dX")
    ref.check(got_w, want_w, ref.rounded(want_w, ew, dw), "dW")
    assert untouched(out, around)
    only_x, none = tgemm.gemm_ce_grad(X, W, t, lse.cuda(), dloss.cuda(), alpha=alpha, w_grad=False, dx_dtype=dx)
    assert none is None and torch.equal(only_x, got_x)
    none, only_w = tgemm.gemm_ce_grad(X, W, t, lse.cuda(), dloss.cuda(), alpha=alpha, x_grad=False, dw_dtype=dw)
    assert none is None and torch.equal(only_w, got_w)
    assert tgemm.device_status() == 0


def test_gradients_over_several_pieces_of_the_vocabulary(tgemm):
    """40000 tokens: pieces of 3328 columns, the last one short and odd."""
    T, V, D = 40000, 7003, 72
    g = generator(T)
    x, w, target = inputs(g, T, V, D)
    rows = torch.randint(0, T, (200,), generator=g)
    X, W, t = x.cuda(), w.cuda(), target.cuda()
    loss, lse = tgemm.gemm_ce(X, W, t)
    want, want_lse, z, ez = ref.ce(x[rows].double(), w.double(), target[rows], 1.0)
    e_lse, e_loss = ref.ce_bounds(z, ez, want_lse)
    ref.check(lse[rows.cuda()], want_lse, e_lse, "lse")
    ref.check(loss[rows.cuda()], want, e_loss, "loss")
    dloss = torch.full((T,), 1.0 / T)
    for dtype in (BF16, F32):
        dx, dw = tgemm.gemm_ce_grad(X, W, t, lse, dloss.cuda(), dx_dtype=dtype, dw_dtype=F32)
        want_x, _, ex, _ = ref.ce_grad(x[rows].double(), w.double(), target[rows], lse.double().cpu()[rows], dloss[rows].double(), 1.0)
        ref.check(dx[rows.cuda()], want_x, ref.rounded(want_x, ex, dtype), "dX")
    # dW of some columns, over all rows.
    cols = torch.tensor([0, 1, 3327, 3328, 6655, 6656, 7001, 7002])
    zc = x.double() @ w[cols].double().t()
    p = torch.exp(zc - lse.double().cpu()[:, None]) - (target[:, None] == cols).double()
    kept = (target >= 0) & (target < V)
    dz = torch.where(kept[:, None], p / T, torch.zeros_like(p))
    err = 2.0 ** -8 * dz.abs() + torch.where(kept[:, None], (p.abs() + 1) / T, torch.zeros_like(p)) * 2.0 ** -16
    want_w, ew = ref.sums(dz.t(), x.double())
    ref.check(dw[cols.cuda()], want_w, ew + err.t() @ x.double().abs(), "dW")


def test_losses_over_several_turns_of_tokens(tgemm):
    """Maxima and sums of 131072 x 70000 / 128 columns pass 256 MB: two turns."""
    T, V, D = 131072, 70000, 16
    g = generator(3)
    w = (torch.randn(V, D, generator=g) / 4).to(BF16)
    x = torch.randn(T, D, generator=g).to(BF16)
    target = torch.randint(0, V, (T,), generator=g)
    loss, lse = tgemm.gemm_ce(x.cuda(), w.cuda(), target.cuda())
    rows = torch.cat([torch.arange(40), torch.arange(61100, 61900, 7), torch.arange(T - 40, T)])
    want, want_lse, z, ez = ref.ce(x[rows].double(), w.double(), target[rows], 1.0)
    e_lse, e_loss = ref.ce_bounds(z, ez, want_lse)
    ref.check(lse[rows.cuda()], want_lse, e_lse, "lse")
    ref.check(loss[rows.cuda()], want, e_loss, "loss")


def test_dw_is_added_to_what_is_there(tgemm, kernel):
    T, V, D = 140, 300, 72
    g = generator(11)
    x, w, target = inputs(g, T, V, D)
    X, W, t = x.cuda(), w.cuda(), target.cuda()
    _, lse = tgemm.gemm_ce(X, W, t)
    dloss = torch.rand(T, generator=g).cuda()
    for dtype in (F32, BF16):
        _, dw = tgemm.gemm_ce_grad(X, W, t, lse, dloss, dw_dtype=F32)
        old = torch.randn(V, D, generator=g).to(dtype)
        out = old.cuda()
        tgemm.gemm_ce_grad(X, W, t, lse, dloss, dw_out=out, beta=0.5, x_grad=False)
        want = dw.double().cpu() + 0.5 * old.double()
        ref.check(out, want, ref.rounded(want, 2.0 ** -22 * (dw.double().cpu().abs() + old.double().abs()), dtype), str(dtype))
        out = torch.full((V, D), float("nan"), dtype=dtype, device="cuda")
        tgemm.gemm_ce_grad(X, W, t, lse, dloss, dw_out=out)
        assert torch.equal(out, dw.to(dtype))


@pytest.mark.parametrize("D", [100, 104, 1000])
def test_rows_left_out_add_nothing_whatever_they_hold(tgemm, kernel, D):
    T, V = 290, 520
    g = generator(12)
    x, w, target = inputs(g, T, V, D, left_out=0.3)
    out = (target < 0) | (target >= V)
    X, W, t = x.cuda(), w.cuda(), target.cuda()
    loss, lse = tgemm.gemm_ce(X, W, t)
    dloss = torch.rand(T, generator=g)
    want = tgemm.gemm_ce_grad(X, W, t, lse, dloss.cuda())
    for value in (float("nan"), float("inf"), -3e38):
        bad = x.clone()
        bad[out] = value
        l2, lse2 = tgemm.gemm_ce(bad.cuda(), W, t)
        assert torch.equal(l2, loss)
        lse2 = torch.where(out.cuda(), torch.full_like(lse2, value), lse2)
        d2 = torch.where(out, torch.full_like(dloss, value), dloss)
        got = tgemm.gemm_ce_grad(bad.cuda(), W, t, lse2, d2.cuda())
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    nothing = torch.full((T,), -100, device="cuda")
    l3, _ = tgemm.gemm_ce(X, W, nothing)
    dx, dw = tgemm.gemm_ce_grad(X, W, nothing, lse, dloss.cuda())
    assert not l3.any() and not dx.any() and not dw.any()


def test_a_vocabulary_past_32_bits(tgemm):
    """W and dW of more than 2^31 elements; targets and checked rows at both ends."""
    T, V, D = 6, 1100000, 2048
    g = torch.Generator(device="cuda").manual_seed(21)
    W = torch.empty(V, D, dtype=BF16, device="cuda")
    for part in W.split(100000):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * D ** -0.5)
    target = torch.tensor([0, 1048575, 1048577, V - 1, 7, -1])
    X = (torch.randn(T, D, generator=g, device="cuda") + 12 * W[target.clamp(min=0).cuda()].float()).to(BF16)
    z = torch.cat([(X.double() @ part.double().t()) for part in W.split(100000)], dim=1)
    size = torch.cat([(X.double().abs() @ part.double().abs().t()).max(dim=1, keepdim=True).values for part in W.split(100000)], 1)
    want_lse = torch.logsumexp(z, dim=1)
    loss, lse = tgemm.gemm_ce(X, W, target.cuda())
    tol = (D / 16 + 4) * 2.0 ** -22 * size.max(dim=1).values + 2.0 ** -18 + 2.0 ** -21 * want_lse.abs()
    want = torch.where(target.cuda() >= 0, want_lse - z.gather(1, target.clamp(min=0).cuda()[:, None])[:, 0], want_lse * 0)
    assert ((lse.double() - want_lse).abs() <= tol).all() and ((loss.double() - want).abs() <= 2 * tol).all()
    dloss = torch.rand(T, generator=g, device="cuda")
    dx, dw = tgemm.gemm_ce_grad(X, W, target.cuda(), lse, dloss)
    rows = torch.tensor([0, 7, 1048574, 1048575, 1048576, 1048577, V - 2, V - 1])
    p = torch.exp(z.cpu() - lse.double().cpu()[:, None])
    p[target >= 0, target[target >= 0]] -= 1
    dz = torch.where((target >= 0)[:, None], p * dloss.double().cpu()[:, None], torch.zeros_like(p))
    x = X.double().cpu()
    err = 2.0 ** -8 * dz.abs() + torch.where((target >= 0)[:, None], (p.abs() + 1e-30) * tol.cpu()[:, None] * 2, torch.zeros_like(p))
    want_w = dz[:, rows].t() @ x
    ref.check(dw[rows.cuda()], want_w, ref.rounded(want_w, (err[:, rows].t() + 2.0 ** -18 * dz[:, rows].abs().t()) @ x.abs() + 1e-12, BF16), "dW")
    want_x = sum(dz[:, i:i + 100000].cuda() @ W[i:i + 100000].double() for i in range(0, V, 100000)).cpu()
    mag = sum((err + 2.0 ** -14 * dz.abs())[:, i:i + 100000].cuda() @ W[i:i + 100000].double().abs() for i in range(0, V, 100000)).cpu()
    ref.check(dx, want_x, ref.rounded(want_x, mag, BF16), "dX")
    assert tgemm.device_status() == 0


def test_a_sure_loss_keeps_its_digits(tgemm, kernel):
    """A target 20 above two others: loss = log1p(2 exp(-20)), exactly representable sums."""
    D = 64
    w = torch.zeros(3, D)
    w[0, 0], w[1, 0], w[2, 0] = 20.0, 0.0, 0.0
    x = torch.zeros(2, D)
    x[:, 0] = 1.0
    loss, lse = tgemm.gemm_ce(x.to(BF16).cuda(), w.to(BF16).cuda(), torch.tensor([0, 1]).cuda())
    small = 2 * torch.exp(torch.tensor(-20.0, dtype=torch.float64))
    # 1 + 2 e^-20 is rounded to FP32: half a step of 1, 2^-24.
    assert abs(loss[0].double().cpu() - small) <= 2.0 ** -24 and loss[0] >= 0
    assert abs(loss[1].double().cpu() - (20 + small)) <= 20 * 2.0 ** -23


def test_infinite_logits(tgemm, kernel):
    """Logits of minus infinity count nothing; plus infinity makes NaN, in its row alone."""
    D, V, T = 64, 300, 5
    x = torch.zeros(T, D)
    x[:, 0], x[3, 1] = 1.0, 1.0
    w = torch.zeros(V, D)
    w[:200, 0] = float("-inf")
    w[10:200, 1] = 0.0
    w[299, 0] = 3.0
    X, W = x.to(BF16), w.to(BF16)
    # (0 times an infinity is NaN: columns of W that hold one are met by ones only.)
    X[:, 0] = 1.0
    loss, lse = tgemm.gemm_ce(X.cuda(), W.cuda(), torch.tensor([299, 250, -1, 299, 299]).cuda())
    want = torch.logsumexp(torch.cat([torch.zeros(99), torch.tensor([3.0])]).double(), 0)
    assert (lse.double().cpu() - want).abs().max() <= 2.0 ** -18
    assert torch.allclose(loss.double().cpu(), torch.stack([want - 3, want, want * 0, want - 3, want - 3]), atol=2.0 ** -18, rtol=0)
    W[5, 0] = float("inf")
    loss, lse = tgemm.gemm_ce(X.cuda(), W.cuda(), torch.tensor([299, 250, -1, 299, 299]).cuda())
    assert lse.isnan().all() and loss.cpu().isnan().tolist() == [True, True, False, True, True]


@pytest.mark.parametrize("T,V,D", [(0, 10, 8), (4, 0, 8), (4, 10, 0), (0, 0, 8)])
def test_sizes_of_zero(tgemm, kernel, T, V, D):
    X, W = torch.ones(T, D, dtype=BF16, device="cuda"), torch.ones(V, D, dtype=BF16, device="cuda")
    t = torch.zeros(T, dtype=torch.int64, device="cuda")
    loss, lse = tgemm.gemm_ce(X, W, t)
    if V == 0:
        assert (lse == float("-inf")).all() and not loss.any()
    elif T > 0:
        want = torch.log(torch.tensor(float(V)))
        assert torch.allclose(lse.cpu(), want.expand(T)) and torch.allclose(loss.cpu(), want.expand(T))
    dx, dw = tgemm.gemm_ce_grad(X, W, t, lse, torch.ones(T, device="cuda"))
    assert dx.shape == (T, D) and dw.shape == (V, D)
    assert not dx.any() and not dw.any()
    old = torch.full((V, D), 3.0, device="cuda")
    if T == 0 and V > 0:
        tgemm.gemm_ce_grad(X, W, t, lse, torch.ones(T, device="cuda"), dw_out=old, beta=2.0)
        assert (old == 6).all()


def test_gradients_are_differences_of_the_loss(tgemm):
    """sum(dloss loss) moved along entries of X and W."""
    T, V, D = 40, 130, 64
    g = generator(13)
    x, w, target = inputs(g, T, V, D)
    dloss = torch.rand(T, generator=g)
    X, W, t = x.cuda(), w.cuda(), target.cuda()
    loss, lse = tgemm.gemm_ce(X, W, t)
    dx, dw = tgemm.gemm_ce_grad(X, W, t, lse, dloss.cuda(), dx_dtype=F32, dw_dtype=F32)

    def total(a, b):
        return (tgemm.gemm_ce(a.cuda(), b.cuda(), t)[0].double().cpu() * dloss.double()).sum()

    kept = ((target >= 0) & (target < V)).nonzero()[:, 0]
    size = (dloss.double() * loss.double().cpu()).abs().sum()
    for which, m, grad, spots in (("x", x, dx, [(int(kept[0]), 3), (int(kept[5]), 60)]), ("w", w, dw, [(0, 0), (77, 30), (129, 63)])):
        for i, j in spots:
            up, down = m.clone(), m.clone()
            up[i, j], down[i, j] = m[i, j] + 0.125, m[i, j] - 0.125
            h = up[i, j].double() - down[i, j].double()
            f = (total(up, w) - total(down, w)) if which == "x" else (total(x, up) - total(x, down))
            # The third derivative of lse along z is below 1/4 of |dz|^3, dz a row of W's entry or of X's; sums to 2^-18.
            slopes = (w[:, j].double().abs().max() ** 3 * dloss[i] if which == "x" else (x[:, j].double().abs() ** 3 * dloss).sum())
            bound = slopes * h * h / 24 + 2 * 2.0 ** -18 * (size + dloss.sum()) / h + 2.0 ** -8 * (
                dloss[i] * w[:, j].double().abs().max() * 2 if which == "x" else (dloss * x[:, j].double().abs()).sum())
            assert abs(f / h - grad[i, j].double().cpu()) <= bound


def test_calls_on_streams_and_in_graphs(tgemm, kernel):
    g = generator(14)
    cases = []
    for i in range(2):
        x, w, target = inputs(g, 290, 515, 137)
        cases.append((place(x, BF16, "odd"), place(w, BF16, "odd"), target.cuda(), torch.rand(290, generator=g).cuda()))
    want = []
    for X, W, t, d in cases:
        loss, lse = tgemm.gemm_ce(X, W, t)
        want.append((loss, lse) + tgemm.gemm_ce_grad(X, W, t, lse, d))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]

    def both(X, W, t, d, stream=None):
        loss, lse = tgemm.gemm_ce(X, W, t, stream=stream)
        return (loss, lse) + tgemm.gemm_ce_grad(X, W, t, lse, d, stream=stream)

    for _ in range(3):
        got = [both(*c, stream=s) for s, c in zip(streams, cases)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for p, q in zip(got, want) for a, b in zip(p, q))
    graphs, got = [], []
    for s, c in zip(streams, cases):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got.append(both(*c))
        graphs.append(graph)
    for _ in range(3):
        for outs in got:
            for o in outs:
                o.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for p, q in zip(got, want) for a, b in zip(p, q))


@pytest.mark.parametrize("T", [4, 300])
def test_a_stage_that_never_fills_is_reported(tgemm, kernel, T):
    g = generator(15)
    x, w, target = inputs(g, T, 600, 512)
    X, W, t = x.cuda(), w.cuda(), target.cuda()
    want = tgemm.gemm_ce(X, W, t)
    assert tgemm.device_status() == 0
    tgemm.binding.set_wait_limit_ns(20_000_000)
    tgemm.binding.set_debug_stall(True)
    try:
        tgemm.gemm_ce(X, W, t)
        assert tgemm.device_status() == tgemm.binding.TGEMM_ERR_DEVICE_TIMEOUT
    finally:
        tgemm.binding.set_debug_stall(False)
        tgemm.binding.set_wait_limit_ns(2_000_000_000)
    got = tgemm.gemm_ce(X, W, t)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_binding_refuses(tgemm):
    X = torch.zeros(4, 8, dtype=BF16, device="cuda")
    W = torch.zeros(6, 8, dtype=BF16, device="cuda")
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    f = torch.zeros(4, device="cuda")
    for error, call in [
            (TypeError, lambda: tgemm.gemm_ce(X.float(), W, t)),
            (ValueError, lambda: tgemm.gemm_ce(X, W[:, :7], t)),
            (TypeError, lambda: tgemm.gemm_ce(X, W, t.int())),
            (ValueError, lambda: tgemm.gemm_ce(X, W, t[:3])),
            (ValueError, lambda: tgemm.gemm_ce(X, W, t.cpu())),
            (ValueError, lambda: tgemm.gemm_ce(X, W, t.repeat_interleave(2)[::2])),
            (tgemm.TgemmError, lambda: tgemm.gemm_ce(X, W, t, alpha=float("nan"))),
            (TypeError, lambda: tgemm.gemm_ce_grad(X, W, t, f.double(), f)),
            (ValueError, lambda: tgemm.gemm_ce_grad(X, W, t, f, f[:2])),
            (ValueError, lambda: tgemm.gemm_ce_grad(X, W, t, f, f, beta=1.0)),
            (ValueError, lambda: tgemm.gemm_ce_grad(X, W, t, f, f, dw_out=X)),
            (ValueError, lambda: tgemm.gemm_ce_grad(X, W, t, f, f, dw_out=W, w_grad=False)),
            (TypeError, lambda: tgemm.gemm_ce_grad(X, W, t, f, f, dx_dtype=torch.float16))]:
        with pytest.raises(error):
            call()
