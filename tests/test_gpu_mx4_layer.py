"""The linear layer of examples/mx4_linear.py: its gradients against the
formulas in 64 bits and against differences of the layer itself."""
import os
import sys

import numpy as np
import pytest
import torch

import mx4_reference as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import mx4_linear  # noqa: E402

pytestmark = pytest.mark.gpu


def host(t):
    return t.detach().double().cpu().numpy()


def as_held(x, fmt):
    """x's values in 4 bits along its rows, 64 bits."""
    g = ref.tensor_scale(x) if fmt == "nvfp4" else 1.0
    return ref.values(*ref.quantize(x, fmt, g), fmt, g)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(40, 48, 64), (129, 100, 300), (300, 260, 33), (1, 16, 16)])
def test_gradients_are_those_of_the_formulas(tgemm, fmt, M, N, K):
    rng = np.random.default_rng(M + N + K)
    x, w, dy = (torch.from_numpy(rng.standard_normal(s)).bfloat16().cuda() for s in ((M, K), (N, K), (M, N)))
    b = torch.from_numpy(rng.standard_normal(N)).float().cuda().requires_grad_()
    x.requires_grad_()
    w = w.float().requires_grad_()
    y = mx4_linear.LinearMx4.apply(x, w, b, fmt)
    y.backward(dy)
    xv, wv, dv = host(x), host(w), host(dy)
    q = lambda m: as_held(m, fmt)  # noqa: E731
    for got, p, r, extra in ((y, q(xv), q(wv).T, host(b)), (x.grad, q(dv), q(wv.T).T, 0.0), (w.grad, q(dv.T), q(xv.T).T, 0.0)):
        want, size = p @ r + extra, np.abs(p) @ np.abs(r) + np.abs(extra)
        tol = (1e-5 + 2.0 ** -20) * size                     # FP32 sums, and the output rule's roundings
        if got.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
        assert (np.abs(host(got) - want) <= tol).all()
    # FP32 sums of BF16 numbers: M - 1 additions.
    assert (np.abs(host(b.grad) - dv.sum(0)) <= M * 2.0 ** -24 * np.abs(dv).sum(0)).all()


def test_gradients_are_differences_of_the_layer(tgemm):
    """On values that 4 bits hold exactly along rows and columns alike
    (multiples of 0.5 beside a 4 in every block, so that scales are 1), the
    layer is bilinear: its differences are its gradients, exactly."""
    M, N, K = 40, 48, 64
    rng = np.random.default_rng(7)

    def draw(R, C):
        v = rng.choice([-3.0, -2.0, -1.5, -1.0, -0.5, 0.0, 0.5, 1.0, 1.5, 2.0, 3.0], (R, C))
        i, j = np.indices((R, C))
        v[(i + j) % 8 == 0] = 4.0
        return v

    x, w, dy = draw(M, K), draw(N, K), draw(M, N)
    run = lambda a, c: host(mx4_linear.LinearMx4.apply(  # noqa: E731
        torch.from_numpy(a).float().cuda(), torch.from_numpy(c).float().cuda(), None, "mxfp4"))
    X, W = (torch.from_numpy(v).float().cuda().requires_grad_() for v in (x, w))
    mx4_linear.LinearMx4.apply(X, W, None, "mxfp4").backward(torch.from_numpy(dy).bfloat16().cuda())
    # y is BF16: differences of y are taken where both are whole BF16 numbers.
    y = run(x, w)
    assert np.array_equal(y, torch.from_numpy(x @ w.T).bfloat16().double().numpy())
    exact = np.abs(x @ w.T - y) == 0
    for which, grad in (("x", host(X.grad)), ("w", host(W.grad))):
        v = {"x": x, "w": w}[which]
        full = dy @ w if which == "x" else dy.T @ x
        if which == "x":
            full = torch.from_numpy(full).bfloat16().double().numpy()      # dx is rounded to BF16
        assert np.array_equal(grad, full)
        for _ in range(12):
            i, j = rng.integers(v.shape[0]), rng.integers(v.shape[1])
            if v[i, j] == 4.0:
                continue
            moved = v.copy()
            moved[i, j] = 1.0 if v[i, j] != 1.0 else 2.0
            h = moved[i, j] - v[i, j]
            y2 = run(moved, w) if which == "x" else run(x, moved)
            true2 = moved @ w.T if which == "x" else x @ moved.T
            ok = exact & (true2 == y2)
            rows = ok[i] if which == "x" else ok[:, i]
            change = ((y2 - y) / h)[i][rows] if which == "x" else ((y2 - y) / h)[:, i][rows]
            slope = w[rows, j] if which == "x" else x[rows, j]
            assert rows.any() and np.array_equal(change, slope)


def test_the_example_trains_and_serves(tgemm, capsys):
    first, last = mx4_linear.main(["--steps", "30", "--tokens", "512", "--inner", "256", "--outer", "128"])
    assert last < 0.2 * first
    assert "one token" in capsys.readouterr().out
