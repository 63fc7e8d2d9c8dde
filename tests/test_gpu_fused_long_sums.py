"""What results of 32 bits of the fused products keep of long sums, against 64 bits:
the header's bounds, relative to the result's norm.

A tensor-core step of 16 columns of K adds to an FP32 sum with low bits cut off,
which takes some 1.5e-8 of the sum from it each time where terms have random signs
(6e-8 a stage of 64), and up to 2^-23 of it where all have one: a part of 13 stages
loses 0.8e-6 and 1.5e-6 in the norm, however many parts there are, and activations
make at most 1.2 of it (the largest ratio of z act'(z) to act(z) in the norm, z normal).
"""
import pytest
import torch

import fused_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
KERNELS = {"auto": -1, "pairs": 0, "few": 1}


@pytest.fixture(autouse=True)
def by_the_model(tgemm):
    yield
    tgemm.fused.set_fused_kernel(-1)


def normal(seed, *size, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(size, generator=g, device="cuda") * scale).to(BF16)


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


# Boxes and a column a lane (513), pairs that share sums (tiles few, sums long) and that do
# not, few tiles alone and in clusters; sums of a little over one part, of several, of many.
SIZES = [("pairs", 300, 512, 1040), ("pairs", 4096, 2560, 1664), ("pairs", 4096, 2565, 1664), ("pairs", 300, 512, 2100),
         ("pairs", 300, 512, 4096), ("pairs", 300, 513, 4096), ("pairs", 1500, 1500, 4096), ("pairs", 300, 512, 14336),
         ("pairs", 300, 513, 14336), ("pairs", 2600, 4096, 14336), ("few", 300, 512, 1040), ("few", 40, 512, 1664),
         ("few", 300, 512, 2100), ("few", 1500, 1500, 4096), ("few", 8, 513, 4096), ("few", 300, 512, 14336), ("few", 8, 512, 65536),
         ("auto", 300, 512, 1024), ("auto", 16, 4096, 14336), ("auto", 3000, 5001, 1537)]


@pytest.mark.parametrize("kernel,M,N,K", SIZES)
def test_fp32_results_of_long_sums(tgemm, kernel, M, N, K):
    A, B = normal(M + K, M, K), normal(N + K, N, K, scale=K ** -0.5)
    z = A.double() @ B.double().t()
    tgemm.fused.set_fused_kernel(KERNELS[kernel])
    for act in ref.ACTS:
        got, want = tgemm.gemm_act(A, B, act, trans_b=True, out_dtype=F32), ref.act(act, z)[0]
        bound = 1e-6
        if M == N:
            # One seed: B is A's numbers, and terms on the diagonal are squares, of one sign: 2e-6 of
            # them (the next test's), 1e-6 of the others; errors of different entries add in squares.
            squares, all_of_it = want.diagonal().norm() ** 2, want.norm() ** 2
            bound = (((1e-6) ** 2 * (all_of_it - squares) + (2e-6) ** 2 * squares) / all_of_it).sqrt().item()
        assert off(got, want) <= bound, act


@pytest.mark.parametrize("kernel,M,N,K", [s for s in SIZES if s[3] >= 1537])
def test_fp32_results_of_long_sums_of_one_sign(tgemm, kernel, M, N, K):
    A, B = normal(M + K, M, K).abs(), normal(N + K, N, K, scale=1 / K).abs()
    tgemm.fused.set_fused_kernel(KERNELS[kernel])
    got = tgemm.gemm_act(A, B, trans_b=True, out_dtype=F32)
    assert off(got, A.double() @ B.double().t()) <= 2e-6


@pytest.mark.parametrize("kernel,T,V,D", [("pairs", 300, 5000, 1024), ("pairs", 300, 5001, 4096), ("pairs", 300, 5000, 14336),
                                          ("pairs", 300, 20000, 4096), ("pairs", 2000, 20000, 4096), ("pairs", 300, 50000, 1024),
                                          ("pairs", 40, 30000, 14336), ("few", 300, 20000, 4096), ("few", 8, 30000, 4096),
                                          ("auto", 4, 30000, 2048), ("auto", 1300, 20001, 2049)])
def test_losses_of_long_sums(tgemm, kernel, T, V, D):
    """Targets some 8 above logits of spread 1, as a trained head's are. With every logit z losing c z a loss is
    off by c (1 - p) z_t, p the target's probability: 4 c of the loss at V = 5000 (p = 0.27, loss 1.3), 3 c at 20000
    (0.08, 2.5), less at larger V; c is 2.5e-7 in parts of 4 stages. lse is dominated by the largest logits: c of itself."""
    W = normal(D, V, D, scale=D ** -0.5)
    g = torch.Generator(device="cuda").manual_seed(T)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    X = (torch.randn((T, D), generator=g, device="cuda") + 8 * W[target].float()).to(BF16)
    z = X.double() @ W.double().t()
    want = torch.logsumexp(z, dim=1)
    tgemm.fused.set_fused_kernel(KERNELS[kernel])
    loss, lse = tgemm.gemm_ce(X, W, target)
    assert off(lse, want) <= 2.5e-7
    assert off(loss, want - z.gather(1, target[:, None])[:, 0]) <= 1e-6


@pytest.mark.parametrize("kernel,M,N,K", [("pairs", 300, 512, 1152), ("pairs", 300, 513, 2100), ("pairs", 1500, 1500, 4096),
                                          ("pairs", 8192, 512, 4096), ("pairs", 300, 512, 14336), ("few", 300, 512, 1152),
                                          ("few", 1500, 1504, 4096), ("few", 40, 513, 4096), ("few", 300, 512, 14336),
                                          ("auto", 256, 1024, 1024), ("auto", 2000, 4099, 2048)])
@pytest.mark.parametrize("gated", [False, True])
def test_bias_gradients_of_long_sums(tgemm, kernel, M, N, K, gated):
    """db, and dZ in 32 bits: slopes leave the sums' relative error as it is."""
    A, B, Z = normal(M + 1, M, K, scale=1e-3), normal(N + 2, K, N, scale=K ** -0.5), normal(K + 3, M, 2 * N if gated else N)
    d, z = A.double() @ B.double(), Z.double()
    tgemm.fused.set_fused_kernel(KERNELS[kernel])
    for act in ref.ACTS:
        if gated:
            v, s = ref.act(act, z[:, :N])
            want = torch.cat((d * z[:, N:] * s, d * v), dim=1)
        else:
            want = d * ref.act(act, z)[1]
        got, db = tgemm.gemm_act_grad(A, B, Z, act, gated=gated, out_dtype=BF16 if gated else F32)
        assert off(db, want.sum(dim=0)) <= 1e-6, act
        if not gated:
            assert off(got, want) <= 1e-6, act


@pytest.mark.parametrize("kernel,M,N,K", [("pairs", 300, 512, 1152), ("pairs", 2048, 513, 4096), ("few", 300, 512, 4096)])
@pytest.mark.parametrize("gated", [False, True])
def test_bias_gradients_of_long_sums_of_one_sign(tgemm, kernel, M, N, K, gated):
    A, B = normal(M + 1, M, K).abs(), normal(N + 2, K, N, scale=1 / K).abs()
    Z = normal(K + 3, M, 2 * N if gated else N).abs() + 1
    d, z = A.double() @ B.double(), Z.double()
    want = (torch.cat((d * z[:, N:], d * z[:, :N]), dim=1) if gated else d).sum(dim=0)
    tgemm.fused.set_fused_kernel(KERNELS[kernel])
    assert off(tgemm.gemm_act_grad(A, B, Z, "relu", gated=gated)[1], want) <= 2e-6


def test_bias_gradients_of_many_rows_of_long_sums(tgemm):
    """The dZ's errors add up over the rows as they themselves do: db is off by as much of its norm."""
    M, N, K = 65536, 256, 4096
    A, B, Z = normal(3, M, K, scale=1e-3), normal(4, K, N, scale=K ** -0.5), normal(5, M, N)
    d = A.double() @ B.double()
    for act in ref.ACTS:
        assert off(tgemm.gemm_act_grad(A, B, Z, act)[1], (d * ref.act(act, Z.double())[1]).sum(dim=0)) <= 1e-6, act


@pytest.mark.parametrize("kernel", ["pairs", "few"])
@pytest.mark.parametrize("N", [64, 61])
def test_bias_gradients_of_a_million_rows(tgemm, kernel, N):
    """One stage of K: 0.7e-7 of the norm. What is left is the sum over the rows: one of n terms takes n additions of
    2^-25 of the sum so far each, as an error's standard deviation at most, and the sum grows as the root of its terms:
    (n / 2)^(1/2) 2^-25 of it. A block of 32 or 64 rows, 64 blocks, 64 such sums to a warp, and 8 warps: below 5e-7."""
    M, K = 2 ** 20 + 77, 64
    A, B, Z = normal(1, M, K), normal(2, K, N, scale=K ** -0.5), normal(3, M, N)
    want = ((A.double() @ B.double()) * ref.act("silu", Z.double())[1]).sum(dim=0)
    tgemm.fused.set_fused_kernel(KERNELS[kernel])
    assert off(tgemm.gemm_act_grad(A, B, Z, "silu")[1], want) <= 5e-7


@pytest.mark.parametrize("kernel", ["pairs", "few", "auto"])
@pytest.mark.parametrize("k", [12, 16, 20])
@pytest.mark.parametrize("T,V,D", [(1, 1000, 256), (40, 3000, 4096), (300, 1001, 1024), (600, 8000, 4096)])
def test_gradients_of_sure_tokens(tgemm, kernel, k, T, V, D):
    """Targets k above logits of spread 1: 1 - p is down to 1e-5, and p - 1, the most of a row's dX, is the difference of
    an exponential and 1. Against the gradient with an exact lse it is off by lse's roundings (2^-23 of lse), an exponential's
    (2^-21), what logits lose in parts of 4 stages (2.5e-7 of the target's, where lse and dz come from
    different kernels), and its own rounding to BF16. The other entries share a row's relative error."""
    W = normal(D + k, V, D, scale=D ** -0.5)
    g = torch.Generator(device="cuda").manual_seed(T)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    X = (torch.randn((T, D), generator=g, device="cuda") + k * W[target].float()).to(BF16)
    rows = torch.arange(T, device="cuda")
    z = X.double() @ W.double().t()
    exact = torch.logsumexp(z, dim=1)
    p, picked = torch.exp(z - exact[:, None]), z[rows, target]
    sure = -torch.expm1(picked - exact)
    p[rows, target] = -sure
    want_x, want_w = p @ W.double(), p.t() @ X.double()
    each = 2.0 ** -8 + (2.0 ** -23 * exact + 2.0 ** -21 + 2.5e-7 * picked) / sure
    tgemm.fused.set_fused_kernel(KERNELS[kernel])
    _, lse = tgemm.gemm_ce(X, W, target)
    dx, dw = tgemm.gemm_ce_grad(X, W, target, lse, torch.ones(T, device="cuda"), dx_dtype=F32, dw_dtype=F32)
    assert (dx.double() - want_x).norm() <= (each * want_x.norm(dim=1)).norm()
    assert (dw.double() - want_w).norm() <= (each[:, None] * (p.abs() * X.double().norm(dim=1)[:, None])).norm()
