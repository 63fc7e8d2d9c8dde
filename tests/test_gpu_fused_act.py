"""gemm_act and gemm_act_grad against 64-bit forms: whole numbers exactly, over
sizes, storage, strides and alignments; activations within derived bounds."""
import itertools
import zlib

import pytest
import torch

import fused_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
SENTINEL = -77.0


@pytest.fixture(params=["pairs", "few"])
def kernel(request, tgemm):
    """Every test that takes it runs in both of the products' kernels."""
    assert tgemm.fused.set_fused_kernel({"pairs": 0, "few": 1}[request.param]) == 0
    yield request.param
    tgemm.fused.set_fused_kernel(-1)


def generator(*seed):
    return torch.Generator().manual_seed(zlib.crc32(repr(seed).encode()))


def whole(g, *size, most=3):
    return torch.randint(-most, most + 1, size, generator=g).double()


def place(x, dtype, way):
    """x on the GPU: "packed"; "padded", rows 8 elements apart in NaN; "odd", rows an
    odd number apart and off 16 bytes, in NaN."""
    x = x.to(dtype)
    if way == "packed":
        return x.cuda()
    pad, shift = (8, 0) if way == "padded" else (7 - x.shape[1] % 2 * 3 % 2, 1)
    wide = torch.full((x.shape[0] + 1, x.shape[1] + pad + (0 if way == "padded" else (x.shape[1] + pad + 1) % 2)), float("nan"),
                      dtype=dtype, device="cuda")
    view = wide.flatten()[shift:shift + x.shape[0] * wide.shape[1]].view(x.shape[0], wide.shape[1])[:, :x.shape[1]]
    view.copy_(x)
    return view


def room(rows, cols, dtype, way):
    """(a matrix to write, everything around it)."""
    pad, shift = {"packed": (0, 0), "padded": (16, 0), "odd": (5 - cols % 2 * 5 % 2, 3)}[way]
    width = cols + pad
    around = torch.full(((rows + 2) * width + shift,), SENTINEL, dtype=dtype, device="cuda")
    return around[shift:shift + rows * width].view(rows, width)[:, :cols], around


def untouched(view, around):
    before = view.clone()
    view.fill_(SENTINEL)
    ok = bool((around == SENTINEL).all())
    view.copy_(before)
    return ok


def operands(g, M, N, K, ta, tb, way, wide=None, most=3):
    a, b = whole(g, M, K, most=most), whole(g, K, wide or N, most=most)
    A = place(a.t().contiguous() if ta else a, BF16, way)
    B = place(b.t().contiguous() if tb else b, BF16, way)
    return a, b, A, B


SIZES = [(1, 1, 1), (1, 264, 64), (5, 7, 3), (16, 96, 40), (31, 33, 65), (64, 128, 64), (129, 250, 200), (256, 256, 128),
         (257, 513, 130), (300, 1000, 72), (700, 520, 264)]


@pytest.mark.parametrize("way", ["packed", "padded", "odd"])
@pytest.mark.parametrize("ta,tb", list(itertools.product([False, True], repeat=2)))
@pytest.mark.parametrize("M,N,K", SIZES)
def test_whole_numbers_are_exact(tgemm, kernel, M, N, K, ta, tb, way):
    """relu(a b + bias) + R, FP32, with every operand's storage; nothing around C is written."""
    g = generator(M, N, K, ta, tb, way)
    a, b, A, B = operands(g, M, N, K, ta, tb, way)
    bias, r = whole(g, N), whole(g, M, N)
    out, around = room(M, N, F32, way)
    want = (a @ b + bias).clamp(min=0) + r
    got = tgemm.gemm_act(A, B, "relu", trans_a=ta, trans_b=tb, bias=bias.float().cuda(), residual=place(r, F32, way), out=out)
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(out.double().cpu(), want)
    assert untouched(out, around)
    assert tgemm.device_status() == 0


@pytest.mark.parametrize("way", ["packed", "odd"])
@pytest.mark.parametrize("c,r", list(itertools.product([BF16, F32], [None, BF16, F32])))
@pytest.mark.parametrize("keep_z,bias", list(itertools.product([False, True], repeat=2)))
@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (40, 104, 96), (290, 600, 136)])
def test_every_mix_of_types_and_extras(tgemm, kernel, M, N, K, c, r, keep_z, bias, way):
    g = generator(M, N, K, str(c), str(r), keep_z, bias, way)
    a, b, A, B = operands(g, M, N, K, False, True, way, most=1)
    z = a @ b
    e = whole(g, N) if bias else None
    if bias:
        z = z + e
    want = z.clamp(min=0)
    R = None
    if r is not None:
        res = whole(g, M, N)
        want, R = want + res, place(res, r, way)
    assert z.abs().max() <= 256 and want.abs().max() <= 256           # whole numbers that BF16 holds
    out, around = room(M, N, c, way)
    got = tgemm.gemm_act(A, B, "relu", trans_b=True, bias=e.float().cuda() if bias else None, residual=R, keep_z=keep_z, out=out)
    if keep_z:
        assert got[1].dtype == BF16 and torch.equal(got[1].double().cpu(), z)
    assert torch.equal(out.double().cpu(), want)
    assert untouched(out, around)


@pytest.mark.parametrize("way", ["packed", "odd"])
@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("extras", ["", "bias", "residual", "keep_z", "bias residual keep_z"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 136, 64), (17, 100, 72), (130, 129, 200), (300, 392, 136), (260, 1000, 40)])
def test_gated_whole_numbers_are_exact(tgemm, kernel, M, N, K, extras, tb, way):
    g = generator(M, N, K, extras, tb, way)
    a, b, A, B = operands(g, M, N, K, False, tb, way, wide=2 * N, most=1)
    z = a @ b
    bias = whole(g, 2 * N) if "bias" in extras else None
    if bias is not None:
        z = z + bias
    want = z[:, :N].clamp(min=0) * z[:, N:]
    res = whole(g, M, N) if "residual" in extras else None
    if res is not None:
        want = want + res
    out, around = room(M, N, BF16, way)
    got = tgemm.gemm_act(A, B, "relu", trans_b=tb, gated=True, bias=None if bias is None else bias.float().cuda(),
                         residual=None if res is None else place(res, BF16, way), keep_z="keep_z" in extras, out=out)
    if "keep_z" in extras:
        assert torch.equal(got[1].double().cpu(), z.bfloat16().double())
    # Whole numbers below 2^24: the sum before the rounding is exact.
    assert torch.equal(out.cpu(), want.bfloat16())
    assert untouched(out, around)


@pytest.mark.parametrize("gated,residual", [(False, None), (False, F32), (True, F32), (True, BF16)])
def test_long_rows_and_many_tiles(tgemm, kernel, gated, residual):
    """More tiles than SM pairs, sums of several parts, residuals of both types."""
    M, N, K = 1300, 5000, 1160
    g = generator(gated, str(residual))
    a, b, A, B = operands(g, M, N, K, False, True, "packed", wide=2 * N if gated else N, most=1)
    z = (a.float() @ b.float()).double()                              # exact: below 2^24
    want = z[:, :N] * z[:, N:] if gated else z
    R = None
    if residual is not None:
        res = whole(g, M, N)
        want, R = want + res, res.to(residual).cuda()
    c = BF16 if gated else F32
    got = tgemm.gemm_act(A, B, "none", trans_b=True, gated=gated, residual=R, out_dtype=c)
    assert torch.equal(got.cpu(), want.to(c))
    assert tgemm.device_status() == 0


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("c", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(3, 72, 64), (200, 300, 520), (300, 328, 2100), (40, 200, 4000)])
def test_activations_are_within_their_bounds(tgemm, kernel, act, c, M, N, K):
    g = generator(act, str(c), M)
    a = torch.randn(M, K, generator=g).to(BF16)
    b = (torch.randn(N, K, generator=g) * 2.5 / K ** 0.5).to(BF16)    # z as far as some 10
    bias, r = torch.randn(N, generator=g), torch.randn(M, N, generator=g).to(BF16)
    z, ez = ref.sums(a.double(), b.double().t(), bias.double())
    v, ev = ref.act_bound(act, z, ez)
    want = v + r.double()
    got, Z = tgemm.gemm_act(a.cuda(), b.cuda(), act, trans_b=True, bias=bias.cuda(), residual=r.cuda(), keep_z=True, out_dtype=c)
    ref.check(got, want, ref.rounded(want, ev + 2.0 ** -22 * (v.abs() + r.double().abs()), c), "C")
    ref.check(Z, z, ref.rounded(z, ez, BF16), "Z")


@pytest.mark.parametrize("act", ref.ACTS)
def test_activations_of_every_size_of_number(tgemm, act):
    """z from -1e4 to 1e4, one product a sum, exactly z."""
    z = torch.cat([torch.linspace(-12, 12, 4001), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e4, -1e4, 88.0, -88.0, -89.0, -104.0])])
    z = z.to(BF16)[:, None]
    one = torch.ones(1, 8, dtype=BF16)
    got = tgemm.gemm_act(z.cuda(), one.cuda(), act, out_dtype=F32)
    want = ref.act(act, z.double())[0].expand(-1, 8)
    # (2^-40: what FP32's smallest numbers and erfc's far tail leave.)
    ref.check(got, want, 2.0 ** -17 * want.abs() + 2.0 ** -40, act)


@pytest.mark.parametrize("way", ["packed", "odd"])
@pytest.mark.parametrize("c", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 72, 64), (33, 250, 40), (256, 256, 64), (290, 520, 136), (700, 264, 72)])
def test_gradients_of_whole_numbers_are_exact(tgemm, kernel, M, N, K, c, way):
    """relu's: d where z > 0; db sums them exactly."""
    g = generator(M, N, K, str(c), way)
    a, b, A, B = operands(g, M, N, K, False, False, way, most=1)
    z = whole(g, M, N)
    Z = place(z, BF16, way)
    want = (a @ b) * (z > 0)
    out, around = room(M, N, c, way)
    got, db = tgemm.gemm_act_grad(A, B, Z, "relu", out=out)
    assert torch.equal(got.double().cpu(), want)
    assert db.dtype == F32 and torch.equal(db.double().cpu(), want.sum(dim=0))
    assert untouched(out, around)
    alone = tgemm.gemm_act_grad(A, B, Z, "relu", bias_grad=False, out_dtype=c)
    assert torch.equal(alone, got)
    assert tgemm.device_status() == 0


@pytest.mark.parametrize("way", ["packed", "odd"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (5, 72, 64), (290, 130, 136), (300, 520, 200)])
def test_gated_gradients_of_whole_numbers_are_exact(tgemm, kernel, M, N, K, way):
    g = generator(M, N, K, way)
    a, b, A, B = operands(g, M, N, K, False, False, way, most=1)
    z = whole(g, M, 2 * N)
    d, gate, up = a @ b, z[:, :N], z[:, N:]
    want = torch.cat((d * up * (gate > 0), d * gate.clamp(min=0)), dim=1)
    out, around = room(M, 2 * N, BF16, way)
    got, db = tgemm.gemm_act_grad(A, B, place(z, BF16, way), "relu", gated=True, out=out)
    assert torch.equal(got.cpu(), want.bfloat16())
    assert torch.equal(db.double().cpu(), want.sum(dim=0))
    assert untouched(out, around)


@pytest.mark.parametrize("gated,in_place", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M,N,K", [(1300, 5000, 200), (1100, 2200, 72)])
def test_gradients_of_many_tiles(tgemm, kernel, M, N, K, gated, in_place):
    """Tiles of fewer than 256 columns, whose last turn is short."""
    g = generator(M, gated, in_place)
    a, b, A, B = operands(g, M, N, K, False, False, "packed", most=1)
    z = whole(g, M, 2 * N if gated else N)
    Z = z.to(BF16).cuda()
    d = (a.float() @ b.float()).double()
    want = torch.cat((d * z[:, N:] * (z[:, :N] > 0), d * z[:, :N].clamp(min=0)), dim=1) if gated else d * (z > 0)
    dz, db = tgemm.gemm_act_grad(A, B, Z, "relu", gated=gated, out=Z if in_place else None)
    assert torch.equal(dz.cpu(), want.bfloat16()) and torch.equal(db.double().cpu(), want.sum(dim=0))


@pytest.mark.parametrize("M,N", [(1300, 5000), (700, 2208), (700, 2207), (2400, 1500)])
@pytest.mark.parametrize("c,r", [(BF16, None), (BF16, BF16), (F32, F32), (BF16, F32)])
def test_residuals_of_many_tiles(tgemm, kernel, M, N, c, r):
    """The same, C in place of R where the types agree, and Z beside it."""
    K = 200
    g = generator(M, N, str(c), str(r))
    a, b, A, B = operands(g, M, N, K, False, True, "packed", most=1)
    z = (a.float() @ b.float()).double()
    assert z.abs().max() <= 256
    res = whole(g, M, N) if r is not None else torch.zeros(M, N).double()
    R = None if r is None else res.to(r).cuda()
    out = R if c == r else None
    C, Z = tgemm.gemm_act(A, B, "relu", trans_b=True, residual=R, keep_z=True, out_dtype=c, out=out)
    assert torch.equal(C.cpu(), (z.clamp(min=0) + res).to(c)) and torch.equal(Z.double().cpu(), z)
    R = None if r is None else res.to(r).cuda()
    C = tgemm.gemm_act(A, B, trans_b=True, residual=R, out_dtype=c, out=R if c == r else None)
    assert torch.equal(C.cpu(), (z + res).to(c))


@pytest.mark.parametrize("ta,tb", [(True, False), (False, True), (True, True)])
def test_gradients_take_every_storage(tgemm, kernel, ta, tb):
    M, N, K = 150, 300, 90
    g = generator(ta, tb)
    a, b, A, B = operands(g, M, N, K, ta, tb, "odd", most=1)
    z = whole(g, M, N)
    got, db = tgemm.gemm_act_grad(A, B, z.to(BF16).cuda(), "relu", trans_a=ta, trans_b=tb)
    want = (a @ b) * (z > 0)
    assert torch.equal(got.double().cpu(), want) and torch.equal(db.double().cpu(), want.sum(dim=0))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("M,N,K", [(3, 72, 64), (330, 200, 520), (300, 328, 2100)])
def test_gradients_are_within_their_bounds(tgemm, kernel, act, gated, M, N, K):
    g = generator(act, gated, M)
    a = torch.randn(M, K, generator=g).to(BF16)
    b = (torch.randn(K, N, generator=g) / K ** 0.5).to(BF16)
    z = (torch.randn(M, 2 * N if gated else N, generator=g) * 2).to(BF16)
    d, ed = ref.sums(a.double(), b.double())
    zd = z.double()
    if gated:
        gate, up = zd[:, :N], zd[:, N:]
        v, ev = ref.act_bound(act, gate, torch.zeros_like(gate))
        s, es = ref.grad_bound(act, gate)
        want = torch.cat((d * up * s, d * v), dim=1)
        tol = torch.cat((ed * (up * s).abs() + (d.abs() + ed) * up.abs() * es, ed * v.abs() + (d.abs() + ed) * ev), dim=1)
    else:
        s, es = ref.grad_bound(act, zd)
        want, tol = d * s, ed * s.abs() + (d.abs() + ed) * es
    tol = tol + 2.0 ** -22 * want.abs()
    got, db = tgemm.gemm_act_grad(a.cuda(), b.cuda(), z.cuda(), act, gated=gated)
    ref.check(got, want, ref.rounded(want, tol, BF16), "dZ")
    # Sums of 32, then of blocks: each addition rounds to 2^-24.
    ref.check(db, want.sum(dim=0), tol.sum(dim=0) + (32 + M / 32 + 8) * 2.0 ** -24 * (want.abs() + tol).sum(dim=0), "db")


def test_a_gradient_is_a_difference_of_the_layer(tgemm):
    """C of gemm_act moved along one entry of A changes as gemm_act_grad says: with
    t = A + h E, d/dh sum(C U) = (dZ B^T)[E], dZ = U act'(Z) (U through an identity)."""
    M, N, K = 64, 64, 64
    g = generator(9)
    a = torch.randn(M, K, generator=g).to(BF16)
    w = (torch.randn(N, K, generator=g) / 8).to(BF16)
    u = torch.randn(M, N, generator=g).to(BF16)
    for act in ref.ACTS[2:]:
        c, z = tgemm.gemm_act(a.cuda(), w.cuda(), act, trans_b=True, keep_z=True, out_dtype=F32)
        dz, _ = tgemm.gemm_act_grad(u.cuda(), torch.eye(N, dtype=BF16).cuda(), z, act, out_dtype=F32)
        da = tgemm.gemm_act(dz.to(BF16), w.cuda(), out_dtype=F32).double().cpu()
        for i, k in ((0, 0), (5, 17), (63, 40)):
            up, down = a.clone(), a.clone()
            up[i, k], down[i, k] = a[i, k] + 0.25, a[i, k] - 0.25
            h = (up[i, k].double() - down[i, k].double())
            f = [(tgemm.gemm_act(x.cuda(), w.cuda(), act, trans_b=True, out_dtype=F32)[i].double().cpu() * u[i].double()).sum()
                 for x in (up, down)]
            # A central difference is off by h^2 / 24 of the third derivative (below 2 here) of each
            # of the row's terms, h w at most; Z and dZ are BF16: 2^-8 of each term, twice.
            terms = (u[i].double() * w[:, k].double()).abs().sum()
            third = (u[i].double().abs() * w[:, k].double().abs() ** 3).sum() * 2 * h * h / 24
            assert abs((f[0] - f[1]) / h - da[i, k]) <= third + 3 * 2.0 ** -8 * 1.13 * terms


def test_in_place(tgemm, kernel):
    """R may be C, and dZ may be Z."""
    g = generator(4)
    for M, N, K in ((40, 104, 64), (290, 520, 136), (290, 521, 136)):
        a, b, A, B = operands(g, M, N, K, False, True, "packed", most=1)
        r, z = whole(g, M, N), whole(g, M, N)
        for dtype in (BF16, F32):
            C = r.to(dtype).cuda()
            tgemm.gemm_act(A, B, trans_b=True, residual=C, out=C)
            assert torch.equal(C.double().cpu(), a @ b + r)
        Z = z.to(BF16).cuda()
        tgemm.gemm_act_grad(A, B, Z, "relu", trans_b=True, out=Z)
        assert torch.equal(Z.double().cpu(), (a @ b) * (z > 0))
        z2 = whole(g, M, 2 * N)
        Z = z2.to(BF16).cuda()
        tgemm.gemm_act_grad(A, B, Z, "relu", trans_b=True, gated=True, out=Z)
        d = a @ b
        assert torch.equal(Z.cpu(), torch.cat((d * z2[:, N:] * (z2[:, :N] > 0), d * z2[:, :N].clamp(min=0)), 1).bfloat16())


@pytest.mark.parametrize("M,N,K", [(4, 24, 0), (0, 24, 8), (4, 0, 8), (0, 0, 0), (300, 40, 0)])
def test_sizes_of_zero(tgemm, kernel, M, N, K):
    A, B = torch.ones(M, K, dtype=BF16, device="cuda"), torch.ones(N, K, dtype=BF16, device="cuda")
    bias = torch.arange(N, dtype=F32, device="cuda") - 5
    r = torch.full((M, N), 2.0, dtype=BF16, device="cuda")
    want = bias.clamp(min=0).expand(M, N) + 2 if K == 0 else torch.empty(M, N, device="cuda")
    C, Z = tgemm.gemm_act(A, B, "relu", trans_b=True, bias=bias, residual=r, keep_z=True)
    assert C.shape == (M, N) and Z.shape == (M, N)
    if K == 0:
        assert torch.equal(C.float(), want) and torch.equal(Z.float(), bias.expand(M, N))
    dz, db = tgemm.gemm_act_grad(A, B.t().contiguous(), torch.ones(M, N, dtype=BF16, device="cuda"), "silu")
    assert dz.shape == (M, N) and torch.equal(db, torch.zeros(N, device="cuda"))
    assert not dz.any()


def test_infinities_and_nan_stay_in_their_rows_and_columns(tgemm, kernel):
    M, N, K = 300, 280, 96
    g = generator(5)
    a, b, A, B = operands(g, M, N, K, False, True, "packed", most=1)
    A[7, 3], A[299, 90], B[13, 5] = float("nan"), float("inf"), float("inf")
    C = tgemm.gemm_act(A, B, trans_b=True, out_dtype=F32).double().cpu()
    rows = torch.ones(M, dtype=torch.bool)
    rows[[7, 299]] = False
    cols = torch.ones(N, dtype=torch.bool)
    cols[13] = False
    assert torch.equal(C[rows][:, cols], (a @ b)[rows][:, cols])
    assert C[7].isnan().all() and not C[299].isfinite().any()
    # The column sums of a gradient: rows past M add nothing, whatever B holds.
    dz, db = tgemm.gemm_act_grad(a.to(BF16).cuda()[:130], B, torch.ones(130, N, dtype=BF16, device="cuda"), "relu", trans_b=True)
    assert torch.equal(db.double().cpu()[cols], (a[:130] @ b).sum(0)[cols])


@pytest.mark.parametrize("N", [40000, 40001])
def test_offsets_past_32_bits(tgemm, N):
    """C, R and Z of more than 2^31 elements; rows at both ends and across the middle."""
    M, K = 70000, 16
    g = generator(N)
    a, b = whole(g, M, K, most=1), whole(g, K, N, most=1)
    A, B = a.to(BF16).cuda(), b.to(BF16).cuda()
    rows = torch.tensor([0, 53686, 53687, 53688, 69000, M - 1])
    R = torch.zeros(M, N, dtype=BF16, device="cuda")
    r = whole(g, len(rows), N)
    R[rows.cuda()] = r.to(BF16).cuda()
    C, Z = tgemm.gemm_act(A, B, "relu", residual=R, keep_z=True)
    z = a[rows] @ b
    assert torch.equal(C[rows.cuda()].double().cpu(), z.clamp(min=0) + r)
    assert torch.equal(Z[rows.cuda()].double().cpu(), z)
    del C, R
    dz, db = tgemm.gemm_act_grad(A, B, Z, "relu", out=Z)
    assert torch.equal(dz[rows.cuda()].double().cpu(), z.clamp(min=0))
    assert tgemm.device_status() == 0


def test_calls_on_streams_and_in_graphs(tgemm, kernel):
    """Two calls at once on two streams, and two graphs that replay together, with
    scratch (operands off 16 bytes, column sums) in both."""
    g = generator(6)
    M, N, K = 290, 515, 137
    cases = []
    for i in range(2):
        a, b, A, B = operands(g, M, N, K, False, False, "odd", most=1)
        z = whole(g, M, N)
        cases.append((A, B, z.to(BF16).cuda(), (a @ b) * (z > 0)))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()

    def right(outs):
        for (dz, db), (_, _, _, want) in zip(outs, cases):
            assert torch.equal(dz.double().cpu(), want) and torch.equal(db.double().cpu(), want.sum(0))

    for _ in range(3):
        outs = [tgemm.gemm_act_grad(A, B, Z, "relu", stream=s) for s, (A, B, Z, _) in zip(streams, cases)]
        torch.cuda.synchronize()
        right(outs)
    graphs, outs = [], []
    for s, (A, B, Z, _) in zip(streams, cases):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(tgemm.gemm_act_grad(A, B, Z, "relu"))
        graphs.append(graph)
    for _ in range(3):
        for dz, db in outs:
            dz.zero_(), db.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        right(outs)
    assert tgemm.device_status() == 0


def test_results_do_not_depend_on_timing(tgemm, kernel):
    g = generator(8)
    a, b = (torch.randn(s, generator=g).to(BF16).cuda() for s in ((1000, 1500), (1500, 900)))
    z = torch.randn(1000, 900, generator=g).to(BF16).cuda()
    first = tgemm.gemm_act_grad(a, b, z, "gelu")
    for _ in range(5):
        again = tgemm.gemm_act_grad(a, b, z, "gelu")
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("M,N", [(4, 200), (300, 600)])
@pytest.mark.parametrize("grad", [False, True])
def test_a_stage_that_never_fills_is_reported(tgemm, kernel, grad, M, N):
    g = generator(7)
    a, b, A, B = operands(g, M, N, 512, False, True, "packed", most=1)
    z = whole(g, M, N)
    call = (lambda: tgemm.gemm_act_grad(A, B, z.to(BF16).cuda(), "relu", trans_b=True, bias_grad=False, out_dtype=F32)) if grad else \
           (lambda: tgemm.gemm_act(A, B, "relu", trans_b=True, out_dtype=F32))
    want = (a @ b) * (z > 0) if grad else (a @ b).clamp(min=0)
    assert tgemm.device_status() == 0
    tgemm.binding.set_wait_limit_ns(20_000_000)
    tgemm.binding.set_debug_stall(True)
    try:
        call()
        assert tgemm.device_status() == tgemm.binding.TGEMM_ERR_DEVICE_TIMEOUT
    finally:
        tgemm.binding.set_debug_stall(False)
        tgemm.binding.set_wait_limit_ns(2_000_000_000)
    assert tgemm.device_status() == 0
    assert torch.equal(call().double().cpu(), want)


def test_binding_refuses(tgemm):
    A = torch.zeros(4, 8, dtype=BF16, device="cuda")
    B = torch.zeros(6, 8, dtype=BF16, device="cuda")
    Z = torch.zeros(4, 6, dtype=BF16, device="cuda")
    for error, call in [
            (TypeError, lambda: tgemm.gemm_act(A.float(), B, trans_b=True)),
            (TypeError, lambda: tgemm.gemm_act(A, B.half(), trans_b=True)),
            (ValueError, lambda: tgemm.gemm_act(A, B)),
            (ValueError, lambda: tgemm.gemm_act(A, B, "tanh", trans_b=True)),
            (ValueError, lambda: tgemm.gemm_act(A[:, ::2], B[:, ::2], trans_b=True)),
            (ValueError, lambda: tgemm.gemm_act(A[:1].expand(4, 8), B, trans_b=True)),
            (ValueError, lambda: tgemm.gemm_act(A, B, trans_b=True, bias=torch.zeros(5, device="cuda"))),
            (TypeError, lambda: tgemm.gemm_act(A, B, trans_b=True, bias=torch.zeros(6, device="cuda", dtype=BF16))),
            (ValueError, lambda: tgemm.gemm_act(A, B, trans_b=True, bias=torch.zeros(6))),
            (ValueError, lambda: tgemm.gemm_act(A, B, trans_b=True, residual=A)),
            (TypeError, lambda: tgemm.gemm_act(A, B, trans_b=True, residual=Z.half())),
            (TypeError, lambda: tgemm.gemm_act(A, B, trans_b=True, out_dtype=torch.float16)),
            (ValueError, lambda: tgemm.gemm_act(A, B, trans_b=True, out=A)),
            (TypeError, lambda: tgemm.gemm_act(A, B, trans_b=True, gated=True, out_dtype=F32)),
            (ValueError, lambda: tgemm.gemm_act(A, B[:5], trans_b=True, gated=True)),
            (ValueError, lambda: tgemm.gemm_act_grad(A, B, A, trans_b=True)),
            (TypeError, lambda: tgemm.gemm_act_grad(A, B, Z.float(), trans_b=True)),
            (ValueError, lambda: tgemm.gemm_act_grad(A, B, Z, trans_b=True, gated=True)),
            (TypeError, lambda: tgemm.gemm_act_grad(A, B[:3], Z, trans_b=True, gated=True, out_dtype=F32))]:
        with pytest.raises(error):
            call()
