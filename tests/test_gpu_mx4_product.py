"""gemm_mx4 (both operands in 4 bits) and gemm_w4 (BF16 rows x 4-bit weights)
against products in 64 bits.

Two kinds of operands. "whole": products of codes and scales are multiples of
a unit, and sum |a||b| stays below 2^24 units (checked), so every order of
summation in FP32 is exact and the result has to be equal. "wide": scales over
many octaves; a sum of FP32 additions is within the FP32 path's tolerance,
1e-5 sum |a||b|. alpha, beta, bias and the tensor scales add at most eight FP32
roundings of terms no larger than the sum of the terms' magnitudes (2^-20 of
it), a BF16 result half a unit in the last place (2^-8 of it, with the next
binade).
"""
import threading

import numpy as np
import pytest
import torch

import mx4_reference as ref

pytestmark = pytest.mark.gpu
FMTS = ["mxfp4", "nvfp4"]
OPS = ["mx4", "w4"]
F32_REL = 1e-5
SIZES = [(1, 1, 1), (1, 1, 16), (1, 8, 31), (2, 3, 33), (3, 17, 32), (16, 128, 64), (17, 129, 96), (127, 255, 100),
         (128, 256, 256), (129, 257, 257), (130, 64, 513), (256, 512, 300), (300, 520, 1537), (1, 4096, 1024),
         (8, 1000, 2048), (9, 33, 1027), (24, 200, 700), (25, 130, 640), (33, 97, 1600), (64, 320, 1999), (65, 40, 1024), (260, 1030, 768), (2100, 2600, 300)]


class Operand:
    """A 4-bit matrix on the device and its values in 64 bits."""

    def __init__(self, tgemm, R, C, fmt, kind, seed, g=None):
        rng = np.random.default_rng(seed)
        codes = rng.integers(0, 16, (R, C))
        nb = ref.blocks(C, fmt)
        if fmt == "mxfp4":
            scales = rng.integers(126, 129, (R, nb)) if kind == "whole" else rng.integers(100, 150, (R, nb))
        else:
            scales = rng.integers(0x38, 0x42, (R, nb)) if kind == "whole" else rng.integers(0, 0x7F, (R, nb))
        if kind == "normal":
            scales = rng.integers(*{"mxfp4": (117, 121), "nvfp4": (0x58, 0x7F)}[fmt], (R, nb))
        self.g = None if g is None else torch.tensor([g], device="cuda")
        self.q = tgemm.mx4_pack(torch.from_numpy(ref.pack_codes(codes)).cuda(),
                                torch.from_numpy(np.ascontiguousarray(scales.astype(np.uint8))).cuda(), fmt, cols=C, tensor_scale=self.g)
        self.v = ref.values(codes, scales, fmt)
        if self.g is not None:
            self.v = self.v * float(self.g)


def activations(M, K, kind, seed, ld=None):
    rng = np.random.default_rng(seed)
    x = rng.integers(-4, 5, (M, K)) / 2.0 if kind == "whole" else rng.standard_normal((M, K)) * 2.0 ** rng.integers(-9, 9, (M, 1))
    if kind == "normal":
        x = rng.standard_normal((M, K))
    X = torch.full((M, ld or K), float("nan"), dtype=torch.bfloat16)
    X[:, :K] = torch.from_numpy(x).to(torch.bfloat16)
    X = X.cuda()[:, :K]
    return X, X.double().cpu().numpy()


def operands(tgemm, op, M, N, K, fmt, kind, g=None):
    """(call's A, call's B, A and B in 64 bits)."""
    B = Operand(tgemm, N, K, fmt, kind, M + 3 * N + 7 * K + 1, g)
    if op == "mx4":
        A = Operand(tgemm, M, K, fmt, kind, M + 5 * N + 11 * K, g)
        return A.q, B.q, A.v, B.v
    X, x = activations(M, K, kind, M + K, ld=K + (M + N) % 3 * 3)
    return X, B.q, x, B.v


def call(tgemm, op):
    return tgemm.gemm_mx4 if op == "mx4" else tgemm.gemm_w4


def guarded(M, N, dtype, pad):
    """An M x N view with `pad` columns after each row, and a row before and after."""
    store = torch.full((M + 2, N + pad), -77.0, dtype=dtype, device="cuda")
    return store, store[1:M + 1, :N]


def untouched(store, M, N):
    return bool((store[0] == -77).all() and (store[-1] == -77).all() and (store[:, N:] == -77).all())


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("op", OPS)
def test_whole_numbers_are_exact(tgemm, op, fmt, M, N, K):
    A, B, a, b = operands(tgemm, op, M, N, K, fmt, "whole")
    unit = {"mxfp4": 2.0 ** -4, "nvfp4": 2.0 ** -8}[fmt]      # 0.5 x 0.5 x smallest scale steps
    if op == "w4":
        unit = 2.0 ** -5
    assert (np.abs(a) @ np.abs(b).T).max(initial=0.0) < unit * 2.0 ** 24
    want = a @ b.T
    for pad in (0, 3):
        store, out = guarded(M, N, torch.float32, pad)
        call(tgemm, op)(A, B, out=out)
        assert tgemm.device_status() == 0
        assert np.array_equal(out.double().cpu().numpy(), want)
        assert untouched(store, M, N)
    store, out = guarded(M, N, torch.bfloat16, 1)
    call(tgemm, op)(A, B, out=out)
    assert torch.equal(out.cpu(), torch.from_numpy(want).float().bfloat16())
    assert untouched(store, M, N)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("op", OPS)
def test_wide_scales_and_the_output_rule(tgemm, op, fmt, M, N, K):
    g = 0.0123 if fmt == "nvfp4" else None
    A, B, a, b = operands(tgemm, op, M, N, K, fmt, "wide", g)
    rng = np.random.default_rng(K)
    size = float(np.abs(a @ b.T).mean()) + 1e-30
    bias = torch.from_numpy(rng.standard_normal(N) * size).float().cuda()
    old = torch.from_numpy(rng.standard_normal((M, N)) * size).float().cuda()
    absab = np.abs(a) @ np.abs(b).T
    fn = call(tgemm, op)
    for dtype in (torch.float32, torch.bfloat16):
        def check(got, want, terms):
            tol = F32_REL * absab * 1.0 + 2.0 ** -20 * terms
            if dtype == torch.bfloat16:
                tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
            err = np.abs(got.double().cpu().numpy() - want)
            assert got.dtype == dtype and np.isfinite(err).all() and (err <= tol).all(), float((err - tol).max())

        check(fn(A, B, out_dtype=dtype), a @ b.T, absab)
        check(fn(A, B, out_dtype=dtype, bias=bias), a @ b.T + bias.double().cpu().numpy(),
              absab + np.abs(bias.double().cpu().numpy()))
        store, out = guarded(M, N, dtype, 2)
        out.copy_(old)
        c = out.double().cpu().numpy()
        fn(A, B, alpha=-0.75, beta=0.5, bias=bias, out=out)
        check(out, -0.75 * (a @ b.T) + 0.5 * c + bias.double().cpu().numpy(),
              absab + np.abs(c) + np.abs(bias.double().cpu().numpy()))
        assert untouched(store, M, N)
    assert tgemm.device_status() == 0


@pytest.mark.parametrize("op", OPS)
def test_a_long_sum(tgemm, op):
    A, B, a, b = operands(tgemm, op, 20, 260, 14336, "nvfp4", "wide", 0.5)
    got = call(tgemm, op)(A, B).double().cpu().numpy()
    assert (np.abs(got - a @ b.T) <= (F32_REL + 2.0 ** -20) * (np.abs(a) @ np.abs(b).T)).all()


@pytest.mark.parametrize("M,N,K", [(16, 4096, 14336), (100, 300, 9000), (60, 20000, 4096), (2100, 1100, 14336)])
@pytest.mark.parametrize("fmt", FMTS)
def test_long_sums_keep_their_low_bits(tgemm, fmt, M, N, K):
    """Positive terms, whose roundings all go one way where they are cut off.

    A part of 1024 columns is 64 steps of an MMA; each step cuts off at most
    2^-23 of the partial sum in adding its 16 products up and as much in adding
    to the accumulator. Partial sums of such terms grow evenly: (64 + 1) / 2 of
    the part's in all. Fourteen parts, a cluster's shares and the output rule
    round to nearest, 20 additions at most. 5 % for the uneven growth.
    """
    rng = np.random.default_rng(K + N)
    codes = rng.integers(1, 8, (N, K))
    scales = np.full((N, ref.blocks(K, fmt)), {"mxfp4": 127, "nvfp4": 0x38}[fmt], np.uint8)
    B = tgemm.mx4_pack(torch.from_numpy(ref.pack_codes(codes)).cuda(), torch.from_numpy(scales).cuda(), fmt, cols=K)
    A = torch.from_numpy(rng.uniform(0.5, 1.5, (M, K))).to(torch.bfloat16)
    want = A.double().numpy() @ ref.values(codes, scales, fmt).T
    got = tgemm.gemm_w4(A.cuda(), B).double().cpu().numpy()
    rel = np.abs(got / want - 1.0).max()
    assert rel <= 1.05 * (2 * 2.0 ** -23 * (64 + 1) / 2 + 20 * 2.0 ** -24), rel


@pytest.mark.parametrize("M,N,K", [(16, 4096, 14336), (128, 2000, 14336), (300, 4096, 14336)])
def test_long_sums_are_as_exact_as_fp32(tgemm, M, N, K):
    """Terms of both signs, against the result's norm.

    A step of an MMA cuts off 2^-24 of the partial sum on average. Partial sums
    of such terms grow as the root of their number: 2/3 of a part's end on
    average over its 64 steps, and the parts' errors add up as the parts do.
    """
    A, B, a, b = operands(tgemm, "w4", M, N, K, "nvfp4", "normal")
    got = tgemm.gemm_w4(A, B).double().cpu().numpy()
    want = a @ b.T
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel <= 64 * (2 / 3) * 2.0 ** -24, rel


@pytest.mark.parametrize("tiles", [2, 16, 25, 30, 40, 70])      # shared by 8, 6, 5, 4, 3 and 2 blocks each on 152 SMs
@pytest.mark.parametrize("op", OPS)
def test_tiles_shared_by_clusters_of_each_size(tgemm, op, tiles):
    M, N, K = 26, 128 * tiles - 5, 5300
    A, B, a, b = operands(tgemm, op, M, N, K, FMTS[tiles % 4 // 2], "wide")
    store, out = guarded(M, N, torch.float32, 3)
    call(tgemm, op)(A, B, out=out)
    err = np.abs(out.double().cpu().numpy() - a @ b.T)
    assert (err <= F32_REL * (np.abs(a) @ np.abs(b).T)).all()
    assert untouched(store, M, N) and tgemm.device_status() == 0


@pytest.mark.parametrize("M", [9, 16, 24])
@pytest.mark.parametrize("fmt", FMTS)
def test_few_rows_of_much_weight(tgemm, fmt, M):
    N, K = 4100, 4130
    A, B, a, b = operands(tgemm, "w4", M, N, K, fmt, "wide")
    store, out = guarded(M, N, torch.float32, 1)
    call(tgemm, "w4")(A, B, out=out)
    err = np.abs(out.double().cpu().numpy() - a @ b.T)
    assert (err <= F32_REL * (np.abs(a) @ np.abs(b).T)).all()
    assert untouched(store, M, N) and tgemm.device_status() == 0


@pytest.mark.parametrize("M", [1, 40, 200, 600])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("op", OPS)
def test_nan_and_infinity_stay_in_their_rows_and_columns(tgemm, op, fmt, M):
    N, K = 70, 300
    rng = np.random.default_rng(1)
    W = torch.from_numpy(rng.standard_normal((N, K))).float().cuda()
    W[11, 299] = float("inf")
    X = torch.from_numpy(rng.standard_normal((M, K))).to(torch.bfloat16).cuda()
    X[M - 1, 5] = float("nan")
    B = tgemm.mx4_quantize(W, fmt)
    A = tgemm.mx4_quantize(X, fmt) if op == "mx4" else X
    nan = torch.isnan(call(tgemm, op)(A, B)).cpu()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[:, 11] = True
    want[M - 1] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("op", OPS)
def test_smallest_and_largest_scales(tgemm, op, fmt):
    """Every scale byte of a format on one side, 1 on the other."""
    bytes_ = np.arange(255 if fmt == "mxfp4" else 127)
    N, K = len(bytes_), ref.BLOCK[fmt]
    codes = np.full((N, K), 2)                                          # 1.0
    B = tgemm.mx4_pack(torch.from_numpy(ref.pack_codes(codes)).cuda(),
                       torch.from_numpy(bytes_[:, None].astype(np.uint8)).cuda(), fmt, cols=K)
    one = torch.zeros(1, K)
    one[0, 0] = 4.0 if fmt == "mxfp4" else 6.0         # with block scale 1
    A = tgemm.mx4_quantize(one.cuda(), fmt, **({"tensor_scale": torch.ones(1, device="cuda")} if fmt == "nvfp4" else {}))
    if op == "w4":
        A = one.bfloat16().cuda()
    C = call(tgemm, op)(A, B).double().cpu().numpy()[0]
    want = ref.scale_value(bytes_, fmt) * float(one[0, 0])
    fine = (np.abs(want) < 2.0 ** 128) & ((np.abs(want) >= 2.0 ** -126) | (want == 0))
    assert np.array_equal(C[fine], want[fine])


@pytest.mark.parametrize("op", OPS)
def test_products_over_nothing(tgemm, op):
    for M, N in ((0, 5), (5, 0), (3, 4)):
        K = 0 if M and N else 32
        A, B, _, _ = operands(tgemm, op, M, N, K, "mxfp4", "whole")
        bias = torch.arange(N, dtype=torch.float32, device="cuda")
        assert torch.equal(call(tgemm, op)(A, B, bias=bias), bias.expand(M, N))
    out = torch.ones(3, 4, device="cuda")
    call(tgemm, op)(A, B, beta=0.5, out=out)
    assert (out == 0.5).all()


@pytest.mark.parametrize("op", OPS)
def test_c_is_not_read_when_beta_is_zero(tgemm, op):
    A, B, a, b = operands(tgemm, op, 50, 60, 64, "mxfp4", "whole")
    out = torch.full((50, 60), float("nan"), device="cuda")
    call(tgemm, op)(A, B, out=out)
    assert np.array_equal(out.double().cpu().numpy(), a @ b.T)


@pytest.mark.parametrize("M", [3, 700])
@pytest.mark.parametrize("op", OPS)
def test_the_same_call_gives_the_same_bits(tgemm, op, M):
    A, B, _, _ = operands(tgemm, op, M, 1500, 4096, "nvfp4", "wide", 0.1)
    first = call(tgemm, op)(A, B)
    for _ in range(4):
        assert torch.equal(call(tgemm, op)(A, B), first)


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("op", OPS)
def test_on_another_stream_and_in_a_graph(tgemm, op, M):
    A, B, a, b = operands(tgemm, op, M, 700, 512, "mxfp4", "whole")
    want = torch.from_numpy(a @ b.T).float().cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(tgemm, op)(A, B, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(tgemm, op)(A, B)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("M", [20, 300])
def test_rows_off_16_bytes_in_a_graph(tgemm, M):
    """With many rows such an A is copied to scratch first."""
    N, K = 500, 321
    X, x = activations(M, K, "whole", 3, ld=K + 2)
    B = Operand(tgemm, N, K, "nvfp4", "whole", 4)
    want = torch.from_numpy(x @ B.v.T).float().cuda()
    assert torch.equal(tgemm.gemm_w4(X, B.q), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tgemm.gemm_w4(X, B.q)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("M", [5, 40, 2100])
@pytest.mark.parametrize("op", OPS)
def test_the_first_cuda_call_of_a_thread(tgemm, op, M):
    """A thread whose first work on the device is a call of this library, as
    the one that runs backward passes."""
    A, B, a, b = operands(tgemm, op, M, 2600, 64, "mxfp4", "whole")
    X = torch.zeros(M, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(M, 2600, device="cuda")
    torch.cuda.synchronize()
    failed = []

    def work(f):
        try:
            f()
        except Exception as e:               # noqa: BLE001 - reported below
            failed.append(e)

    for f in (lambda: call(tgemm, op)(A, B, out=out), lambda: tgemm.mx4_quantize_both(X)):
        t = threading.Thread(target=work, args=(f,))
        t.start()
        t.join()
    assert not failed
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), a @ b.T)


@pytest.mark.parametrize("op", OPS)
def test_more_than_two_to_the_31_outputs(tgemm, op):
    M, N, K = 70001, 32768, 32                # C is 4.6 GB of BF16
    A, B, a, b = operands(tgemm, op, M, N, K, "mxfp4", "whole")
    C = call(tgemm, op)(A, B, out_dtype=torch.bfloat16)
    rows = [0, 1, 255, 32767, 65535, 65536, 69999, 70000]
    want = torch.from_numpy(a[rows] @ b.T).float().bfloat16()
    assert torch.equal(C[rows].cpu(), want)


def test_binding_refusals(tgemm):
    A, B, _, _ = operands(tgemm, "mx4", 4, 5, 64, "mxfp4", "whole")
    X = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    odd, nv = Operand(tgemm, 5, 63, "mxfp4", "whole", 1).q, Operand(tgemm, 5, 64, "nvfp4", "whole", 1).q
    for bad in (lambda: tgemm.gemm_mx4(A, odd), lambda: tgemm.gemm_mx4(A, nv), lambda: tgemm.gemm_w4(X, odd),
                lambda: tgemm.gemm_mx4(A, B, beta=1.0), lambda: tgemm.gemm_w4(X.t(), B),
                lambda: tgemm.gemm_w4(X[:1].expand(4, 64), B),
                lambda: tgemm.gemm_mx4(A, B, out=torch.empty(5, 4, device="cuda")),
                lambda: tgemm.gemm_mx4(A, B, bias=torch.zeros(4, device="cuda")),
                lambda: tgemm.gemm_w4(X, B, bias=torch.zeros(5))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: tgemm.gemm_w4(X.float(), B), lambda: tgemm.gemm_mx4(A, X),
                lambda: tgemm.gemm_mx4(A, B, out_dtype=torch.float16),
                lambda: tgemm.gemm_w4(X, B, out=torch.empty(4, 5, dtype=torch.float64, device="cuda"))):
        with pytest.raises(TypeError):
            bad()
