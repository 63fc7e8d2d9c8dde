"""Quantising to 4 bits, reading back and packing against the 64-bit reference.

Inputs have at most 16 significant bits, so that a quotient x / scale either
is a midpoint of two codes exactly or lies at least 2^-17 of itself away from
one: the kernel's FP32 quotients then decide as 64 bits do, and codes, scales
and values have to be equal.
"""
import numpy as np
import pytest
import torch

import mx4_reference as ref

pytestmark = pytest.mark.gpu
FMTS = ["mxfp4", "nvfp4"]
TYPES = [torch.float32, torch.bfloat16]
SIZES = [(1, 1), (1, 16), (1, 32), (2, 15), (3, 17), (5, 31), (33, 33), (31, 64), (127, 255), (128, 256),
         (130, 257), (200, 513), (7, 4096), (1537, 40), (64, 1024)]


def draw(R, C, dtype, seed, ld=None):
    """16 significant bits at most, magnitudes over 2^-20 .. 2^3; NaN between C and ld."""
    rng = np.random.default_rng(seed)
    x = np.round(rng.standard_normal((R, C)) * 2.0 ** 12) * 2.0 ** (rng.integers(-8, 1, (R, 1)) - 12.0)
    x[rng.random((R, C)) < 0.02] = 0.0
    X = torch.full((R, ld or C), float("nan"), dtype=dtype)
    X[:, :C] = torch.from_numpy(x).to(dtype)
    return X.cuda()[:, :C]


def host(X):
    return X.double().cpu().numpy()


def check(tg, q, X, fmt, g):
    """q is X's quantised form, bit for bit (a zero's sign aside)."""
    codes, scales = ref.unpack(q)
    want_codes, want_scales = ref.quantize(X, fmt, g)
    assert np.array_equal(scales, want_scales)
    want = ref.values(want_codes, want_scales, fmt, g)
    assert np.array_equal(ref.values(codes, scales, fmt, g), want, equal_nan=True)
    for dtype in TYPES:        # code x scale has 6 significant bits, g is a power of two here
        got = host(tg.mx4_dequantize(q, dtype))
        assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,C", SIZES)
def test_rows_trans_and_both(tgemm, fmt, dtype, R, C):
    X = draw(R, C, dtype, R * 10007 + C, ld=C + (R % 3) * 5)
    g = ref.tensor_scale(host(X)) if fmt == "nvfp4" else 1.0
    if fmt == "nvfp4":
        assert tgemm.mx4_tensor_scale(X).item() == g
    check(tgemm, tgemm.mx4_quantize(X, fmt), host(X), fmt, g)
    check(tgemm, tgemm.mx4_quantize(X, fmt, trans=True), host(X).T, fmt, g)
    q, t = tgemm.mx4_quantize_both(X, fmt)
    check(tgemm, q, host(X), fmt, g)
    check(tgemm, t, host(X).T, fmt, g)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
def test_every_alignment_of_the_first_element(tgemm, fmt, dtype):
    store = draw(1, 40 * 300, dtype, 3)[0]
    for offset in range(9):
        X = store[offset:offset + 37 * 289].view(37, 289)[:, :281]
        g = ref.tensor_scale(host(X)) if fmt == "nvfp4" else 1.0
        q, t = tgemm.mx4_quantize_both(X, fmt)
        check(tgemm, q, host(X), fmt, g)
        check(tgemm, t, host(X).T, fmt, g)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
def test_extremes_of_the_number_range(tgemm, fmt, dtype):
    X = torch.zeros(12, 96, dtype=dtype, device="cuda")
    tiny = 2.0 ** -133 if dtype == torch.bfloat16 else 2.0 ** -149
    big = 2.0 ** 127
    for i, v in enumerate([tiny, 2.0 ** -127, 2.0 ** -126, 2.0 ** -125, 1.5 * 2.0 ** -124, 1e-3, 448.0, big]):
        X[i, i] = v
        X[i, 40] = -v / 2
    X[8, :] = -0.0
    X[9, 3] = 1.5 * big                         # all of a block within a factor two of the range's end
    X[9, 4] = -big / 4
    if fmt == "mxfp4":
        check(tgemm, tgemm.mx4_quantize(X, fmt), host(X), fmt, 1.0)
        check(tgemm, tgemm.mx4_quantize(X, fmt, trans=True), host(X).T, fmt, 1.0)
        return
    for rows in (slice(0, 6), slice(6, 7), slice(7, 12)):
        Y = X[rows]
        g = ref.tensor_scale(host(Y))
        assert tgemm.mx4_tensor_scale(Y).item() == g
        codes, scales = ref.unpack(tgemm.mx4_quantize(Y, fmt))
        want_codes, want_scales = ref.quantize(host(Y), fmt, g)
        assert np.array_equal(scales, want_scales)
        assert np.array_equal(ref.e2m1(codes), ref.e2m1(want_codes))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), float("-inf")])
def test_a_block_with_an_infinity_or_nan_reads_back_as_nan(tgemm, fmt, dtype, poison):
    X = draw(40, 100, dtype, 8)
    X[7, 50] = poison
    X[39, 99] = poison
    g = ref.tensor_scale(host(X)) if fmt == "nvfp4" else 1.0
    if fmt == "nvfp4":
        assert tgemm.mx4_tensor_scale(X).item() == g          # of the finite values
    q, t = tgemm.mx4_quantize_both(X, fmt)
    check(tgemm, q, host(X), fmt, g)
    check(tgemm, t, host(X).T, fmt, g)
    nan = np.isnan(host(tgemm.mx4_dequantize(q)))
    B = ref.BLOCK[fmt]
    assert nan[7, 50 // B * B:(50 // B + 1) * B].all() and nan.sum() == B + (100 - 99 // B * B)


def test_tensor_scale_of_zeros_and_of_nothing(tgemm):
    for X in (torch.zeros(5, 7, device="cuda"), torch.empty(0, 7, device="cuda"),
              torch.full((3, 3), float("nan"), device="cuda")):
        assert tgemm.mx4_tensor_scale(X).item() == 2.0 ** -100


@pytest.mark.parametrize("R,C", [(1, 8191), (1, 8193), (31, 260), (500, 20), (20, 70000)])
def test_tensor_scale_finds_the_largest_wherever_it_is(tgemm, R, C):
    X = torch.full((R, C), 0.001, device="cuda")
    for r, c in ((0, 0), (R - 1, C - 1), (R // 2, C // 3), (0, C - 1)):
        Y = X.clone()
        Y[r, c] = -4000.0
        assert tgemm.mx4_tensor_scale(Y).item() == 2.0
        assert tgemm.mx4_tensor_scale(Y.bfloat16()).item() == 2.0
        assert tgemm.mx4_quantize(Y, "nvfp4").tensor_scale.item() == 2.0


@pytest.mark.parametrize("value", [21.0, 21.000002, 20.999998, 2688.0, 2688.0002, 1e-30, 3e38, 1e-38])
def test_tensor_scale_at_the_steps_of_its_powers(tgemm, value):
    X = torch.tensor([[value, -value / 3]], device="cuda")
    assert tgemm.mx4_tensor_scale(X).item() == ref.tensor_scale(host(X))


@pytest.mark.parametrize("g", [3e-4, 1.0, 0.01])
def test_a_given_tensor_scale_is_used(tgemm, g):
    """Any positive g: the codes are within one step of the 64-bit ones, and
    values saturate at 2688 g."""
    X = draw(50, 200, torch.float32, 5)
    gt = torch.tensor([g], device="cuda")
    q = tgemm.mx4_quantize(X, "nvfp4", tensor_scale=gt)
    assert q.tensor_scale is gt
    codes, scales = ref.unpack(q)
    want_codes, want_scales = ref.quantize(host(X), "nvfp4", float(gt))
    # An FP32 quotient is off by 2^-24 of itself: only a quotient that close to
    # a midpoint may round otherwise.
    assert np.mean(scales != want_scales) < 1e-3 and np.mean(codes != want_codes) < 1e-3
    got = host(tgemm.mx4_dequantize(q))
    want = ref.values(codes, scales, "nvfp4", float(gt))
    assert np.allclose(got, want, rtol=2.0 ** -23, atol=0)


@pytest.mark.parametrize("g", [0.0, -1.0, float("nan"), float("inf"), 2.0 ** -101, 2.0 ** 118])
def test_an_unusable_tensor_scale_gives_nan(tgemm, g):
    q = tgemm.mx4_quantize(torch.ones(4, 40, device="cuda"), "nvfp4", tensor_scale=torch.tensor([g], device="cuda"))
    assert torch.isnan(tgemm.mx4_dequantize(q)).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,C", [(1, 1), (3, 33), (129, 250), (40, 512)])
def test_pack_and_every_code_and_scale_byte(tgemm, fmt, R, C):
    rng = np.random.default_rng(R + C)
    codes = rng.integers(0, 16, (R, C))
    scales = rng.integers(0, 256 if fmt == "mxfp4" else 128, (R, ref.blocks(C, fmt)))
    wide_c = torch.full((R, (C + 1) // 2 + 3), 255, dtype=torch.uint8)
    wide_c[:, :(C + 1) // 2] = torch.from_numpy(ref.pack_codes(codes))
    if C % 2:
        wide_c[:, C // 2] |= 0xF0                # a code past the last column
    wide_s = torch.full((R, scales.shape[1] + 1), 255, dtype=torch.uint8)
    wide_s[:, 1:] = torch.from_numpy(scales)
    g = torch.tensor([0.37], device="cuda") if fmt == "nvfp4" else None
    q = tgemm.mx4_pack(wide_c.cuda()[:, :(C + 1) // 2], wide_s.cuda()[:, 1:], fmt, cols=C, tensor_scale=g)
    got_codes, got_scales = ref.unpack(q)
    assert np.array_equal(got_codes, codes) and np.array_equal(got_scales, scales)
    want = (ref.values(codes, scales, fmt).astype(np.float32) * np.float32(1.0 if g is None else 0.37))
    assert np.array_equal(tgemm.mx4_dequantize(q).cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("fmt", FMTS)
def test_nothing_is_written_outside_the_buffers(tgemm, fmt):
    from tiled_matrix_multiplication_sm_gb300 import mx4
    lib = mx4.load()
    R, C = 130, 70
    code = mx4._FORMATS[fmt]
    X = draw(R, C, torch.bfloat16, 2)
    g = torch.ones(1, device="cuda")

    def guarded(n):
        t = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        return t, t.data_ptr() + 256, n

    bufs = [guarded(R * lib.gemm_mx4_codes_pitch(C)), guarded(lib.gemm_mx4_scales_bytes(R, C, code)),
            guarded(C * lib.gemm_mx4_codes_pitch(R)), guarded(lib.gemm_mx4_scales_bytes(C, R, code))]
    s = torch.cuda.current_stream().cuda_stream
    gp = g.data_ptr() if fmt == "nvfp4" else 0
    assert lib.gemm_mx4_quantize(R, C, X.data_ptr(), X.stride(0), 1, code, gp, 0, *(b[1] for b in bufs), s) == 0
    back = torch.full((R + 2, C + 5), 7.0, device="cuda")
    assert lib.gemm_mx4_dequantize(R, C, bufs[0][1], bufs[1][1], code, gp, back[1:].data_ptr(), C + 5, 0, s) == 0
    for t, _, n in bufs:
        assert (t[:256] == 0xA5).all() and (t[256 + n:] == 0xA5).all()
    assert (back[0] == 7).all() and (back[-1] == 7).all() and (back[:, C:] == 7).all()


def test_empty_matrices(tgemm):
    for shape in ((0, 32), (4, 0)):
        for fmt in FMTS:
            q, t = tgemm.mx4_quantize_both(torch.empty(shape, device="cuda"), fmt)
            assert q.shape == shape and t.shape == shape[::-1]
            assert tgemm.mx4_dequantize(q).shape == shape


def test_more_than_two_to_the_31_elements(tgemm):
    R, C = 70001, 32768                       # 2.29e9 elements of BF16, 4.6 GB
    X = torch.zeros(R, C, dtype=torch.bfloat16, device="cuda")
    X[-1] = draw(1, C, torch.bfloat16, 1)[0]
    X[R - 300:, -1] = draw(1, 300, torch.bfloat16, 2)[0]
    q, t = tgemm.mx4_quantize_both(X, "mxfp4")
    back = tgemm.mx4_dequantize(q, torch.bfloat16)
    want = ref.values(*ref.quantize(host(X[-1:]), "mxfp4"), "mxfp4")
    assert np.array_equal(host(back[-1:]), want)
    assert not back[:R - 300].any()
    del back
    last = tgemm.Mx4Matrix("mxfp4", 1, R, t.codes[(C - 1) * 16 * (-(-R // 32)):].contiguous(), t.scales)
    # Row C - 1 of the transpose is row 127 of its last scale tile.
    raw = last.codes.cpu().numpy()
    codes = np.stack((raw & 15, raw >> 4), axis=1).reshape(1, -1)[:, :R]
    want_codes, want_scales = ref.quantize(host(X[:, -1:]).T, "mxfp4")
    assert np.array_equal(ref.e2m1(codes), ref.e2m1(want_codes))
    tiles_k = -(-R // 256) * 2
    tile = t.scales.cpu().numpy().reshape(C // 128, tiles_k, 32, 4, 4)[-1, :, 31, 3, :].reshape(1, -1)
    assert np.array_equal(tile[:, :want_scales.shape[1]], want_scales)


@pytest.mark.parametrize("fmt", FMTS)
def test_on_another_stream_and_in_a_graph(tgemm, fmt):
    X = draw(100, 300, torch.bfloat16, 4)
    want = tgemm.mx4_dequantize(tgemm.mx4_quantize(X, fmt))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = tgemm.mx4_dequantize(tgemm.mx4_quantize(X, fmt, stream=s), stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tgemm.mx4_dequantize(tgemm.mx4_quantize(X, fmt))
    X.copy_(draw(100, 300, torch.bfloat16, 5))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, tgemm.mx4_dequantize(tgemm.mx4_quantize(X, fmt)))


def test_refusals(tgemm):
    X = torch.zeros(4, 64, device="cuda")
    g = torch.ones(1, device="cuda")
    for bad in (lambda: tgemm.mx4_quantize(X, "mxfp4", tensor_scale=g), lambda: tgemm.mx4_quantize(X.t()),
                lambda: tgemm.mx4_quantize(X[0]), lambda: tgemm.mx4_quantize(X[:1].expand(4, 64)),
                lambda: tgemm.mx4_quantize(X.view(-1).as_strided((4, 64), (32, 1))),
                lambda: tgemm.mx4_dequantize(tgemm.mx4_quantize(X), out=torch.empty(1, 64, device="cuda").expand(4, 64)),
                lambda: tgemm.mx4_dequantize(tgemm.mx4_quantize(X), out=torch.empty(4, 63, device="cuda")),
                lambda: tgemm.mx4_pack(torch.zeros(4, 3, dtype=torch.uint8, device="cuda"),
                                       torch.zeros(4, 1, dtype=torch.uint8, device="cuda"), cols=7),
                lambda: tgemm.mx4_quantize(X, "nvfp4", tensor_scale=torch.ones(1))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: tgemm.mx4_quantize(X.half()), lambda: tgemm.mx4_quantize(X, "nvfp4", tensor_scale=g.double()),
                lambda: tgemm.mx4_dequantize(tgemm.mx4_quantize(X), torch.float16)):
        with pytest.raises(TypeError):
            bad()
