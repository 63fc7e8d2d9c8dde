"""The C ABI and the binding of the 4-bit operators on the host (no GPU), and
the 64-bit reference of their tests against the formats' definitions."""
import os
import re

import numpy as np
import pytest
import torch

import mx4_reference as ref
import tiled_matrix_multiplication_sm_gb300 as tg
from tiled_matrix_multiplication_sm_gb300 import mx4

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "tgemm_mx4.h")
FAKE = 0x10000           # never dereferenced: every call below is rejected first
MX, NV, F32, BF16 = 1, 2, 0, 1
INVALID, ALIGNMENT = 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tg.library_path()):
        from tiled_matrix_multiplication_sm_gb300 import build
        build.build()
    return mx4.load()


def test_header_and_binding_declare_the_same_symbols(lib):
    with open(HEADER) as f:
        names = set(re.findall(r"^TGEMM_API\s+[\w\s\*]*?\b(\w+)\s*\(", f.read(), re.M))
    assert names == set(mx4._SIGNATURES)
    for name in names:
        assert hasattr(lib, name)


MOST = 2147482624


@pytest.mark.parametrize("where", ["rows", "cols"])
def test_sizes_past_the_largest_are_refused(lib, where):
    r, c = (MOST + 1, 1) if where == "rows" else (1, MOST + 1)
    ld = max(c, 64)
    assert lib.gemm_mx4_codes_pitch(MOST + 1) == -INVALID
    assert lib.gemm_mx4_codes_pitch(MOST) == MOST // 2
    assert lib.gemm_mx4_scales_bytes(r, c, MX) == -INVALID
    assert lib.gemm_mx4_tensor_scale(r, c, FAKE, ld, F32, FAKE, 0) == INVALID
    assert lib.gemm_mx4_quantize(r, c, FAKE, ld, F32, MX, 0, 0, FAKE, FAKE, 0, 0, 0) == INVALID
    assert lib.gemm_mx4_dequantize(r, c, FAKE, FAKE, MX, 0, FAKE, ld, F32, 0) == INVALID
    assert lib.gemm_mx4_pack(r, c, MX, FAKE, ld, FAKE, ld, FAKE, FAKE, 0) == INVALID
    for M, N, K in ((MOST + 1, 1, 1), (1, MOST + 1, 1), (1, 1, MOST + 1)):
        out = (MX, FAKE, 2 ** 31, F32, 1.0, 0.0, 0, 0)
        assert lib.gemm_mx4(M, N, K, FAKE, FAKE, 0, FAKE, FAKE, 0, *out) == INVALID
        assert lib.gemm_w4(M, N, K, FAKE, 2 ** 31, FAKE, FAKE, 0, *out) == INVALID


@pytest.mark.parametrize("cols,pitch", [(0, 0), (1, 16), (32, 16), (33, 32), (4096, 2048), (-1, -INVALID)])
def test_codes_pitch(lib, cols, pitch):
    assert lib.gemm_mx4_codes_pitch(cols) == pitch


@pytest.mark.parametrize("rows,cols,fmt,size", [
    (1, 1, MX, 1024), (1, 1, NV, 2048), (128, 256, MX, 1024), (129, 256, NV, 4096), (128, 257, MX, 2048),
    (0, 5, MX, 0), (5, 0, NV, 0), (1 << 20, 1 << 20, NV, 1 << 36),
    (-1, 4, MX, -INVALID), (4, -1, MX, -INVALID), (4, 4, 0, -INVALID), (4, 4, 3, -INVALID)])
def test_scales_bytes(lib, rows, cols, fmt, size):
    assert lib.gemm_mx4_scales_bytes(rows, cols, fmt) == size


@pytest.mark.parametrize("rows,cols", [(0, 0), (1, 1), (127, 31), (128, 32), (129, 33), (3000, 1537), (5, 4096), (1 << 17, 257)])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_the_binding_allocates_what_the_library_asks_for(lib, fmt, rows, cols):
    assert mx4._sizes(rows, cols, fmt) == (rows * lib.gemm_mx4_codes_pitch(cols),
                                           lib.gemm_mx4_scales_bytes(rows, cols, mx4._FORMATS[fmt]))


@pytest.mark.parametrize("args,status", [
    ((-1, 4, FAKE, 4, F32, FAKE, 0), INVALID), ((4, -1, FAKE, 4, F32, FAKE, 0), INVALID),
    ((4, 4, FAKE, 3, F32, FAKE, 0), INVALID), ((4, 4, 0, 4, F32, FAKE, 0), INVALID),
    ((4, 4, FAKE + 2, 4, F32, FAKE, 0), INVALID), ((4, 4, FAKE + 1, 4, BF16, FAKE, 0), INVALID),
    ((4, 4, FAKE, 4, 2, FAKE, 0), INVALID), ((4, 4, FAKE, 4, F32, 0, 0), INVALID),
    ((4, 4, FAKE, 4, F32, FAKE + 2, 0), INVALID)])
def test_tensor_scale_refuses(lib, args, status):
    assert lib.gemm_mx4_tensor_scale(*args) == status


@pytest.mark.parametrize("change,status", [
    ({"rows": -1}, INVALID), ({"cols": -1}, INVALID), ({"ldx": 3}, INVALID), ({"X": 0}, INVALID),
    ({"X": FAKE + 1}, INVALID), ({"type": 7}, INVALID), ({"fmt": 0}, INVALID), ({"g": FAKE}, INVALID),
    ({"fmt": NV, "g": FAKE + 1}, INVALID), ({"codes": 0}, INVALID), ({"scales": 0}, INVALID),
    ({"flags": 1}, INVALID), ({"fmt": NV, "g": FAKE, "flags": 2}, INVALID), ({"fmt": NV, "flags": 1}, INVALID),
    ({"codes_t": FAKE}, INVALID), ({"codes": 0, "scales": 0}, INVALID),
    ({"codes": FAKE + 8}, ALIGNMENT), ({"scales": FAKE + 1}, ALIGNMENT),
    ({"codes_t": FAKE + 8, "scales_t": FAKE}, ALIGNMENT)])
def test_quantize_refuses(lib, change, status):
    a = {"rows": 4, "cols": 4, "X": FAKE, "ldx": 4, "type": F32, "fmt": MX, "g": 0, "flags": 0, "codes": FAKE,
         "scales": FAKE, "codes_t": 0, "scales_t": 0, "stream": 0, **change}
    assert lib.gemm_mx4_quantize(*a.values()) == status


@pytest.mark.parametrize("change,status", [
    ({"rows": -1}, INVALID), ({"cols": -1}, INVALID), ({"ldx": 3}, INVALID), ({"X": 0}, INVALID),
    ({"type": -1}, INVALID), ({"fmt": 9}, INVALID), ({"g": FAKE}, INVALID), ({"codes": 0}, INVALID),
    ({"scales": 0}, INVALID), ({"codes": FAKE + 4}, ALIGNMENT), ({"scales": FAKE + 8}, ALIGNMENT)])
def test_dequantize_refuses(lib, change, status):
    a = {"rows": 4, "cols": 4, "codes": FAKE, "scales": FAKE, "fmt": MX, "g": 0, "X": FAKE, "ldx": 4,
         "type": BF16, "stream": 0, **change}
    assert lib.gemm_mx4_dequantize(*a.values()) == status


@pytest.mark.parametrize("change,status", [
    ({"rows": -1}, INVALID), ({"cols": -1}, INVALID), ({"fmt": 0}, INVALID), ({"ldc": 19}, INVALID),
    ({"lds": 1}, INVALID), ({"src": 0}, INVALID), ({"src_s": 0}, INVALID), ({"codes": 0}, INVALID),
    ({"codes": FAKE + 1}, ALIGNMENT), ({"scales": FAKE + 4}, ALIGNMENT)])
def test_pack_refuses(lib, change, status):
    a = {"rows": 4, "cols": 40, "fmt": MX, "src": FAKE, "ldc": 20, "src_s": FAKE, "lds": 2, "codes": FAKE,
         "scales": FAKE, "stream": 0, **change}
    assert lib.gemm_mx4_pack(*a.values()) == status


OUT = {"fmt": MX, "C": FAKE, "ldc": 4, "type": F32, "alpha": 1.0, "beta": 0.0, "bias": 0, "stream": 0}
PRODUCT_REFUSALS = [
    ({"M": -1}, INVALID), ({"N": -1}, INVALID), ({"K": -1}, INVALID), ({"fmt": 5}, INVALID),
    ({"type": 2}, INVALID), ({"ldc": 3}, INVALID), ({"C": 0}, INVALID), ({"C": FAKE + 2}, INVALID),
    ({"type": BF16, "C": FAKE + 1}, INVALID), ({"bias": FAKE + 2}, INVALID), ({"gb": FAKE}, INVALID),
    ({"fmt": NV, "gb": FAKE + 2}, INVALID), ({"b": 0}, INVALID), ({"bs": 0}, INVALID),
    ({"b": FAKE + 8}, ALIGNMENT), ({"bs": FAKE + 8}, ALIGNMENT)]


@pytest.mark.parametrize("change,status", PRODUCT_REFUSALS + [
    ({"a": 0}, INVALID), ({"as": 0}, INVALID), ({"ga": FAKE}, INVALID), ({"a": FAKE + 4}, ALIGNMENT),
    ({"as": FAKE + 1}, ALIGNMENT)])
def test_gemm_mx4_refuses(lib, change, status):
    a = {"M": 4, "N": 4, "K": 64, "a": FAKE, "as": FAKE, "ga": 0, "b": FAKE, "bs": FAKE, "gb": 0, **OUT, **change}
    assert lib.gemm_mx4(*a.values()) == status


@pytest.mark.parametrize("change,status", PRODUCT_REFUSALS + [
    ({"A": 0}, INVALID), ({"A": FAKE + 1}, INVALID), ({"lda": 63}, INVALID)])
def test_gemm_w4_refuses(lib, change, status):
    a = {"M": 4, "N": 4, "K": 64, "A": FAKE, "lda": 64, "b": FAKE, "bs": FAKE, "gb": 0, **OUT, **change}
    assert lib.gemm_w4(*a.values()) == status


def test_empty_outputs_are_accepted_without_a_device(lib):
    for M, N in ((0, 4), (4, 0)):
        a = {"M": M, "N": N, "K": 64, "a": 0, "as": 0, "ga": 0, "b": 0, "bs": 0, "gb": 0, **OUT, "C": 0}
        assert lib.gemm_mx4(*a.values()) == 0
        a = {"M": M, "N": N, "K": 64, "A": 0, "lda": 64, "b": 0, "bs": 0, "gb": 0, **OUT, "C": 0}
        assert lib.gemm_w4(*a.values()) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    X = torch.zeros(4, 32)
    with pytest.raises(ValueError):
        tg.mx4_quantize(X)
    with pytest.raises(ValueError):
        tg.mx4_quantize(X, "fp4")
    with pytest.raises(TypeError):
        tg.mx4_quantize([1.0])
    with pytest.raises(TypeError):
        tg.mx4_dequantize(X)
    with pytest.raises(TypeError):
        tg.gemm_mx4(X, X)
    with pytest.raises(TypeError):
        tg.gemm_w4(X, X)
    with pytest.raises(ValueError):
        tg.Mx4Matrix("mxfp4", 4, 32, torch.zeros(64, dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8))


# ------------------------------------------------ the reference of the GPU tests

def test_reference_codes_round_to_the_nearest_value():
    v = np.linspace(-8, 8, 4001)
    got = ref.e2m1(ref.round_e2m1(v))
    both = np.concatenate([-ref.E2M1[::-1], ref.E2M1])
    assert np.array_equal(np.abs(got - v), np.abs(both[None] - v[:, None]).min(axis=1))
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0]
    assert ref.e2m1(ref.round_e2m1(np.array(ties))).tolist() == [0, 1, 1, 2, 2, 4, 4, -4]


def test_reference_scales_match_torch_e4m3():
    b = torch.arange(127, dtype=torch.uint8)
    want = b.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.scale_value(b.numpy(), "nvfp4"), want)
    v = np.concatenate([want, (want[1:] + want[:-1]) / 2, np.random.default_rng(0).uniform(0, 460, 2000)])
    v = np.minimum(v, 448.0)
    assert np.array_equal(ref.round_e4m3(v), torch.tensor(v).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_reference_worked_block():
    x = np.zeros((1, 32))
    x[0, :4] = [7.0, -1.3, 0.4, 0.2]          # largest 7: scale 2^(2 - 2) = 1; 7 is above 6
    codes, scales = ref.quantize(x, "mxfp4")
    assert scales.tolist() == [[127]]
    assert ref.values(codes, scales, "mxfp4")[0, :4].tolist() == [6.0, -1.5, 0.5, 0.0]
    x[0, 0] = 2688.0
    g = ref.tensor_scale(x)
    assert g == 1.0
    codes, scales = ref.quantize(x, "nvfp4", g)
    assert scales.tolist() == [[0x7E, 0]] and ref.values(codes, scales, "nvfp4", g)[0, 0] == 2688.0
