"""The C ABI and the binding of the fused products on the host (no GPU), and the
64-bit reference of their tests."""
import os
import re

import pytest
import torch

import fused_reference as ref
import tiled_matrix_multiplication_sm_gb300 as tg
from tiled_matrix_multiplication_sm_gb300 import fused

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "tgemm_fused.h")
FAKE = 0x10000           # never dereferenced: every call below is rejected first
F32, BF16 = 0, 1
INVALID = 1
MOST = 1073741312


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tg.library_path()):
        from tiled_matrix_multiplication_sm_gb300 import build
        build.build()
    return fused.load()


def test_header_and_binding_declare_the_same_symbols(lib):
    with open(HEADER) as f:
        text = f.read()
    names = set(re.findall(r"^TGEMM_API\s+[\w\s\*]*?\b(\w+)\s*\(", text, re.M))
    assert names == set(fused._SIGNATURES)
    for name in names:
        assert hasattr(lib, name)
    assert int(re.search(r"TGEMM_FUSED_MAX_DIM (\d+)", text)[1]) == MOST
    for act, code in fused._ACTIVATIONS.items():
        assert int(re.search(rf"TGEMM_ACT_{act.upper()} +(\d+)", text)[1]) == code


SIZES = {"M": 4, "N": 4, "K": 8, "A": FAKE, "lda": 8, "B": FAKE, "ldb": 4, "flags": 0, "act": 1}
ACT = {**SIZES, "bias": 0, "R": 0, "ldr": 0, "r_type": 0, "Z": 0, "ldz": 0, "C": FAKE, "ldc": 4, "c_type": BF16, "stream": 0}
OPERANDS = [{"M": -1}, {"N": -1}, {"K": -1}, {"M": MOST + 1}, {"N": MOST + 1, "ldb": 2 ** 31}, {"K": MOST + 1, "lda": 2 ** 31},
            {"A": 0}, {"B": 0}, {"A": FAKE + 1}, {"B": FAKE + 1}, {"lda": 7}, {"ldb": 3}, {"flags": 8}, {"act": 5}, {"act": -1},
            {"M": 9, "flags": 1, "lda": 8}, {"flags": 2, "ldb": 7}]


@pytest.mark.parametrize("change", OPERANDS + [
    {"bias": FAKE + 2}, {"C": 0}, {"C": FAKE + 1}, {"ldc": 3}, {"c_type": 2}, {"c_type": F32, "C": FAKE + 2},
    {"R": FAKE + 0x1000, "ldr": 3, "r_type": BF16}, {"R": FAKE + 0x1001, "ldr": 4, "r_type": BF16},
    {"R": FAKE + 0x1002, "ldr": 4, "r_type": F32}, {"R": FAKE + 0x1000, "ldr": 4, "r_type": 3},
    {"R": FAKE, "ldr": 5, "r_type": BF16}, {"R": FAKE, "ldr": 4, "r_type": F32},
    {"Z": FAKE + 0x1000, "ldz": 3}, {"Z": FAKE + 0x1001, "ldz": 4},
    {"flags": 4, "ldb": 7}, {"flags": 4, "ldb": 8, "c_type": F32}, {"flags": 4, "ldb": 8, "Z": FAKE + 0x1000, "ldz": 7}])
def test_gemm_act_refuses(lib, change):
    assert lib.gemm_act(*{**ACT, **change}.values()) == INVALID


GRAD = {**SIZES, "Z": FAKE + 0x1000, "ldz": 4, "dZ": FAKE + 0x2000, "lddz": 4, "dz_type": BF16, "db": 0, "stream": 0}


@pytest.mark.parametrize("change", OPERANDS + [
    {"Z": 0}, {"Z": FAKE + 1}, {"ldz": 3}, {"dZ": 0}, {"dZ": FAKE + 1}, {"lddz": 3}, {"dz_type": 2}, {"db": FAKE + 2},
    {"dZ": FAKE + 0x1000, "lddz": 5}, {"dZ": FAKE + 0x1000, "dz_type": F32},
    {"flags": 4}, {"flags": 4, "ldz": 8, "lddz": 7}, {"flags": 4, "ldz": 7, "lddz": 8},
    {"flags": 4, "ldz": 8, "lddz": 8, "dz_type": F32}])
def test_gemm_act_grad_refuses(lib, change):
    assert lib.gemm_act_grad(*{**GRAD, **change}.values()) == INVALID


CE = {"T": 4, "V": 4, "D": 8, "X": FAKE, "ldx": 8, "W": FAKE, "ldw": 8, "alpha": 1.0, "target": FAKE}
HEAD = [{"T": -1}, {"V": -1}, {"D": -1}, {"T": MOST + 1}, {"V": MOST + 1}, {"D": MOST + 1, "ldx": 2 ** 31, "ldw": 2 ** 31},
        {"X": 0}, {"W": 0}, {"X": FAKE + 1}, {"W": FAKE + 1}, {"ldx": 7}, {"ldw": 7}, {"alpha": float("inf")},
        {"alpha": float("nan")}, {"target": 0}, {"target": FAKE + 4}]


@pytest.mark.parametrize("change", HEAD + [{"loss": 0}, {"lse": 0}, {"loss": FAKE + 2}, {"lse": FAKE + 2}])
def test_gemm_ce_refuses(lib, change):
    assert lib.gemm_ce(*{**CE, "loss": FAKE, "lse": FAKE, "stream": 0, **change}.values()) == INVALID


CE_GRAD = {**CE, "lse": FAKE, "dloss": FAKE, "dX": FAKE, "lddx": 8, "dx_type": BF16, "dW": FAKE, "lddw": 8, "dw_type": F32,
           "beta": 0.0, "stream": 0}


@pytest.mark.parametrize("change", HEAD + [
    {"lse": 0}, {"dloss": 0}, {"lse": FAKE + 2}, {"dloss": FAKE + 1}, {"lddx": 7}, {"lddw": 7}, {"dx_type": 2}, {"dw_type": -1},
    {"dX": FAKE + 1}, {"dW": FAKE + 2}, {"beta": float("inf")}, {"beta": float("nan")}])
def test_gemm_ce_grad_refuses(lib, change):
    assert lib.gemm_ce_grad(*{**CE_GRAD, **change}.values()) == INVALID


def test_the_kernel_setter_validates(lib):
    for mode in (-2, 2):
        assert fused.set_fused_kernel(mode) == INVALID
    assert fused.set_fused_kernel(0) == 0 and fused.set_fused_kernel(-1) == 0


def test_empty_results_are_accepted_without_a_device(lib):
    for M, N in ((0, 4), (4, 0)):
        assert lib.gemm_act(*{**ACT, "M": M, "N": N, "A": 0, "B": 0, "C": 0}.values()) == 0
        assert lib.gemm_act_grad(*{**GRAD, "M": M, "N": N, "A": 0, "B": 0, "Z": 0, "dZ": 0}.values()) == 0
    assert lib.gemm_ce(*{**CE, "T": 0, "X": 0, "target": 0, "loss": 0, "lse": 0, "stream": 0}.values()) == 0
    assert lib.gemm_ce_grad(*{**CE_GRAD, "dX": 0, "dW": 0}.values()) == 0
    assert lib.gemm_ce_grad(*{**CE_GRAD, "D": 0}.values()) == 0
    assert lib.gemm_ce_grad(*{**CE_GRAD, "T": 0, "dW": 0, "X": 0, "target": 0, "lse": 0, "dloss": 0}.values()) == 0


def test_binding_refuses():
    X = torch.zeros(4, 8, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        tg.gemm_act(X, X, trans_b=True)                   # a host tensor
    with pytest.raises(ValueError):
        tg.gemm_act(X, X, "swish")
    with pytest.raises(TypeError):
        tg.gemm_act([1.0], X)
    with pytest.raises(ValueError):
        tg.gemm_act_grad(X, X, X)
    with pytest.raises(ValueError):
        tg.gemm_ce(X, X, t)
    with pytest.raises(ValueError):
        tg.gemm_ce_grad(X, X, t, t.float(), t.float())


# ------------------------------------------------ the reference of the GPU tests

@pytest.mark.parametrize("name", ref.ACTS)
def test_reference_slopes_are_differences(name):
    z = torch.linspace(-6, 6, 1001, dtype=torch.float64)
    z = z[z.abs() > 1e-3]
    h = 1e-5
    d = (ref.act(name, z + h)[0] - ref.act(name, z - h)[0]) / (2 * h)
    assert (ref.act(name, z)[1] - d).abs().max() < 1e-9
    plain = {"none": z, "relu": torch.relu(z), "gelu": torch.nn.functional.gelu(z), "silu": torch.nn.functional.silu(z),
             "gelu_tanh": torch.nn.functional.gelu(z, approximate="tanh")}[name]
    assert torch.allclose(ref.act(name, z)[0], plain, rtol=1e-12, atol=1e-14)


def test_reference_cross_entropy_is_torchs():
    g = torch.Generator().manual_seed(1)
    x, w = (torch.randn(s, 8, generator=g, dtype=torch.float64).requires_grad_() for s in (20, 30))
    target = torch.randint(0, 30, (20,), generator=g)
    target[::5] = -100
    dloss = torch.rand(20, generator=g, dtype=torch.float64)
    loss = torch.nn.functional.cross_entropy(0.7 * x @ w.t(), target, ignore_index=-100, reduction="none")
    (loss * dloss).sum().backward()
    got, lse, z, _ = ref.ce(x.detach(), w.detach(), target, 0.7)
    assert torch.allclose(got, loss.detach())
    dx, dw, *_ = ref.ce_grad(x.detach(), w.detach(), target, lse, dloss, 0.7)
    assert torch.allclose(dx, x.grad) and torch.allclose(dw, w.grad)
