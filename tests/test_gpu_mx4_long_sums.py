"""Long sums of the 4-bit products with an FP32 result, against 64 bits.

The bounds are those of test_gpu_mx4_product.py: an MMA of 16 columns cuts off
at most 2^-23 of the partial sum twice, a part has 1024 columns, 64 steps; the
parts, the warps' or blocks' shares and the output rule add with rounding to
nearest.
"""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from test_gpu_mx4_product import call, operands

pytestmark = pytest.mark.gpu

# (M, N, K): the whole sum in one block's eight warps, in one warp's share of many
# columns within clusters, with few rows of W, and with a last part cut short.
FEW_ROWS = [(1, 8192, 28672), (8, 8192, 28672), (3, 64, 300000), (16, 40, 400000), (24, 30, 500033), (8, 5000, 28700)]


@pytest.mark.parametrize("M,N,K", FEW_ROWS)
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_few_rows_keep_the_low_bits_of_positive_terms(tgemm, fmt, M, N, K):
    rng = np.random.default_rng(K + N)
    codes = rng.integers(1, 8, (N, K))
    scales = np.full((N, ref.blocks(K, fmt)), {"mxfp4": 127, "nvfp4": 0x38}[fmt], np.uint8)
    B = tgemm.mx4_pack(torch.from_numpy(ref.pack_codes(codes)).cuda(), torch.from_numpy(scales).cuda(), fmt, cols=K)
    A = torch.from_numpy(rng.uniform(0.5, 1.5, (M, K))).to(torch.bfloat16)
    want = A.double().numpy() @ ref.e2m1(codes).T
    got = tgemm.gemm_w4(A.cuda(), B).double().cpu().numpy()
    # Parts of a warp (at most 8 here), eight warps, eight blocks, the output rule.
    additions = max(8, -(-K // (8 * 1024))) + 8 + 8 + 4
    rel = np.abs(got / want - 1.0).max()
    assert rel <= 1.05 * (2 * 2.0 ** -23 * (64 + 1) / 2 + additions * 2.0 ** -24), rel


@pytest.mark.parametrize("M,N,K", FEW_ROWS)
def test_few_rows_are_as_exact_as_fp32(tgemm, M, N, K):
    A, B, a, b = operands(tgemm, "w4", M, N, K, "nvfp4", "normal")
    got = tgemm.gemm_w4(A, B).double().cpu().numpy()
    want = a @ b.T
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel <= 64 * (2 / 3) * 2.0 ** -24, rel


# ------------------------------------------------- products of two 4-bit matrices

def matrix(tgemm, R, K, fmt, positive, octaves, seed):
    """A matrix on the device and its values in 64 bits, there too."""
    rng = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(1 if positive else 0, 8 if positive else 16, (R, K + K % 2), generator=rng, device="cuda").byte()
    codes[:, K:] = 0
    lo, hi = {("mxfp4", 4): (117, 121), ("mxfp4", 16): (110, 126), ("nvfp4", 4): (0x58, 0x7F), ("nvfp4", 16): (1, 0x7F)}[fmt, octaves]
    scales = torch.randint(lo, hi, (R, ref.blocks(K, fmt)), generator=rng, device="cuda").byte()
    q = tgemm.mx4_pack((codes[:, 0::2] | codes[:, 1::2] << 4).contiguous(), scales, fmt, cols=K)
    v = torch.from_numpy(ref.e2m1(np.arange(16))).cuda()[codes[:, :K].long()]
    s = torch.from_numpy(ref.scale_value(np.arange(256), fmt)).cuda()[scales.long()]
    return q, v * s.repeat_interleave(ref.BLOCK[fmt], dim=1)[:, :K]


# SM pairs, single SMs, clusters that share the sum; C with and without TMA stores.
MX4 = [(600, 3300, 60000), (2100, 1303, 8255), (500, 1000, 60000), (130, 1001, 66000), (20, 260, 400000)]


@pytest.mark.parametrize("M,N,K", MX4)
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_products_keep_the_low_bits_of_positive_terms(tgemm, fmt, M, N, K):
    """A step of 64 columns is taken as one of 16: its products are summed
    exactly before they are scaled and added."""
    A, a = matrix(tgemm, M, K, fmt, True, 4, K)
    B, b = matrix(tgemm, N, K, fmt, True, 4, K + 1)
    want = a @ b.t()
    additions = -(-K // 4096) + 8 + 4
    rel = float((tgemm.gemm_mx4(A, B).double() / want - 1.0).abs().max())
    assert rel <= 1.05 * (2 * 2.0 ** -23 * (64 + 1) / 2 + additions * 2.0 ** -24), rel


@pytest.mark.parametrize("M,N,K", MX4)
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_products_over_many_octaves_are_as_exact_as_fp32(tgemm, fmt, M, N, K):
    A, a = matrix(tgemm, M, K, fmt, False, 16, K)
    B, b = matrix(tgemm, N, K, fmt, False, 16, K + 1)
    want = a @ b.t()
    rel = float((tgemm.gemm_mx4(A, B).double() - want).norm() / want.norm())
    assert rel <= 64 * (2 / 3) * 2.0 ** -24, rel


@pytest.mark.parametrize("M,N", [(20, 260), (500, 1000), (2100, 1303)])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_long_products_of_whole_numbers_under_the_output_rule(tgemm, fmt, M, N):
    """Terms that are whole halves of a unit: every sum is exact, and so is the
    rule's result; rows and columns outside C stay as they were."""
    K = 12345
    rng = np.random.default_rng(M)
    store = torch.full((M + 2, N + 5), -77.0, device="cuda")
    codes = [rng.choice([0, 1, 2, 9, 10], (R, K)) for R in (M, N)]
    q = [tgemm.mx4_pack(torch.from_numpy(ref.pack_codes(c)).cuda(),
                        torch.full((len(c), ref.blocks(K, fmt)), {"mxfp4": 127, "nvfp4": 0x38}[fmt], dtype=torch.uint8, device="cuda"),
                        fmt, cols=K) for c in codes]
    a, b = (torch.from_numpy(ref.e2m1(c)).cuda() for c in codes)
    want = a @ b.t()
    bias = torch.arange(N, device="cuda", dtype=torch.float32)
    assert torch.equal(tgemm.gemm_mx4(*q).double(), want)
    assert torch.equal(tgemm.gemm_mx4(*q, bias=bias, alpha=2.0).double(), 2 * want + bias.double())
    out = store[1:M + 1, :N]
    out.copy_(torch.from_numpy(rng.integers(-50, 50, (M, N))))
    rule = -0.5 * want + 2.0 * out.double() + bias.double()
    tgemm.gemm_mx4(*q, alpha=-0.5, beta=2.0, bias=bias, out=out)
    assert torch.equal(out.double(), rule)
    assert (store[0] == -77).all() and (store[-1] == -77).all() and (store[:, N:] == -77).all()
    assert tgemm.device_status() == 0


@pytest.mark.parametrize("M,N", [(40, 200), (500, 1000), (2100, 2600)])
@pytest.mark.parametrize("op", ["mx4", "w4"])
def test_a_stage_of_a_long_sum_that_never_fills_is_reported(tgemm, op, M, N):
    A, B, a, b = operands(tgemm, op, M, N, 9000, "nvfp4", "normal")
    want = call(tgemm, op)(A, B)
    assert tgemm.device_status() == 0
    tgemm.binding.set_wait_limit_ns(20_000_000)
    tgemm.binding.set_debug_stall(True)
    try:
        call(tgemm, op)(A, B)
        assert tgemm.device_status() == tgemm.binding.TGEMM_ERR_DEVICE_TIMEOUT
    finally:
        tgemm.binding.set_debug_stall(False)
        tgemm.binding.set_wait_limit_ns(2_000_000_000)
    assert tgemm.device_status() == 0
    assert torch.equal(call(tgemm, op)(A, B), want)
    assert tgemm.device_status() == 0
