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
