"""Bounded waits of the 4-bit tensor-core kernels: a stage that never fills is
reported by gemm_device_status, and the next call is right."""
import numpy as np
import pytest
import torch

from test_gpu_mx4_product import call, operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N", [(40, 200), (2100, 2600)])      # one SM, SM pairs
@pytest.mark.parametrize("op", ["mx4", "w4"])
def test_a_stage_that_never_fills_is_reported(tgemm, op, M, N):
    A, B, a, b = operands(tgemm, op, M, N, 512, "nvfp4", "whole")
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
    assert np.array_equal(call(tgemm, op)(A, B).double().cpu().numpy(), a @ b.T)
    assert tgemm.device_status() == 0
