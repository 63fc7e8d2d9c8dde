"""Products on SM pairs, whose blocks hand shared memory and accumulators to
each other, repeated while another stream keeps the GPU's memory busy."""
import numpy as np
import pytest
import torch

from test_gpu_mx4_product import F32_REL, call, operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dtype", [("mxfp4", torch.float32), ("nvfp4", torch.bfloat16)])
@pytest.mark.parametrize("op", ["mx4", "w4"])
def test_long_pair_products_give_the_same_bits_beside_other_work(tgemm, op, fmt, dtype):
    M, N, K = 2100, 2600, 9000
    A, B, a, b = operands(tgemm, op, M, N, K, fmt, "wide")
    first = call(tgemm, op)(A, B, out_dtype=dtype)
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = F32_REL * size + (2.0 ** -8 * np.abs(want) * (1 + F32_REL) + 2.0 ** -8 * F32_REL * size if dtype == torch.bfloat16 else 0.0)
    assert (np.abs(first.double().cpu().numpy() - want) <= tol).all()
    src = torch.arange(1 << 27, dtype=torch.int32, device="cuda")        # 512 MB
    dst = torch.empty_like(src)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(first) for _ in range(8)]
    for _ in range(10):
        with torch.cuda.stream(side):
            for _ in range(4):
                dst.copy_(src, non_blocking=True)
                dst.add_(1)
        for out in outs:
            out.zero_()
            call(tgemm, op)(A, B, out=out)
        for out in outs:
            assert torch.equal(out, first)
    side.synchronize()
    assert tgemm.device_status() == 0
