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


@pytest.mark.parametrize("M", [1, 20, 260])
def test_operands_written_just_before_they_are_read(tgemm, M):
    """Chains of calls whose operands (values, tensor scales, codes, bias) the
    calls before them on the stream have just written, in the same buffers each
    time, against the same chain with a wait after each call."""
    N, K = 520, 1100
    rng = torch.Generator(device="cuda").manual_seed(M)
    X = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    W = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
    bias, g = torch.empty(N, device="cuda"), torch.empty(1, device="cuda")
    back = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    seeds = [torch.randn(3, generator=rng, device="cuda") for _ in range(30)]
    base = torch.randn(N, K, generator=rng, device="cuda"), torch.randn(M, K, generator=rng, device="cuda")

    def chain(seed, wait):
        def then(x):
            if wait:
                torch.cuda.synchronize()
            return x

        torch.mul(base[1], seed[0] * 30, out=X)
        then(torch.mul(base[0], seed[1], out=W))
        torch.mul(base[0][:, 0], seed[2], out=bias)
        g.copy_(then(tgemm.mx4_tensor_scale(X)))
        x = then(tgemm.mx4_quantize(X, "nvfp4", tensor_scale=g))
        w, w_t = then(tgemm.mx4_quantize_both(W, "nvfp4"))
        tgemm.mx4_dequantize(x, out=back)
        then(None)
        y = then(tgemm.gemm_w4(back, w, bias=bias))
        z = then(tgemm.gemm_mx4(x, w, bias=bias, out_dtype=torch.bfloat16))
        v = then(tgemm.mx4_dequantize(w_t, torch.bfloat16))
        return y, z, v, back.clone()

    fast = [chain(s, False) for s in seeds]
    slow = [chain(s, True) for s in seeds]
    for f, s in zip(fast, slow):
        for a, b in zip(f, s):
            assert torch.equal(a, b)
    assert tgemm.device_status() == 0


@pytest.mark.parametrize("M,N,K", [(9, 4100, 4130), (20, 4100, 4130), (8, 4100, 4130), (16, 300, 4130), (40, 300, 1030)])
def test_rows_off_16_bytes_of_either_route_in_a_graph(tgemm, M, N, K):
    """9 to 24 rows of much weight: such an A is copied to scratch first."""
    A, B, a, b = operands(tgemm, "w4", M, N, K, "mxfp4", "whole")
    A = torch.cat([A, A[:, :3]], dim=1)[:, :K]
    assert A.stride(0) % 8 != 0
    want = torch.from_numpy(a @ b.T).float().cuda()
    assert torch.equal(tgemm.gemm_w4(A, B), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tgemm.gemm_w4(A, B)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert tgemm.device_status() == 0
