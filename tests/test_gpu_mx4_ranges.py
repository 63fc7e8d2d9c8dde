"""4-bit operators at the ends of the number range, against 64 bits."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from test_gpu_mx4_quantize import check, draw, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,C,ld", [(40, 100, 100), (130, 64, 64), (3, 33, 40)])       # rows off and on 16 bytes
def test_values_far_above_a_kept_tensor_scale_keep_their_sign(tgemm, dtype, R, C, ld):
    """g of an earlier step whose matrix was zero: magnitudes above 6 go to 6, even
    where x / (scale g) is past FP32's range. Beside them in the same block
    values in the middle of two codes, and a zero."""
    g = 2.0 ** -100
    X = torch.zeros(R, ld, dtype=dtype, device="cuda")[:, :C]
    d = 448 * g
    few = np.array([2.0 ** 37, 2.0 ** 60, 3.3e38, 5 * d, 2.5 * d, 0.25 * d, 7 * d, 2.0 ** 28 * 1.75, 0.0, d])
    i, j = np.indices((R, C))
    x = few[(i * 3 + j * 7) % len(few)] * np.where((i + j // 2) % 2 == 0, 1.0, -1.0)
    x[1] = 1e-3 * d                                   # a row without large values
    X.copy_(torch.from_numpy(x))
    gt = torch.tensor([g], device="cuda")
    check(tgemm, tgemm.mx4_quantize(X, "nvfp4", tensor_scale=gt), host(X), "nvfp4", g)
    check(tgemm, tgemm.mx4_quantize(X, "nvfp4", trans=True, tensor_scale=gt), host(X).T, "nvfp4", g)
    q, t = tgemm.mx4_quantize_both(X, "nvfp4", tensor_scale=gt)
    check(tgemm, q, host(X), "nvfp4", g)
    check(tgemm, t, host(X).T, "nvfp4", g)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("power", [-100, -60, 0, 40, 59, 60, 99, 117])
def test_every_tensor_scale(tgemm, dtype, power):
    """g over its range, the values about g, far below it and up to the range's end."""
    g = 2.0 ** power
    X = torch.zeros(60, 200, dtype=dtype, device="cuda")
    x = host(draw(60, 200, dtype, 9))
    for i, up in enumerate((power + 10, power, power - 40, 0, 100, 124)):
        X[10 * i:10 * i + 10] = torch.from_numpy(np.ldexp(x[10 * i:10 * i + 10], min(max(up, -105), 124)))
    gt = torch.tensor([g], device="cuda")
    q, t = tgemm.mx4_quantize_both(X, "nvfp4", tensor_scale=gt)
    for q, x in ((q, host(X)), (t, host(X).T)):
        codes, scales = ref.unpack(q)
        want_codes, want_scales = ref.quantize(x, "nvfp4", g)
        assert np.array_equal(scales, want_scales)
        assert np.array_equal(ref.e2m1(codes), ref.e2m1(want_codes))


@pytest.mark.parametrize("power", [-100, -3, 0, 30, 117])
def test_quotients_one_step_from_the_midpoints(tgemm, power):
    """FP32 values that are the midpoint of two codes times a scale, or next to
    one: every code is the nearest."""
    g = 2.0 ** power
    scales = ref.scale_value(np.arange(8, 127), "nvfp4")            # normal numbers
    scales = scales[scales * 6.0 * g < 2.0 ** 127]
    x = np.zeros((len(scales), 32), dtype=np.float32)
    for i, mid in enumerate(ref.MIDPOINTS):
        v = (mid * scales * g).astype(np.float32)
        assert np.array_equal(v.astype(np.float64), mid * scales * g)
        x[:, 4 * i], x[:, 4 * i + 1], x[:, 4 * i + 2] = v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(np.inf))
        x[:, 4 * i + 1] *= -1
    x[:, 31] = x[:, 15] = (6 * scales * g).astype(np.float32)       # the largest of both blocks
    X = torch.from_numpy(x).cuda()
    q = tgemm.mx4_quantize(X, "nvfp4", tensor_scale=torch.tensor([g], device="cuda"))
    codes, got = ref.unpack(q)
    want_codes, want = ref.quantize(x.astype(np.float64), "nvfp4", g)
    assert np.array_equal(got, want)
    assert np.array_equal(ref.e2m1(codes), ref.e2m1(want_codes))


@pytest.mark.parametrize("M", [1, 12, 40, 2100])             # each kernel of gemm_w4
@pytest.mark.parametrize("op", ["w4", "mx4"])
def test_every_code_under_every_mxfp4_scale(tgemm, op, M):
    """Weights up to 6 x 2^127, which no FP32 holds, times small activations."""
    scales, codes = (v.ravel() for v in np.meshgrid(np.arange(255), np.arange(16)))
    order = np.random.default_rng(2).permutation(len(scales))
    scales, codes = scales[order], codes[order]
    N, K = len(scales), 32
    B = tgemm.mx4_pack(torch.from_numpy(ref.pack_codes(np.repeat(codes[:, None], K, axis=1))).cuda(),
                       torch.from_numpy(scales[:, None].astype(np.uint8)).cuda(), "mxfp4", cols=K)
    X = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    X[:, 5] = 3 * 2.0 ** -12
    A = X if op == "w4" else tgemm.mx4_quantize(X, "mxfp4")
    got = (tgemm.gemm_w4 if op == "w4" else tgemm.gemm_mx4)(A, B).double().cpu().numpy()
    want = ref.e2m1(codes) * ref.scale_value(scales, "mxfp4") * (3 * 2.0 ** -12)
    fine = (np.abs(want) >= 2.0 ** -120) | (want == 0)
    assert fine.sum() > 0.9 * N and np.array_equal(got[:, fine], np.broadcast_to(want[fine], (M, fine.sum())))
