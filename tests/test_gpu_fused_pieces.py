"""gemm_ce_grad over several pieces of the vocabulary: dX's sum in scratch or where it is."""
import os
import subprocess
import sys

import pytest
import torch

from test_gpu_fused_act import BF16, F32, SENTINEL, generator
from test_gpu_fused_ce import inputs

pytestmark = pytest.mark.gpu

T, V = 40000, 7003                      # pieces of 3328 columns


def call(tgemm, X, W, t, lse, dloss, dX, D):
    lib = tgemm.fused.load()
    assert lib.gemm_ce_grad(len(X), len(W), D, X.data_ptr(), X.stride(0), W.data_ptr(), W.stride(0), 1.0, t.data_ptr(),
                            lse.data_ptr(), dloss.data_ptr(), dX.data_ptr(), dX.stride(0), 0, None, D, 0, 0.0,
                            torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.parametrize("D,pad,shift", [(72, 0, 0), (72, 8, 0), (72, 8, 4), (72, 8, 1), (72, 9, 0), (70, 10, 0), (2056, 0, 0)])
def test_an_fp32_dx_in_any_storage(tgemm, D, pad, shift):
    x, w, target = inputs(generator(D), T, V, D)
    X, W, t = x.cuda(), w.cuda(), target.cuda()
    loss, lse = tgemm.gemm_ce(X, W, t)
    dloss = torch.rand(T, generator=torch.Generator().manual_seed(D)).cuda()
    around = torch.full(((T + 1) * (D + pad) + shift,), SENTINEL, device="cuda")
    view = around[shift:shift + T * (D + pad)].view(T, D + pad)[:, :D]
    call(tgemm, X, W, t, lse, dloss, view, D)
    # In 64 bits from the same dz, rounded to BF16 as it is there (an element of dz that lies next to a border
    # may round the other way: 2^-8 of it), and 1e-6 for the sums.
    kept = (t >= 0) & (t < V)
    rows = torch.arange(0, T, 37, device="cuda")
    z = X[rows].double() @ W.double().t()
    p = torch.exp(z - lse[rows].double()[:, None])
    p[kept[rows].nonzero()[:, 0], t[rows][kept[rows]]] -= 1
    dz = torch.where(kept[rows, None], p * dloss[rows].double()[:, None], torch.zeros_like(p))
    want = dz @ W.double()
    tol = 2.0 ** -8 * (dz.abs() @ W.double().abs()) + 2.0 ** -18 * want.abs().max()
    assert ((view[rows].double() - want).abs() <= tol).all()
    got = view.clone()
    view.fill_(SENTINEL)
    assert (around == SENTINEL).all()
    # The same sums wherever they are kept, and whatever dX held before.
    view.fill_(float("nan"))
    call(tgemm, X, W, t, lse, dloss, view, D)
    assert torch.equal(view, got)
    dx, _ = tgemm.gemm_ce_grad(X, W, t, lse, dloss, w_grad=False, dx_dtype=F32)
    assert (dx.double() - got.double()).norm() <= 1e-6 * got.double().norm()
    dx, _ = tgemm.gemm_ce_grad(X, W, t, lse, dloss, w_grad=False)
    assert ((dx.double() - got.double()).abs() <= 2.0 ** -8 * got.double().abs() + 1e-6 * got.double().abs().max()).all()
    assert tgemm.device_status() == 0


MEMORY = """
import torch, tiled_matrix_multiplication_sm_gb300 as tg
T, V, D = 131072, 1500, 2048
X, W = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
t, f = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.ones(T, device="cuda")
tg.gemm_act(X[:1], W[:16], trans_b=True)
torch.cuda.synchronize()
free, own = torch.cuda.mem_get_info()[0], torch.cuda.memory_reserved()
dx, _ = tg.gemm_ce_grad(X, W, t, f, f, w_grad=False, dx_dtype=torch.float32)
torch.cuda.synchronize()
print(free - torch.cuda.mem_get_info()[0] - (torch.cuda.memory_reserved() - own))
"""


def test_an_fp32_dx_takes_no_second_one():
    """Scratch for dz's piece alone, 268 MB: not 1 GB for a matrix of dX's size and type beside it."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", MEMORY], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    assert int(out.stdout) < 600 << 20
