"""gemm_act and gemm_act_grad on SM pairs that share a tile's sum in clusters of
four, six and eight blocks: whole numbers exactly, long sums within derived bounds."""
import zlib

import pytest
import torch

import fused_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# Tiles of 256 x 256 whose sums are long enough to share: by four pairs (2, 15 tiles), three
# (16, 23) and two (24, 36), 37 by none; K not whole stages, nor the same for every pair.
SIZES = [(300, 256, 2100), (700, 1210, 2240), (1000, 1000, 1990), (256, 5888, 2050), (1500, 1000, 1800), (1500, 1500, 2176),
         (250, 9472, 1600)]


@pytest.fixture(autouse=True)
def pairs(tgemm):
    assert tgemm.fused.set_fused_kernel(0) == 0
    yield
    tgemm.fused.set_fused_kernel(-1)


def generator(*seed):
    return torch.Generator().manual_seed(zlib.crc32(repr(seed).encode()))


def whole(g, *size, most=1):
    return torch.randint(-most, most + 1, size, generator=g).float()


def product(a, b):
    """Of whole numbers, exact: sums below 2^24."""
    return (a.cuda() @ b.cuda()).cpu()


@pytest.mark.parametrize("trans_a,trans_b", [(False, True), (False, False), (True, False), (True, True)])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_whole_numbers_are_exact(tgemm, M, N, K, off, trans_a, trans_b):
    """FP32 C and R, Z, bias; off: rows of C, R and Z off 16 bytes."""
    g = generator(M, N, K, trans_a, trans_b)
    a, b, bias, r = whole(g, M, K), whole(g, K, N), whole(g, N), whole(g, M, N + off)
    z = product(a, b) + bias
    A = (a.t().contiguous() if trans_a else a).to(BF16).cuda()
    B = (b.t().contiguous() if trans_b else b).to(BF16).cuda()
    R = r.cuda()[:, off:]
    out = torch.full((M, N + off), 7.0, device="cuda")
    C, Z = tgemm.gemm_act(A, B, "relu", trans_a=trans_a, trans_b=trans_b, bias=bias.cuda(), residual=R, keep_z=True, out=out[:, off:])
    assert torch.equal(C.cpu(), z.clamp(min=0) + r[:, off:])
    assert torch.equal(Z.cpu(), z.to(BF16))
    assert off == 0 or bool((out[:, 0] == 7.0).all())
    plain = tgemm.gemm_act(A, B, trans_a=trans_a, trans_b=trans_b)
    assert torch.equal(plain.cpu(), (z - bias).to(BF16))
    assert tgemm.device_status() == 0


@pytest.mark.parametrize("extras", ["", "bias keep_z", "residual"])
@pytest.mark.parametrize("M,N,K", [(300, 128, 2100), (700, 605, 2240), (1500, 500, 1800), (1500, 747, 2176), (250, 4736, 1600)])
def test_gated_whole_numbers_are_exact(tgemm, M, N, K, extras):
    g = generator(M, N, K, extras)
    a, b = whole(g, M, K), whole(g, K, 2 * N)
    z = product(a, b)
    bias = whole(g, 2 * N) if "bias" in extras else None
    z = z if bias is None else z + bias
    # Products of two whole numbers below 2^12 and sums of such: exact before the rounding.
    want = z[:, :N].clamp(min=0) * z[:, N:]
    r = whole(g, M, N) if "residual" in extras else None
    want = want if r is None else want + r
    got = tgemm.gemm_act(a.to(BF16).cuda(), b.to(BF16).cuda(), "relu", gated=True, bias=None if bias is None else bias.cuda(),
                         residual=None if r is None else r.to(BF16).cuda(), keep_z="keep_z" in extras)
    if "keep_z" in extras:
        got, Z = got
        assert torch.equal(Z.cpu(), z.to(BF16))
    assert torch.equal(got.cpu(), want.to(BF16))


@pytest.mark.parametrize("c", [BF16, F32])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gradients_of_whole_numbers_are_exact(tgemm, M, N, K, off, c):
    g = generator(M, N, K, str(c))
    a, b, z = whole(g, M, K), whole(g, K, N), whole(g, M, N + off)
    want = product(a, b) * (z[:, off:] > 0)
    dz, db = tgemm.gemm_act_grad(a.to(BF16).cuda(), b.to(BF16).cuda(), z.to(BF16).cuda()[:, off:], "relu", out_dtype=c)
    assert torch.equal(dz.cpu(), want.to(c))
    assert torch.equal(db.cpu(), want.sum(dim=0))
    assert tgemm.device_status() == 0


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("M,N,K", [(300, 520, 9000), (500, 1100, 5000), (1500, 1480, 2500)])
def test_long_sums_are_within_their_bounds(tgemm, M, N, K, act):
    g = generator(M, N, K, act)
    a = torch.randn(M, K, generator=g).to(BF16)
    b = (torch.randn(N, K, generator=g) * 2.5 / K ** 0.5).to(BF16)
    z, ez = ref.sums(a.double(), b.double().t())
    want, ev = ref.act_bound(act, z, ez)
    for c in (BF16, F32):
        got = tgemm.gemm_act(a.cuda(), b.cuda(), act, trans_b=True, out_dtype=c)
        ref.check(got, want, ref.rounded(want, ev, c), str(c))


def test_the_same_call_gives_the_same_bits_alone_and_in_a_graph(tgemm):
    """Shares are added in the pairs' order, whatever arrives first; two graphs run at once."""
    g = generator("bits")
    a, b = (torch.randn(700, 3000, generator=g).to(BF16).cuda(), torch.randn(1200, 3000, generator=g).to(BF16).cuda())
    first = tgemm.gemm_act(a, b, "gelu", trans_b=True, out_dtype=F32)
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, results = [], []
    torch.cuda.synchronize()
    for s in streams:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            results.append([tgemm.gemm_act(a, b, "gelu", trans_b=True, out_dtype=F32) for _ in range(3)])
        graphs.append(graph)
    for _ in range(5):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first, x) for xs in results for x in xs)
    assert tgemm.device_status() == 0


@pytest.mark.parametrize("M,N", [(300, 256), (1500, 1500)])
@pytest.mark.parametrize("c", [BF16, F32])
def test_a_stage_that_never_fills_is_reported(tgemm, M, N, c):
    """Every pair's waits run out, and the cluster's blocks meet all the same."""
    K = 2100
    g = generator("stall", M, N)
    a, b = whole(g, M, K), whole(g, N, K)
    A, B = a.to(BF16).cuda(), b.to(BF16).cuda()
    assert tgemm.device_status() == 0
    tgemm.binding.set_wait_limit_ns(20_000_000)
    tgemm.binding.set_debug_stall(True)
    try:
        tgemm.gemm_act(A, B, "relu", trans_b=True, out_dtype=c)
        assert tgemm.device_status() == tgemm.binding.TGEMM_ERR_DEVICE_TIMEOUT
    finally:
        tgemm.binding.set_debug_stall(False)
        tgemm.binding.set_wait_limit_ns(2_000_000_000)
    assert tgemm.device_status() == 0
    assert torch.equal(tgemm.gemm_act(A, B, "relu", trans_b=True, out_dtype=c).cpu(), product(a, b.t()).clamp(min=0).to(c))
