"""gdn_linear_fp8 for prompts: the persistent kernel on pairs of CTAs, at sizes
where a pair goes through several tiles and its ring of loads wraps, in every
output type, with and without a bias. Bounds as in test_gpu_linear_fp8; the
products in fp64 are taken on the GPU."""

import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from tests.decay_reference import HALF_STEP, TINY, U
from tests.test_gpu_linear_fp8 import DT, codes

pytestmark = pytest.mark.gpu
TILE, STAGES = 256, 6  # rows and features of a tile; K steps of 128 in the ring


def operands(seed, M, N, K, bias):
    gen = torch.Generator().manual_seed(seed)
    x, w = codes(gen, M, K + 16)[:, :K], codes(gen, N, K)
    xs, ws = torch.rand(M, generator=gen).cuda() + 0.1, torch.rand(N, generator=gen).cuda() * 0.1
    return x, xs, w, ws, torch.randn(N, generator=gen).cuda() * 50 if bias else None


def call(ops, dtype, y=None):
    x, xs, w, ws, b = ops
    N = w.shape[0]
    if y is None:
        wide = torch.full((x.shape[0] + 3, (N + 7) // 8 * 8 + 8), 7.25, dtype=DT[dtype], device="cuda")
        y = wide[:x.shape[0], :N]
    gdn.gdn_linear_fp8(x, xs, w, ws, y, bias=b)
    return y


def exact(ops):
    x, xs, w, ws, b = ops
    X, W = x.float().double(), w.float().double()
    sc = xs.double()[:, None] * ws.double()
    Y = X @ W.t() * sc
    mag = X.abs() @ W.abs().t() * sc
    return (Y if b is None else Y + b.double()), mag


def verify(ops, y, dtype, rows=None, cols=None):
    Y, mag = exact(ops)
    bound = ((2 * U * ops[0].shape[1] + 4 * U) * mag + 2 * U * Y.abs()) * 1.01 + HALF_STEP[dtype] * Y.abs() + TINY[dtype]
    over = (y.double() - Y).abs() - bound
    if rows is not None:
        over = over[rows][:, cols]
    assert bool(torch.isfinite(over).all()) and float(over.max()) <= 0, (
        f"{int((over > 0).sum())} beyond the bound, the worst by {float(over.max()):.3e}")


def takes_tiles(M, N):
    tiles = -(-M // TILE) * -(-N // TILE)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return M > 128 and 4 * tiles >= sms, tiles / (sms // 2)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("M,N,K", [(2100, 9001, 1040),   # four tiles a pair and more, nine K steps each
                                   (601, 12999, 2064),   # 17 K steps a tile
                                   (129, 9730, 144)])    # the fewest rows, two K steps
def test_products(dtype, bias, M, N, K):
    assert takes_tiles(M, N)[0]
    ops = operands(M + N, M, N, K, bias)
    y = call(ops, dtype)
    verify(ops, y, dtype)
    wide = y._base
    assert (wide[:, N:] == 7.25).all() and (wide[M:] == 7.25).all()
    assert gdn.gdn_device_error() == 0


def test_sizes_reach_what_they_are_for():
    ok, per_pair = takes_tiles(2100, 9001)
    assert ok and per_pair > 4 and -(-1040 // 128) > STAGES


def test_nan_stays_in_its_row_and_column():
    M, N, K = 2100, 9001, 528
    ops = operands(5, M, N, K, False)
    x, w = ops[0], ops[2]
    rows, cols = [0, 130, 255, 256, 2099], [0, 127, 128, 300, 9000]
    for i, r in enumerate(rows):
        x.view(torch.uint8)[r, 100 * i] = 0x7F
    for i, c in enumerate(cols):
        w.view(torch.uint8)[c, K - 1 - 64 * i] = 0xFF
    y = call(ops, "f32")
    want = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    want[rows, :] = True
    want[:, cols] = True
    assert torch.equal(torch.isnan(y), want)
    keep = lambda n, out: torch.tensor([i for i in range(n) if i not in out], device="cuda")
    verify(ops, y, "f32", keep(M, rows), keep(N, cols))


def test_largest_codes():
    """Every product 448^2: the largest sums."""
    M, N, K = 300, 9001, 2048
    one = lambda n: torch.ones(n, device="cuda")
    x = torch.full((M, K), 448.0).to(torch.float8_e4m3fn).cuda()
    w = torch.full((N, K), -448.0).to(torch.float8_e4m3fn).cuda()
    assert takes_tiles(M, N)[0]
    verify((x, one(M), w, one(N), None), call((x, one(M), w, one(N), None), "f32"), "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_result_every_time_and_in_a_graph(dtype):
    ops = operands(6, 2100, 9001, 1040, True)
    y = call(ops, dtype)
    first = y.clone()
    for _ in range(3):
        y.zero_()
        call(ops, dtype, y)
        assert torch.equal(first, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(ops, dtype, y)
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, y)


def test_two_calls_side_by_side():
    """Two persistent grids at once, on two streams."""
    both = [operands(7 + i, 2100, 9001, 1040, True) for i in range(2)]
    want = [call(ops, "bf16").clone() for ops in both]
    ys = [torch.zeros((2100, 9008), dtype=torch.bfloat16, device="cuda")[:, :9001] for _ in both]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for _ in range(3):
        for (x, xs, w, ws, b), y, s in zip(both, ys, streams):
            gdn.gdn_linear_fp8(x, xs, w, ws, y, bias=b, stream=s)
    torch.cuda.synchronize()
    for y, t in zip(ys, want):
        assert torch.equal(y, t)
    assert gdn.gdn_device_error() == 0
