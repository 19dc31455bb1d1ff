"""gdn_linear_fp8 against the product in fp64. Products of two e4m3 values are
exact in fp32; a sum of K of them in fp32 is off by at most K half steps
(2^-24; the tensor cores may truncate, so a whole step, 2^-23) of the sum of
magnitudes, the scales and the bias add three roundings, the output one."""

import numpy as np
import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from tests.decay_reference import HALF_STEP, TINY, U, check

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().float().cpu().double().numpy()


def codes(gen, rows, cols, std=40.0):
    return (torch.randn((rows, cols), generator=gen) * std).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()


def verify(x, xs, w, ws, bias, y, dtype):
    X, W = f64(x), f64(w)
    sc = f64(xs)[:, None] * f64(ws)
    Y = X @ W.T * sc + (0 if bias is None else f64(bias))
    mag = np.abs(X) @ np.abs(W).T * sc
    bound = (2 * U * X.shape[1] + 4 * U) * mag + 2 * U * np.abs(Y)
    check(f64(y), Y, bound * 1.01 + HALF_STEP[dtype] * np.abs(Y) + TINY[dtype], "y")


def run(seed, M, N, K, dtype="bf16", bias=True, x_pad=0, y_pad=0):
    gen = torch.Generator().manual_seed(seed)
    x = codes(gen, M, K + x_pad)[:, :K]
    w = codes(gen, N, K)
    xs, ws = torch.rand(M, generator=gen).cuda() + 0.1, torch.rand(N, generator=gen).cuda() * 0.1
    b = torch.randn(N, generator=gen).cuda() * 50 if bias else None
    ld = (N + 7) // 8 * 8 + y_pad
    wide = torch.full((M, ld), 7.25, dtype=DT[dtype], device="cuda")
    y = wide[:, :N]
    gdn.gdn_linear_fp8(x, xs, w, ws, y, bias=b)
    verify(x, xs, w, ws, b, y, dtype)
    assert (wide[:, N:] == 7.25).all()
    assert gdn.gdn_device_error() == 0
    return x, xs, w, ws, b, y


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 8, 16), (3, 5, 48), (7, 64, 128), (8, 65, 144), (16, 200, 1024), (33, 129, 2048), (64, 64, 4096),
    (127, 100, 256), (128, 72, 272), (129, 64, 128), (200, 333, 400), (257, 520, 640)])
def test_products(dtype, M, N, K):
    run(M + N + K, M, N, K, dtype, bias=K % 3 != 0, x_pad=16 * (M % 3), y_pad=8 * (N % 2))


@pytest.mark.parametrize("M,N,K", [(1, 12352, 2048), (5, 2048, 4096), (64, 12352, 2048), (128, 2048, 4096),
                                   (300, 12352, 256), (1000, 2048, 1024), (1500, 2056, 528), (2304, 1024, 128)])
def test_layer_sizes(M, N, K):
    run(7, M, N, K)


@pytest.mark.parametrize("M,N,K", [(1, 40960, 128), (16, 38913, 400), (50, 39000, 656), (128, 41000, 256)])
def test_bands_of_several_waves(M, N, K):
    run(8, M, N, K, y_pad=8)


def test_largest_codes_and_zeros():
    """All 448: every sum is K 448^2, the largest that fp32 sums of codes reach; and all zeros."""
    for M in (2, 130):
        x = torch.full((M, 2048), 448.0).to(torch.float8_e4m3fn).cuda()
        w = torch.full((70, 2048), -448.0).to(torch.float8_e4m3fn).cuda()
        xs, ws = torch.ones(M, device="cuda"), torch.ones(70, device="cuda")
        y = torch.empty((M, 72), device="cuda")[:, :70]
        gdn.gdn_linear_fp8(x, xs, w, ws, y)
        verify(x, xs, w, ws, None, y, "f32")
        gdn.gdn_linear_fp8(torch.zeros_like(x), xs, w, ws, y)
        assert not y.any()


@pytest.mark.parametrize("M", [3, 140])
def test_nan_stays_in_its_row_and_column(M):
    gen = torch.Generator().manual_seed(1)
    x, w = codes(gen, M, 256), codes(gen, 80, 256)
    xs, ws = torch.ones(M, device="cuda"), torch.ones(80, device="cuda")
    x.view(torch.uint8)[1, 100] = 0x7F  # NaN
    w.view(torch.uint8)[70, 3] = 0xFF
    y = torch.empty((M, 80), device="cuda")
    gdn.gdn_linear_fp8(x, xs, w, ws, y)
    nan = torch.isnan(y).cpu()
    want = torch.zeros(M, 80, dtype=torch.bool)
    want[1, :] = True
    want[:, 70] = True
    assert torch.equal(nan, want)


def test_same_result_every_time_and_in_a_graph():
    for M in (4, 64, 700):
        x, xs, w, ws, b, y = run(11, M, 2048, 4096)
        first = y.clone()
        for _ in range(3):
            y.zero_()
            gdn.gdn_linear_fp8(x, xs, w, ws, y, bias=b)
            assert torch.equal(first, y)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gdn.gdn_linear_fp8(x, xs, w, ws, y, bias=b)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, y)


def test_refusals():
    gen = torch.Generator().manual_seed(2)
    x, w = codes(gen, 4, 64), codes(gen, 24, 64)
    xs, ws, b = torch.ones(4, device="cuda"), torch.ones(24, device="cuda"), torch.ones(24, device="cuda")
    y = torch.zeros((4, 24), device="cuda")
    for args, kw in [((x.float(), xs, w, ws, y), {}), ((x, xs, w.float(), ws, y), {}), ((x, xs[:3], w, ws, y), {}),
                     ((x, xs, w, ws[:20], y), {}), ((x, xs, w[:, :48], ws, y), {}), ((x, xs, w, ws, y[:3]), {}),
                     ((x, xs, w, ws, y.double()), {}), ((x, xs, w, ws, y), {"bias": b[:23]}),
                     ((x, xs, w, ws, y), {"bias": b.half()}), ((x.cpu(), xs, w, ws, y), {}), ((x[0], xs, w, ws, y), {}),
                     ((x[:, :40].contiguous(), xs, w[:, :40].contiguous(), ws, y), {}),  # K not a multiple of 16
                     ((x, xs, w, ws, torch.zeros((4, 25), device="cuda")[:, :24]), {}),  # y's stride
                     ((x, xs, w, ws, torch.zeros((24, 4), device="cuda").t()), {})]:
        with pytest.raises((ValueError, TypeError, gdn.GdnError)):
            gdn.gdn_linear_fp8(*args, **kw)
    assert not y.any()
