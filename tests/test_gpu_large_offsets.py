"""Rows whose offsets pass 32 bits, and sizes at the ends of a kernel's range: the last rows are checked, and that what
lies behind them is left alone."""

import numpy as np
import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from tests import decay_reference as ref
from tests import test_gpu_add_rmsnorm as norm
from tests import test_gpu_linear_fp8_tiles as tiles
from tests.test_gpu_decay import DT, SPLIT, f64

pytestmark = pytest.mark.gpu


def needs(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GB of device memory")


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_decay_prefill(dtype, D):
    """Two sequences in rows of a wide activation; the second, of 100 tokens, lies past 2^31 elements."""
    needs(24)
    hk, hv, width, T = 1, 2, 12288, 2 ** 31 // 12288 + 150
    act = torch.zeros((T, width), dtype=DT[dtype], device="cuda")
    gen = torch.Generator().manual_seed(91)
    act[T - 100:, width - 6 * D:] = torch.randn((100, 6 * D), generator=gen).to(DT[dtype]).cuda()
    q, k, v, z = act[:, width - 6 * D:].split([D, D, 2 * D, 2 * D], dim=1)
    g = torch.zeros((T, hv), device="cuda")
    g[T - 100:] = -torch.rand((100, hv), generator=gen).cuda()
    w = (1 + 0.2 * torch.randn(D, generator=gen)).cuda()
    state = torch.randn((2, hv, D, D), generator=gen).cuda() * 0.1
    S0 = state.clone()
    core = torch.full((T, hv, D), 7.25, device="cuda")
    out = torch.full((T, hv, D), 7.25, dtype=DT[dtype], device="cuda")
    d = gdn.dims(hk, hv, D, io_dtype=DT[dtype])
    cu = torch.tensor([0, T - 100, T - 3], dtype=torch.int32, device="cuda")  # three rows behind the last sequence
    gdn.gdn_decay_prefill(d, cu, q, k, v, g, state, core_out=core, out=out, z=z, norm_w=w)
    assert torch.equal(state[0], S0[0])  # zeros, and no decay
    a, b = T - 100, T - 3
    r = lambda t, h: f64(t[a:b]).reshape(b - a, h, D)
    o, S, do, mag, dS, A = ref.recurrence(r(q, hk), r(k, hk), r(v, hv), f64(g[a:b]), f64(S0[1]), D ** -0.5, False)
    split = SPLIT if dtype == "bf16" else 0.0
    do = do + split * mag
    ref.check(f64(state[1]), S, dS * 1.02 + split * A, "state")
    ref.check(f64(core[a:b]), o, do * 1.02 + 1e-38, "core_out")
    y, dy = ref.gated(o, r(z, hv), f64(w), 1e-6, dtype, do)
    ref.check(f64(out[a:b]), y, dy, "out")
    assert (core[b:] == 7.25).all() and (out[b:] == 7.25).all()
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("rows,cols", [(2 ** 31 // 8192 + 5, 8192), (2 ** 31 // 515 + 5, 515)])
def test_add_rmsnorm(rows, cols):
    needs(24)
    gen = torch.Generator().manual_seed(92)
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-7:] = torch.randn((7, cols), generator=gen).to(torch.bfloat16).cuda()
    w = (1 + 0.3 * torch.randn(cols, generator=gen)).cuda()
    y, q = torch.full_like(x, 7.25), torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(rows, device="cuda")
    gdn.gdn_add_rmsnorm(x, w, out=y, out_q=q, out_scale=sc)
    norm.verify(x[-7:], None, w, 1e-6, "bf16", None, y[-7:], q.view(torch.uint8)[-7:].view(torch.float8_e4m3fn), sc[-7:])
    assert not y[:-7].any() and not (q.view(torch.uint8)[:-7] & 0x7f).any()  # zeros (of a negative weight: -0)


@pytest.mark.parametrize("M,N,K", [(2 ** 31 // 8192 + 77, 8192, 16), (9801, 5, 16), (16384, 1, 48)])
def test_linear_fp8(M, N, K):
    """Outputs past 2^31 elements; few features for many rows."""
    needs(24)
    assert tiles.takes_tiles(M, N)[0]
    x, xs, w, ws, b = tiles.operands(93, M, N, K, True)
    y = tiles.call((x, xs, w, ws, b), "bf16")
    for rows in (slice(0, 300), slice(M - 300, M)):
        tiles.verify((x[rows], xs[rows], w, ws, b), y[rows], "bf16")
    wide = y._base
    assert (wide[M:] == 7.25).all() and (wide[:, N:] == 7.25).all()
