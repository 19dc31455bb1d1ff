"""gdn_add_rmsnorm against its formula in fp64, within bounds from its
roundings: half a step of the io type for the sum and the 16-bit output, half
a step of e4m3 (2^-4 of the value, 2^-10 below its normal range) for the
codes."""

import numpy as np
import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from tests.decay_reference import HALF_STEP, TINY, U, check

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().to("cpu", torch.float32 if t.dtype == torch.float8_e4m3fn else t.dtype).double().numpy()


def rows_of(gen, rows, cols, stride, dtype, std=1.0):
    return (torch.randn((rows, stride), generator=gen) * std).to(DT[dtype]).cuda()[:, :cols]


def verify(x, r, w, eps, dtype, s, y, q, scale):
    """Outputs (None where not asked for) of the formula; the mean's fp32 sum and the products are allowed
    (cols / 32 + 40) u of the value: a lane sums at most cols / 32 squares, the rest are single operations. Where the
    product s w is below fp32's normal range it is off by half of its smallest step, 2^-150, instead, and what
    multiplies it then is at most eps^(-1/2)."""
    cols = x.shape[1]
    X = f64(x) + (0 if r is None else f64(r))
    if s is not None:
        check(f64(s), X, (HALF_STEP[dtype] + 2 * U) * np.abs(X) + TINY[dtype], "sum_out")
        X = f64(s)
    elif r is not None:
        X = f64((x.float() + r.float()).to(x.dtype))
    rel = (cols / 32 + 40) * U
    low = 0.0 if w is None else 1.01 * 2.0 ** -150 / np.sqrt(eps)
    Y = X if w is None else X / np.sqrt((X * X).mean(-1, keepdims=True) + eps) * f64(w)
    if y is not None:
        check(f64(y), Y, (HALF_STEP[dtype] + 1.01 * rel) * np.abs(Y) + TINY[dtype] + low, "out")
    if q is not None:
        sc = np.maximum(np.abs(Y).max(-1) / 448, 2.0 ** -126)
        check(f64(scale), sc, rel * sc, "out_scale")
        code = Y / sc[:, None]
        assert np.abs(f64(q)).max() <= 448
        # half a step: 2^-4 of the value, or half of e4m3's smallest step 2^-9
        check(f64(q), code, np.maximum(2.0 ** -4 * np.abs(code), 2.0 ** -10) + 3 * rel * np.abs(code) + low / sc[:, None],
              "out_q")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,stride", [
    (1, 1, 1), (3, 7, 7), (17, 32, 32), (9, 64, 80), (8, 513, 520), (5, 512, 512), (2, 2048, 2048), (3, 2051, 2100),
    (4, 4096, 4104), (2, 8192, 8192), (1, 16384, 16384), (2, 20001, 20001), (2, 40000, 40000)])
def test_every_output(dtype, rows, cols, stride):
    gen = torch.Generator().manual_seed(rows * 1000 + cols)
    x, r = rows_of(gen, rows, cols, stride, dtype), rows_of(gen, rows, cols, stride, dtype, 3.0)
    w = (1 + 0.3 * torch.randn(cols, generator=gen)).cuda()
    wide = torch.full((rows, stride), 7.25, dtype=DT[dtype], device="cuda")
    wide_q = torch.zeros((rows, stride), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s, y, q = torch.empty_like(x), wide[:, :cols], wide_q[:, :cols]
    sc = torch.empty(rows, device="cuda")
    gdn.gdn_add_rmsnorm(x, w, residual=r, sum_out=s, out=y, out_q=q, out_scale=sc, eps=1e-5)
    verify(x, r, w, 1e-5, dtype, s, y, q, sc)
    assert (wide[:, cols:] == 7.25).all() and not wide_q.view(torch.uint8)[:, cols:].any()
    # each output alone is the same
    for kw in ({"sum_out": torch.empty_like(s)}, {"out": torch.empty_like(s)},
               {"out_q": torch.empty_like(q), "out_scale": torch.empty_like(sc)}):
        gdn.gdn_add_rmsnorm(x, w, residual=r, eps=1e-5, **kw)
        for name, full in (("sum_out", s), ("out", y), ("out_scale", sc)):
            if name in kw:
                assert torch.equal(kw[name], full)
        if "out_q" in kw:
            assert torch.equal(kw["out_q"].view(torch.uint8), q.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,stride", [(2000, 520, 520), (1999, 2048, 2064), (1850, 8192, 8192),
                                              (1300, 16384, 16384), (3000, 513, 513)])
@pytest.mark.parametrize("residual", [True, False])
def test_many_rows(dtype, rows, cols, stride, residual):
    """Rows enough for every CTA to go through several of them, in place and not; a part of them checked one by one,
    all of them against the same rows given a few at a time."""
    gen = torch.Generator().manual_seed(cols)
    x = rows_of(gen, rows, cols, stride, dtype)
    r = rows_of(gen, rows, cols, stride, dtype, 3.0) if residual else None
    w = (1 + 0.3 * torch.randn(cols, generator=gen)).cuda()
    y, q = torch.empty_like(x), torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(rows, device="cuda")
    s = torch.empty_like(x) if residual else None
    gdn.gdn_add_rmsnorm(x, w, residual=r, sum_out=s, out=y, out_q=q, out_scale=sc)
    some = torch.tensor([0, 1, 2, 700, rows // 2, rows - 2, rows - 1], device="cuda")
    verify(x[some], r[some] if residual else None, w, 1e-6, dtype, s[some] if residual else None, y[some],
           q.view(torch.uint8)[some].view(torch.float8_e4m3fn), sc[some])
    for a in range(0, rows, 304):  # (304 rows of any width end on 16 bytes)
        b = min(a + 304, rows)
        y1 = torch.empty_like(y[a:b])
        gdn.gdn_add_rmsnorm(x[a:b], w, residual=r[a:b] if residual else None, out=y1)
        # another order of the same fp32 sums: each is within verify's bound, half a step and (cols / 32 + 40) u of
        # the value, so the two are within twice that (of the larger, which 1.01 covers)
        bound = 2.02 * (HALF_STEP[dtype] + (cols / 32 + 40) * U) * y1.float().abs() + 2 * TINY[dtype]
        assert ((y1.float() - y[a:b].float()).abs() <= bound).all()
    if residual:
        gdn.gdn_add_rmsnorm(x, w, residual=r, sum_out=r, out=y)
        assert torch.equal(r, s)
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols,stride", [(3001, 3001), (4097, 4104), (5000, 5003), (8191, 8192), (8192, 8193), (8193, 8193)])
def test_rows_without_wide_accesses(dtype, cols, stride):
    """Around the lengths up to which such a row stays in registers."""
    gen = torch.Generator().manual_seed(cols)
    x, r = rows_of(gen, 5, cols, stride, dtype), rows_of(gen, 5, cols, stride, dtype, 3.0)
    w = (1 + 0.3 * torch.randn(cols, generator=gen)).cuda()
    y, q, sc = torch.empty_like(x), torch.empty((5, cols), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(5, device="cuda")
    x0, r0 = x.clone(), r.clone()
    gdn.gdn_add_rmsnorm(x, w, residual=r, sum_out=r, out=y, out_q=q, out_scale=sc)
    verify(x0, r0, w, 1e-6, dtype, r, y, q, sc)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [100, 2048, 20000])
def test_without_residual_or_weight(dtype, cols):
    gen = torch.Generator().manual_seed(cols)
    x = rows_of(gen, 6, cols, cols, dtype)
    w = (1 + 0.3 * torch.randn(cols, generator=gen)).cuda()
    y, q, sc = torch.empty_like(x), torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(6, device="cuda")
    gdn.gdn_add_rmsnorm(x, w, out=y, out_q=q, out_scale=sc)
    verify(x, None, w, 1e-6, dtype, None, y, q, sc)
    gdn.gdn_add_rmsnorm(x, None, out=y, out_q=q, out_scale=sc)
    assert torch.equal(x, y)
    verify(x, None, None, 0.0, dtype, None, None, q, sc)


@pytest.mark.parametrize("cols", [96, 4096, 33333])
@pytest.mark.parametrize("into", ["x", "residual"])
def test_residual_stream_in_place(cols, into):
    gen = torch.Generator().manual_seed(cols)
    x, r = rows_of(gen, 4, cols, cols, "bf16"), rows_of(gen, 4, cols, cols, "bf16", 3.0)
    x0, r0 = x.clone(), r.clone()
    w = (1 + 0.3 * torch.randn(cols, generator=gen)).cuda()
    y = torch.empty_like(x)
    s = x if into == "x" else r
    gdn.gdn_add_rmsnorm(x, w, residual=r, sum_out=s, out=y)
    verify(x0, r0, w, 1e-6, "bf16", s, y, None, None)


def test_zero_tiny_and_large_rows():
    x = torch.zeros((5, 256))
    x[1] = 1e-38
    x[2, 3] = 2.0 ** -149
    x[3] = 1e18
    x[4, 0], x[4, 1] = 1e-30, 448e-30
    x = x.cuda()
    q, sc = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(5, device="cuda")
    y = torch.empty_like(x)
    gdn.gdn_add_rmsnorm(x, None, out_q=q, out_scale=sc)
    assert not f64(q)[0].any() and (f64(sc) > 0).all() and np.isfinite(f64(sc)).all()
    verify(x[2:], None, None, 0, "f32", None, None, q[2:], sc[2:])
    assert (np.abs(f64(q)[1] * f64(sc)[1, None] - 1e-38) <= 2.0 ** -4 * 1e-38).all()
    gdn.gdn_add_rmsnorm(x, torch.ones(256, device="cuda"), out=y, eps=0.0 + 1e-6)
    assert not f64(y)[0].any() and np.allclose(f64(y)[3], 1.0, rtol=1e-5)


@pytest.mark.parametrize("rows", [3, 2000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_codes_of_zero_and_tiny_normed_rows(dtype, rows):
    """Zeros (a padded row) and rows so small that their inverse root over their scale passes fp32's range."""
    x = torch.randn((rows, 512), generator=torch.Generator().manual_seed(2))
    x[0] = 0.0
    x[1] *= 1e-37
    x[rows - 1] = 0.0
    x[rows - 1, 5] = 2e-37
    x = x.to(DT[dtype]).cuda()
    w = (1 + 0.3 * torch.randn(512, generator=torch.Generator().manual_seed(3))).cuda()
    y, q, sc = torch.empty_like(x), torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(rows, device="cuda")
    gdn.gdn_add_rmsnorm(x, w, out=y, out_q=q, out_scale=sc)
    verify(x, None, w, 1e-6, dtype, None, y, q, sc)
    assert not f64(q)[0].any() and not f64(y)[0].any()


def test_nan_and_infinity_stay_in_their_rows():
    x = torch.randn((4, 300), generator=torch.Generator().manual_seed(0)).cuda()
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    w = torch.ones(300, device="cuda")
    y = torch.empty_like(x)
    q, sc = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(4, device="cuda")
    gdn.gdn_add_rmsnorm(x, w, out=y, out_q=q, out_scale=sc)
    good = [0, 3]
    verify(x[good], None, w, 1e-6, "f32", None, y[good], q[good], sc[good])
    assert torch.isnan(y[1]).all() and torch.isnan(q[1].float()).all()
    assert torch.isnan(y[2, 9]) and torch.isnan(q[2].float()[9])
    gdn.gdn_add_rmsnorm(x, None, out_q=q, out_scale=sc)
    assert torch.isnan(q[1].float()[7]) and torch.isnan(q[2].float()[9])
    verify(x[good], None, None, 0, "f32", None, None, q[good], sc[good])


def test_no_rows_graph_and_stream():
    w = torch.ones(64, device="cuda")
    e = torch.empty((0, 64), device="cuda")
    gdn.gdn_add_rmsnorm(e, w, out=e.clone())
    x = torch.randn((33, 64), device="cuda")
    want = torch.empty_like(x)
    gdn.gdn_add_rmsnorm(x, w, out=want)
    y = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_add_rmsnorm(x, w, out=y)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    y.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gdn.gdn_add_rmsnorm(x, w, out=y, stream=s)
    s.synchronize()
    assert torch.equal(y, want)


def test_refusals():
    x, r, w = torch.randn((4, 64), device="cuda"), torch.randn((4, 64), device="cuda"), torch.ones(64, device="cuda")
    out, sc = torch.empty_like(x), torch.empty(4, device="cuda")
    q = torch.empty((4, 64), dtype=torch.float8_e4m3fn, device="cuda")
    bad = [dict(), dict(out_q=q), dict(out_scale=sc, out=out), dict(out=out[:3]), dict(out=out.half()),
           dict(out=out, residual=r.half()), dict(out=out, residual=r[:, :63]), dict(out=out, eps=-1.0),
           dict(out=out, eps=float("nan")), dict(out=out.cpu()), dict(out=x), dict(out=r, residual=r),
           dict(out=out, sum_out=out), dict(out_q=q.view(torch.uint8), out_scale=sc),
           dict(out=out, sum_out=x.view(-1)[4:].as_strided((4, 64), (48, 1)))]
    x0, r0 = x.clone(), r.clone()
    for kw in bad:
        with pytest.raises((ValueError, TypeError, gdn.GdnError)):
            gdn.gdn_add_rmsnorm(x, w, **kw)
    for a, b in ((x[0], w), (x.long(), w), (x, w[:63]), (x, w.half()), (x.expand(4, 64)[:, ::2], w)):
        with pytest.raises((ValueError, TypeError, gdn.GdnError)):
            gdn.gdn_add_rmsnorm(a, b, out=out)
    assert torch.equal(x, x0) and torch.equal(r, r0)
