"""Host-side refusals of gdn_decay_step, gdn_decay_prefill, gdn_add_rmsnorm and
gdn_linear_fp8 through the C ABI, with addresses that are never used."""

import ctypes

import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from gated_delta_net_causal_gb300 import _build

# fake device addresses are only safe where no launch can happen at all
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer validation runs only without a GPU")
OK, INVALID, EXTENT, UNSUPPORTED, ALIAS, ALIGN = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.library()


def test_version(lib):
    assert gdn.gdn_version() >= 500


STEP = dict(batch=2, slots=None, num=2, q=0x100000, qs=2048, k=0x200000, ks=2048, v=0x300000, vs=4096, g=0x400000, gs=0,
            scale=0.1, state=0x10000000, core=0x500000, z=None, zs=0, w=None, out=None)


def step(lib, d, **kw):
    a = STEP | kw
    return lib.gdn_decay_step(ctypes.byref(d) if d is not None else None, a["batch"], a["slots"], a["num"], a["q"],
                              a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["g"], a["gs"], a["scale"], a["state"],
                              a["core"], a["z"], a["zs"], a["w"], a["out"], None)


def test_step_refusals(lib):
    d = gdn.dims(16, 32, 128)
    assert step(lib, None) == INVALID
    assert step(lib, gdn.dims(3, 4, 128)) == INVALID
    assert step(lib, gdn.dims(16, 32, 80)) == UNSUPPORTED
    assert step(lib, d, batch=-1) == INVALID and step(lib, d, num=-1) == INVALID
    assert step(lib, d, num=3) == INVALID  # without a table: one state per row
    assert step(lib, d, batch=70000, num=70000) == EXTENT
    assert step(lib, d, batch=0, num=0) == OK  # nothing launched
    for name in ("q", "k", "v", "g", "state"):
        assert step(lib, d, **{name: None}) == INVALID, name
    assert step(lib, d, core=None) == INVALID  # no output
    assert step(lib, d, z=0x600000, zs=4096, w=0x700000) == INVALID  # z without out
    assert step(lib, d, out=0x800000, z=0x600000, zs=4096) == INVALID  # z without norm_w
    assert step(lib, d, out=0x800000, w=0x600000) == INVALID  # norm_w without z
    for s in (float("inf"), float("nan")):
        assert step(lib, d, scale=s) == INVALID
    for name, least in (("qs", 2047), ("ks", 2047), ("vs", 4095), ("gs", 31), ("gs", -1)):
        assert step(lib, d, **{name: least}) == INVALID, name
    assert step(lib, d, qs=2052) == ALIGN
    assert step(lib, d, out=0x800000, z=0x600000, zs=4100, w=0x700000) == ALIGN
    for name in ("q", "k", "v", "g", "state", "core"):
        assert step(lib, d, **{name: STEP[name] + 8}) == ALIGN, name
    assert step(lib, d, slots=0x900004) == ALIGN
    assert step(lib, d, qs=1 << 61) == EXTENT
    for name in ("q", "k", "v", "g"):
        assert step(lib, d, core=STEP[name]) == ALIAS, name
        assert step(lib, d, state=STEP[name]) == ALIAS, name
    assert step(lib, d, core=0x10000000 + 4096) == ALIAS
    assert step(lib, d, slots=0x900000, core=0x900000) == ALIAS
    # the pool's size, not the batch, is the state's extent: slot 40 of 41 reaches the output
    assert step(lib, d, slots=0x900000, num=41, core=0x10000000 + 40 * 32 * 128 * 128 * 4) == ALIAS


PRE = dict(n=2, cu=0x900000, total=100, q=0x1000000, qs=2048, k=0x2000000, ks=2048, v=0x3000000, vs=4096, g=0x400000,
           gs=32, scale=0.1, state=0x10000000, core=0x5000000, z=None, zs=0, w=None, out=None, ws=None, wsb=0)


def prefill(lib, d, **kw):
    a = PRE | kw
    return lib.gdn_decay_prefill(ctypes.byref(d), a["n"], a["cu"], a["total"], a["q"], a["qs"], a["k"], a["ks"], a["v"],
                                 a["vs"], a["g"], a["gs"], a["scale"], a["state"], a["core"], a["z"], a["zs"], a["w"],
                                 a["out"], a["ws"], a["wsb"], None)


def test_prefill_refusals(lib):
    d = gdn.dims(16, 32, 128)
    assert prefill(lib, d, n=-1) == INVALID and prefill(lib, d, total=-1) == INVALID
    assert prefill(lib, d, n=0) == INVALID  # tokens without a sequence
    assert prefill(lib, d, n=70000) == EXTENT and prefill(lib, d, total=2 ** 31) == EXTENT
    assert prefill(lib, d, total=0) == OK and prefill(lib, d, n=0, total=0) == OK  # nothing launched
    for name in ("cu", "q", "k", "v", "g", "state"):
        assert prefill(lib, d, **{name: None}) == INVALID, name
    assert prefill(lib, d, core=None) == INVALID
    assert prefill(lib, d, cu=0x900004) == ALIGN and prefill(lib, d, vs=4097) == ALIGN
    assert prefill(lib, d, core=PRE["cu"]) == ALIAS
    assert prefill(lib, d, core=PRE["q"] + 99 * 2048 * 2) == ALIAS  # the last row
    total = 4096
    need = gdn.gdn_decay_prefill_workspace_size(d, 1, total)
    assert need > 0
    big = dict(n=1, total=total, v=0x4000000, core=0x8000000, state=0x100000000, ws=0x200000000, wsb=need)
    assert prefill(lib, d, **(big | {"wsb": need - 1})) == INVALID
    assert prefill(lib, d, **(big | {"ws": 0x200000080})) == ALIGN
    for at in (PRE["q"], 0x8000000, 0x100000000):
        assert prefill(lib, d, **(big | {"ws": at})) == ALIAS


def test_workspace_size(lib):
    d = gdn.dims(16, 32, 128)
    assert gdn.gdn_decay_prefill_workspace_size(d, 1, 0) == 0
    assert gdn.gdn_decay_prefill_workspace_size(d, 0, 0) == 0
    assert gdn.gdn_decay_prefill_workspace_size(d, 64, 64 * 512) == 0  # enough (sequence, head) pairs
    for bad in ((-1, 5), (1, -5), (0, 5), (70000, 5), (1, 2 ** 31)):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_decay_prefill_workspace_size(d, *bad)
    assert lib.gdn_decay_prefill_workspace_size(ctypes.byref(d), 1, 5, None) == INVALID


NORM = dict(rows=4, cols=64, io=1, x=0x10000, xs=64, r=0x20000, rs=64, s=0x30000, ss=64, w=0x40000, eps=1e-6, out=0x50000,
            os=64, q=0x60000, qs=64, sc=0x70000)


def norm(lib, **kw):
    a = NORM | kw
    return lib.gdn_add_rmsnorm(*[a[n] for n in NORM], None)


def test_norm_refusals(lib):
    assert norm(lib, io=3) == INVALID and norm(lib, rows=-1) == INVALID and norm(lib, cols=0) == INVALID
    assert norm(lib, rows=2 ** 31) == EXTENT and norm(lib, cols=2 ** 30 + 1) == EXTENT
    assert norm(lib, rows=0) == OK
    assert norm(lib, eps=-1.0) == INVALID and norm(lib, eps=float("inf")) == INVALID
    assert norm(lib, x=None) == INVALID and norm(lib, sc=None) == INVALID and norm(lib, q=None) == INVALID
    assert norm(lib, s=None, out=None, q=None, sc=None) == INVALID
    for name in ("xs", "rs", "ss", "os", "qs"):
        assert norm(lib, **{name: 63}) == INVALID, name
    for name in ("x", "r", "s", "w", "out", "q", "sc"):
        assert norm(lib, **{name: NORM[name] + 4}) == ALIGN, name
    assert norm(lib, xs=1 << 62) == EXTENT
    for o in ("out", "q", "sc"):
        for i in ("x", "r", "w", "s"):
            assert norm(lib, **{o: NORM[i]}) == ALIAS, (o, i)
    assert norm(lib, s=NORM["w"]) == ALIAS
    assert norm(lib, s=NORM["x"], ss=72) == ALIAS  # in place with another stride
    assert norm(lib, s=NORM["r"] + 128) == ALIAS


LIN = dict(M=4, N=64, K=64, x=0x10000, xs=64, xsc=0x20000, w=0x30000, wsc=0x40000, b=0x50000, dt=1, y=0x60000, ys=64)


def linear(lib, **kw):
    a = LIN | kw
    return lib.gdn_linear_fp8(*[a[n] for n in LIN], None)


def test_linear_refusals(lib):
    for kw in (dict(M=0), dict(N=0), dict(K=0), dict(K=24), dict(dt=3), dict(x=None), dict(xsc=None), dict(w=None),
               dict(wsc=None), dict(y=None), dict(xs=48), dict(xs=72), dict(ys=56), dict(ys=68)):
        assert linear(lib, **kw) == INVALID, kw
    assert linear(lib, M=2 ** 22 + 1) == EXTENT and linear(lib, N=2 ** 24 + 1, ys=2 ** 25) == EXTENT
    assert linear(lib, K=2 ** 24 + 16, xs=2 ** 25) == EXTENT and linear(lib, xs=1 << 41) == EXTENT
    for name in ("x", "xsc", "w", "wsc", "b", "y"):
        assert linear(lib, **{name: LIN[name] + 8}) == ALIGN, name
    for name in ("x", "xsc", "w", "wsc", "b"):
        assert linear(lib, y=LIN[name]) == ALIAS, name
