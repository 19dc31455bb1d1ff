"""Host-side refusals and sizes of gdn_rope, gdn_rope_frequencies, gdn_attn_prefill and gdn_attn_shared through the C
ABI, with addresses that are never used."""

import ctypes
import math

import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from gated_delta_net_causal_gb300 import _build
from tests import attn_reference as ref

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer validation runs only without a GPU")
OK, INVALID, EXTENT, UNSUPPORTED, ALIAS, ALIGN = 0, 1, 2, 3, 4, 5
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.library()


def test_version(lib):
    assert gdn.gdn_version() >= 600


# ------------------------------------------------------------------ frequencies


@pytest.mark.parametrize("rotary,base", [(128, 10000.0), (2, 500000.0), (42, 1e6), (64, 1.5)])
@pytest.mark.parametrize("scaling", [dict(scaling="plain"), dict(scaling="linear", factor=4.0),
                                     dict(scaling="bands", factor=8.0, length=8192, low=1.0, high=4.0),
                                     dict(scaling="ramp", factor=16.0, length=4096, low=1.0, high=32.0)])
def test_steps_are_the_frequencies_in_turns(lib, rotary, base, scaling):
    kind = {"plain": gdn.GDN_ROPE_PLAIN, "linear": gdn.GDN_ROPE_LINEAR, "bands": gdn.GDN_ROPE_BANDS,
            "ramp": gdn.GDN_ROPE_RAMP}[scaling["scaling"]]
    t = gdn.rope_spec(rotary, base=base, scaling=kind, factor=scaling.get("factor", 1.0),
                      original_length=scaling.get("length", 0.0), low=scaling.get("low", 0.0),
                      high=scaling.get("high", 0.0), amplitude=1.25)
    want = ref.frequencies(rotary, base, **scaling)
    assert t.rotary_dim == rotary and t.amplitude == 1.25 and t.layout == gdn.GDN_ROPE_HALF
    for i, f in enumerate(want):  # a few roundings of fp64 apart
        assert abs(t.step[i] / 2.0 ** 64 - f / (2 * math.pi)) <= 16 * 2.0 ** -53 * f / (2 * math.pi) + 2.0 ** -63
    assert all(t.step[i] == 0 for i in range(rotary // 2, 64))


FREQ = dict(rotary=64, layout=0, base=1e4, scaling=0, factor=1.0, length=4096.0, low=1.0, high=4.0, amplitude=1.0)


def freq(lib, out=True, **kw):
    a = FREQ | kw
    t = gdn.GdnRopeTable()
    return lib.gdn_rope_frequencies(a["rotary"], a["layout"], a["base"], a["scaling"], a["factor"], a["length"], a["low"],
                                    a["high"], a["amplitude"], ctypes.byref(t) if out else None)


def test_frequency_refusals(lib):
    assert freq(lib) == OK and freq(lib, out=False) == INVALID
    for r in (0, -2, 1, 63, 130):
        assert freq(lib, rotary=r) == INVALID, r
    assert freq(lib, layout=2) == INVALID and freq(lib, layout=-1) == INVALID
    assert freq(lib, scaling=4) == INVALID and freq(lib, scaling=-1) == INVALID
    for b in (1.0, 0.0, -3.0, INF, NAN):
        assert freq(lib, base=b) == INVALID, b
    for a in (INF, NAN, 1e300):
        assert freq(lib, amplitude=a) == INVALID
    for s in (1, 2, 3):
        for f in (0.0, -1.0, INF, NAN):
            assert freq(lib, scaling=s, factor=f) == INVALID, (s, f)
    assert freq(lib, factor=0.0, length=0.0, low=9.0) == OK  # a plain one uses none of them
    for s in (2, 3):
        for kw in (dict(length=0.0), dict(length=INF), dict(low=0.0), dict(low=4.0), dict(high=INF), dict(high=NAN)):
            assert freq(lib, scaling=s, **kw) == INVALID, (s, kw)


# ------------------------------------------------------------------ rotary calls

MB = 1 << 20
ROPE = dict(tokens=3, pos=1 * MB, q=2 * MB, qs=4096, qo=3 * MB, qos=4096, k=4 * MB, ks=1024, ko=5 * MB, kos=1024, v=None,
            vs=0, vo=None, vos=0, rows=None, n=0, flags=0)


def rope(lib, d, table="own", **kw):
    a = ROPE | kw
    t = gdn.rope_spec(128) if table == "own" else table
    return lib.gdn_rope(ctypes.byref(d) if d is not None else None, ctypes.byref(t) if t is not None else None,
                        a["tokens"], a["pos"], a["q"], a["qs"], a["qo"], a["qos"], a["k"], a["ks"], a["ko"], a["kos"],
                        a["v"], a["vs"], a["vo"], a["vos"], a["rows"], a["n"], a["flags"], None)


CACHE = dict(v=6 * MB, vs=1024, vo=7 * MB, vos=1024, rows=8 * MB, n=100)


@no_gpu
def test_rope_refusals(lib):
    d = gdn.dims(8, 32, 128)
    assert rope(lib, None) == INVALID and rope(lib, d, table=None) == INVALID
    assert rope(lib, gdn.dims(8, 32, 80)) == UNSUPPORTED
    assert rope(lib, d, tokens=-1) == INVALID and rope(lib, d, tokens=2 ** 31) == EXTENT
    assert rope(lib, d, tokens=0) == OK and rope(lib, d, tokens=0, pos=None, q=None, qo=None, k=None, ko=None) == OK
    assert rope(lib, gdn.dims(8, 32, 64), qs=2048, qos=2048) == INVALID  # rotary_dim past the head
    assert rope(lib, d, table=gdn.GdnRopeTable()) == INVALID
    assert rope(lib, d, flags=2) == INVALID
    for name in ("pos", "q", "qo", "k", "ko"):
        assert rope(lib, d, **{name: None}) == INVALID, name
    assert rope(lib, d, q=None, qo=None, k=None, ko=None) == INVALID
    assert rope(lib, d, **CACHE | dict(rows=None)) == INVALID  # v without a cache
    assert rope(lib, d, **CACHE | dict(vo=None)) == INVALID
    assert rope(lib, d, **CACHE | dict(n=-1)) == INVALID
    assert rope(lib, d, **CACHE | dict(n=2 ** 31)) == EXTENT
    for name, width in (("qs", 4096), ("qos", 4096), ("ks", 1024), ("kos", 1024)):
        assert rope(lib, d, **{name: width - 8}) == INVALID, name
        assert rope(lib, d, **{name: width + 4}) == ALIGN, name
    for name in ("pos", "q", "qo", "k", "ko"):
        assert rope(lib, d, **{name: ROPE[name] + 8}) == ALIGN, name
    assert rope(lib, d, **CACHE | dict(rows=8 * MB + 4)) == ALIGN


@no_gpu
def test_rope_overlaps(lib):
    d = gdn.dims(8, 32, 128)
    assert rope(lib, d, qo=ROPE["q"] + 16) == ALIAS
    assert rope(lib, d, qo=ROPE["q"], qos=4104) == ALIAS  # in place needs the same stride
    assert rope(lib, d, qo=ROPE["k"]) == ALIAS and rope(lib, d, ko=ROPE["q"]) == ALIAS
    assert rope(lib, d, ko=ROPE["qo"]) == ALIAS
    assert rope(lib, d, qo=ROPE["pos"]) == ALIAS
    assert rope(lib, d, **CACHE | dict(ko=ROPE["k"])) == ALIAS  # rows of a cache are not the tokens' own
    assert rope(lib, d, **CACHE | dict(vo=CACHE["v"])) == ALIAS
    assert rope(lib, d, **CACHE | dict(vo=ROPE["ko"] + 99 * 2048)) == ALIAS  # the cache's last row


# ------------------------------------------------------------------ attention calls

ATTN = dict(n=2, cu=1 * MB, tokens=5, q=2 * MB, qs=4096, k=3 * MB, ks=1024, v=4 * MB, vs=1024, rows=5, start=None,
            len=None, scale=0.1, out=5 * MB, lse=6 * MB, ws=1 << 32, wb=1 << 40)
SHARED = ATTN | dict(rows=100, start=7 * MB, len=8 * MB, groups=1, gcu=9 * MB, ps=10 * MB, pl=11 * MB)


def attn(lib, d, **kw):
    a = ATTN | kw
    return lib.gdn_attn_prefill(ctypes.byref(d) if d is not None else None, a["n"], a["cu"], a["tokens"], a["q"], a["qs"],
                                a["k"], a["ks"], a["v"], a["vs"], a["rows"], a["start"], a["len"], a["scale"], a["out"],
                                a["lse"], a["ws"], a["wb"], None)


def shared(lib, d, **kw):
    a = SHARED | kw
    return lib.gdn_attn_shared(ctypes.byref(d) if d is not None else None, a["n"], a["cu"], a["tokens"], a["q"], a["qs"],
                               a["k"], a["ks"], a["v"], a["vs"], a["rows"], a["start"], a["len"], a["groups"], a["gcu"],
                               a["ps"], a["pl"], a["scale"], a["out"], a["lse"], a["ws"], a["wb"], None)


@no_gpu
@pytest.mark.parametrize("call,base", [(attn, ATTN), (shared, SHARED)])
def test_attention_refusals(lib, call, base):
    d = gdn.dims(8, 32, 128)
    assert call(lib, None) == INVALID
    assert call(lib, gdn.dims(8, 32, 80)) == UNSUPPORTED
    assert call(lib, gdn.dims(1, 65, 128), qs=65 * 128) == UNSUPPORTED  # more query heads than a tile has rows
    assert call(lib, gdn.dims(8, 12, 128)) == INVALID
    assert call(lib, d, n=-1) == INVALID and call(lib, d, tokens=-1) == INVALID
    assert call(lib, d, n=65536) == EXTENT and call(lib, d, tokens=2 ** 31 - 1024) == EXTENT
    assert call(lib, d, rows=2 ** 31, start=7 * MB, len=8 * MB) == EXTENT
    assert call(lib, d, tokens=0) == OK and call(lib, d, tokens=0, n=0, cu=None, q=None, out=None) == OK
    assert call(lib, d, n=0) == INVALID  # tokens of no sequence
    for name in ("cu", "q", "k", "v", "out"):
        assert call(lib, d, **{name: None}) == INVALID, name
    for s in (0.0, -0.1, INF, NAN):
        assert call(lib, d, scale=s) == INVALID, s
    for name, width in (("qs", 4096), ("ks", 1024), ("vs", 1024)):
        assert call(lib, d, **{name: width - 8}) == INVALID, name
        assert call(lib, d, **{name: width + 4}) == ALIGN, name
        assert call(lib, d, **{name: 1 << 40}) == EXTENT, name
    for name in ("cu", "q", "k", "v", "out", "lse"):
        assert call(lib, d, **{name: base[name] + 4}) == ALIGN, name
    assert call(lib, d, ws=base["ws"] + 128) == ALIGN
    assert call(lib, d, wb=1024) == INVALID
    for name in ("cu", "q", "k", "v", "lse", "ws"):
        assert call(lib, d, out=base[name]) == ALIAS, name
    for name in ("cu", "q", "k", "v"):
        assert call(lib, d, lse=base[name]) == ALIAS, name


@no_gpu
def test_key_stretches(lib):
    d = gdn.dims(8, 32, 128)
    assert attn(lib, d, rows=6) == INVALID  # own rows: as many keys as tokens
    assert attn(lib, d, start=7 * MB) == INVALID and attn(lib, d, len=7 * MB) == INVALID
    assert attn(lib, d, start=7 * MB + 4, len=8 * MB) == ALIGN
    assert attn(lib, d, start=5 * MB, len=8 * MB) == ALIAS
    assert shared(lib, d, start=None) == INVALID and shared(lib, d, len=None) == INVALID


@no_gpu
def test_group_refusals(lib):
    d = gdn.dims(8, 32, 128)
    assert shared(lib, d, ws=None) == INVALID
    assert shared(lib, d, groups=-1) == INVALID and shared(lib, d, groups=65536) == EXTENT
    for name in ("gcu", "ps", "pl"):
        assert shared(lib, d, **{name: None}) == INVALID, name
        assert shared(lib, d, **{name: SHARED[name] + 8}) == ALIGN, name
        assert shared(lib, d, lse=SHARED[name]) == ALIAS, name


def test_workspace_sizes(lib):
    d = gdn.dims(8, 32, 128)
    assert gdn.gdn_attn_prefill_workspace_size(d, 3, 0) == 0
    sizes = [gdn.gdn_attn_prefill_workspace_size(d, 3, t) for t in (1, 4, 64, 100000)]
    assert 0 < sizes[0] <= sizes[1] <= sizes[2] <= sizes[3] < 64 << 20
    more = gdn.gdn_attn_shared_workspace_size(d, 3, 64, 1) - sizes[2]
    assert 2 * 64 * 32 * 129 * 4 <= more <= 2 * 64 * 32 * 129 * 4 + 1024
    for f in (lambda: gdn.gdn_attn_prefill_workspace_size(gdn.dims(1, 65, 128), 1, 1),
              lambda: gdn.gdn_attn_prefill_workspace_size(d, 65536, 1),
              lambda: gdn.gdn_attn_shared_workspace_size(d, 1, 1, -1)):
        with pytest.raises(gdn.GdnError):
            f()
    n = ctypes.c_int64(7)
    assert lib.gdn_attn_prefill_workspace_size(ctypes.byref(d), 1, 1, None) == INVALID
    assert lib.gdn_attn_shared_workspace_size(None, 1, 1, 1, ctypes.byref(n)) == INVALID


# ------------------------------------------------------------------ the binding's checks


def test_binding_refusals(monkeypatch):
    """What the binding itself looks at, on CPU tensors that stand for the current device's."""
    monkeypatch.setattr(gdn, "_current_device", lambda: -1)
    bf = torch.bfloat16
    d, t = gdn.dims(2, 4, 64, io_dtype=bf), gdn.rope_spec(64)
    z = lambda *s, dt=bf: torch.zeros(s, dtype=dt)
    pos, q, k = z(3, dt=torch.int32), z(3, 256), z(3, 128)
    for kw in (dict(q=q, q_out=z(2, 256)), dict(q=z(3, 255), q_out=q), dict(q=q.float(), q_out=q), dict(k=k, k_out=z(3, 64)),
               dict(), dict(k=k, cache_rows=pos), dict(k=k, k_out=z(9, 128), cache_rows=z(2, dt=torch.int32)),
               dict(k=k, k_out=z(9, 128), cache_rows=z(3, dt=torch.int64))):
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_rope(d, t, pos, **kw)
    with pytest.raises(TypeError):
        gdn.gdn_rope(d, t, pos.long(), q=q, q_out=q)
    cu, out = torch.tensor([0, 3], dtype=torch.int32), z(3, 4, 64)
    i = lambda n: z(n, dt=torch.int32)
    for args, kw in (((cu, z(3, 250), k, k, out), {}), ((cu, q, k, z(2, 128), out), {}), ((cu, q, k, k, z(2, 4, 64)), {}),
                     ((cu.long(), q, k, k, out), {}), ((cu, q, k, k, out), dict(lse=z(3, 4))),
                     ((cu, q, k, k, out), dict(kv_start=i(2), kv_len=i(1))), ((cu, q, k, k, out), dict(workspace="own"))):
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_attn_prefill(d, *args, **kw)
    with pytest.raises(ValueError):
        gdn.gdn_attn_shared(d, cu, q, k, k, i(1), i(1), i(2), i(2), i(2), out)


def test_workspaces_belong_to_the_calls_stream(monkeypatch):
    """What the binding allocates by itself is allocated on the stream that the call runs on."""
    import contextlib

    seen, current = [], ["current"]

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    real = torch.empty

    def empty(*a, **kw):
        if kw.get("dtype") == torch.uint8:
            seen.append(current[-1])
        return real(*a, **kw)

    class Library:
        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(gdn, "library", Library)
    monkeypatch.setattr(gdn, "_current_device", lambda: -1)
    monkeypatch.setattr(gdn, "_current_raw_stream", lambda dev: 0)
    for name in ("gdn_attn_prefill_workspace_size", "gdn_attn_shared_workspace_size"):
        monkeypatch.setattr(gdn, name, lambda *a: 4096)
    bf, i = torch.bfloat16, lambda *x: torch.tensor(x, dtype=torch.int32)
    d, z = gdn.dims(1, 2, 64, io_dtype=bf), lambda *s: torch.zeros(s, dtype=bf)
    for s, want in ((None, "current"), (7, ("external", 7))):
        gdn.gdn_attn_prefill(d, i(0, 3), z(3, 128), z(3, 64), z(3, 64), z(3, 2, 64), stream=s)
        gdn.gdn_attn_shared(d, i(0, 3), z(3, 128), z(9, 64), z(9, 64), i(0), i(5), i(0, 3), i(5), i(2), z(3, 2, 64), stream=s)
        assert seen == [want, want]
        seen.clear()
