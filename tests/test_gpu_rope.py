"""gdn_rope against the rotation in fp64, within bounds made of the inputs' magnitudes (attn_reference)."""

import numpy as np
import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu
KIND = {"plain": gdn.GDN_ROPE_PLAIN, "linear": gdn.GDN_ROPE_LINEAR, "bands": gdn.GDN_ROPE_BANDS,
        "ramp": gdn.GDN_ROPE_RAMP}
SCALING = {"plain": dict(), "linear": dict(factor=4.0), "bands": dict(factor=8.0, length=8192, low=1.0, high=4.0),
           "ramp": dict(factor=8.0, length=4096, low=1.0, high=32.0)}


class Case:
    def __init__(self, seed, T, hq, hk, D, rotary, dtype="bf16", interleaved=False, scaling="plain", amplitude=1.0,
                 base=10000.0, farthest=100000, pad=0):
        gen = torch.Generator().manual_seed(seed)
        io, a = ref.DT[dtype], SCALING[scaling]
        self.T, self.hq, self.hk, self.D, self.dtype, self.interleaved = T, hq, hk, D, dtype, interleaved
        self.amplitude = float(np.float32(amplitude))
        self.freq = ref.frequencies(rotary, base, scaling, **a)
        self.act = torch.randn((T, (hq + 2 * hk) * D + pad), generator=gen).to(io).cuda()
        self.q, self.k = self.act[:, :hq * D], self.act[:, hq * D:(hq + hk) * D]
        self.v = self.act[:, (hq + hk) * D:(hq + 2 * hk) * D]
        self.pos = torch.randint(-farthest, farthest, (T,), generator=gen, dtype=torch.int32).cuda()
        self.d = gdn.dims(hk, hq, D, io_dtype=io)
        self.table = gdn.rope_spec(rotary, layout=gdn.GDN_ROPE_INTERLEAVED if interleaved else gdn.GDN_ROPE_HALF,
                                   base=base, scaling=KIND[scaling], factor=a.get("factor", 1.0),
                                   original_length=a.get("length", 0.0), low=a.get("low", 0.0), high=a.get("high", 0.0),
                                   amplitude=amplitude)

    def want(self, x, inverse=False):
        return ref.rotate(ref.f64(x).reshape(x.shape[0], -1, self.D), ref.f64(self.pos), self.freq, self.interleaved,
                          self.amplitude, self.dtype, inverse)

    def empty(self, rows, heads, pad=0, fill=7.25):
        return torch.full((rows, heads * self.D + pad), fill, device="cuda", dtype=ref.DT[self.dtype])[:, :heads * self.D]

    def check(self, got, x, what, inverse=False):
        y, tol = self.want(x, inverse)
        ref.check(ref.f64(got).reshape(y.shape), y, tol, what)


SHAPES = [(1, 32, 8, 128, 128), (37, 4, 1, 128, 32), (5, 3, 3, 96, 96), (300, 2, 1, 32, 2), (64, 6, 2, 64, 42),
          (17, 1, 1, 96, 34), (700, 16, 2, 128, 64), (2, 64, 64, 32, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hk,D,rotary", SHAPES)
def test_matches_the_rotation(dtype, interleaved, T, hq, hk, D, rotary):
    scaling = list(SCALING)[(T + D) % 4]
    c = Case(T + D, T, hq, hk, D, rotary, dtype, interleaved, scaling, amplitude=1.1 if scaling == "ramp" else 1.0,
             pad=(T % 3) * 8)
    qo, ko = c.empty(T, hq, pad=16), c.empty(T, hk)
    gdn.gdn_rope(c.d, c.table, c.pos, q=c.q, q_out=qo, k=c.k, k_out=ko)
    c.check(qo, c.q, "q")
    c.check(ko, c.k, "k")
    assert (qo.as_strided((T - 1, 16), (hq * D + 16, 1), hq * D) == 7.25).all()  # between the rows


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scaling", list(SCALING))
def test_far_positions(dtype, scaling):
    """The ends of the positions' range: angles of up to 2^31 radians."""
    c = Case(3, 6, 2, 1, 128, 128, dtype, scaling=scaling)
    c.pos.copy_(torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 1, -1, 1 << 30]))
    qo = c.empty(6, 2)
    gdn.gdn_rope(c.d, c.table, c.pos, q=c.q, q_out=qo)
    # numpy's angle is off by 2^-53 of 2^31 too, which the bound's 2^-50 covers
    c.check(qo, c.q, scaling)
    assert torch.equal(qo[2], c.q[2])  # position 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved,D,rotary", [(False, 128, 128), (True, 64, 64), (False, 96, 20), (True, 32, 6)])
def test_cache_rows(dtype, interleaved, D, rotary):
    T, rows = 29, 50
    c = Case(D, T, 6, 3, D, rotary, dtype, interleaved)
    perm = torch.randperm(rows, generator=torch.Generator().manual_seed(1))[:T].to(torch.int32)
    perm[4], perm[11] = -1, -2 ** 31  # padded tokens
    kc, vc, qo = c.empty(rows, 3, pad=8), c.empty(rows, 3), c.empty(T, 6)
    gdn.gdn_rope(c.d, c.table, c.pos, q=c.q, q_out=qo, k=c.k, k_out=kc, v=c.v, v_out=vc, cache_rows=perm.cuda())
    c.check(qo, c.q, "q")
    live = perm >= 0
    y, tol = c.want(c.k)
    ref.check(ref.f64(kc[perm[live].long().cuda()]).reshape(-1, 3, D), y[live.numpy()], tol[live.numpy()], "k")
    assert torch.equal(vc[perm[live].long().cuda()], c.v[live.cuda()])
    rest = torch.ones(rows, dtype=torch.bool)
    rest[perm[live].long()] = False
    for t in (kc, vc):
        assert (t[rest.cuda()] == 7.25).all()
    assert gdn.gdn_device_error() == 0


def test_cache_row_past_the_end_is_skipped_and_recorded():
    c = Case(1, 4, 2, 1, 64, 64)
    kc, vc = c.empty(8, 1), c.empty(8, 1)
    assert gdn.gdn_device_error() == 0
    rows = torch.tensor([3, 8, 2 ** 31 - 1, 0], dtype=torch.int32, device="cuda")
    gdn.gdn_rope(c.d, c.table, c.pos, k=c.k, k_out=kc, v=c.v, v_out=vc, cache_rows=rows)
    assert gdn.gdn_device_error() == 2 and gdn.gdn_device_error() == 0
    assert torch.equal(vc[3], c.v[0]) and torch.equal(vc[0], c.v[3])
    for r in (1, 2, 4, 5, 6, 7):
        assert (vc[r] == 7.25).all() and (kc[r] == 7.25).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved,rotary", [(False, 64), (True, 64), (False, 26)])
def test_in_place_and_back(dtype, interleaved, rotary):
    """In place is the same, bit for bit; the inverse call matches the transposed map, which at amplitude 1 undoes it."""
    c = Case(5, 33, 4, 2, 64, rotary, dtype, interleaved, amplitude=1.5)
    qo, ko, back = c.empty(33, 4), c.empty(33, 2), c.empty(33, 4)
    gdn.gdn_rope(c.d, c.table, c.pos, q=c.q, q_out=qo, k=c.k, k_out=ko)
    gdn.gdn_rope(c.d, c.table, c.pos, q=c.q, q_out=back, inverse=True)
    c.check(back, c.q, "back", inverse=True)
    act = c.act.clone()
    q, k = act[:, :4 * 64], act[:, 4 * 64:6 * 64]
    gdn.gdn_rope(c.d, c.table, c.pos, q=q, q_out=q, k=k, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(act[:, 6 * 64:], c.act[:, 6 * 64:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(interleaved):
    """The gradient of sum(y u) with respect to x is the inverse call on u: against differences. The rotation is linear,
    so a difference over any step is exact but for the roundings of y: 2^-23 of the outputs' magnitudes, of which a
    coordinate of x touches two, over the step of 1."""
    c = Case(8, 3, 2, 1, 32, 24, "f32", interleaved, amplitude=1.2)
    gen = torch.Generator().manual_seed(2)
    u = torch.randn((3, 64), generator=gen).cuda()
    g = torch.empty_like(u)
    gdn.gdn_rope(c.d, c.table, c.pos, q=u, q_out=g, inverse=True)
    y = [torch.empty((3, 64), device="cuda") for _ in range(2)]
    x = c.q.contiguous()
    gdn.gdn_rope(c.d, c.table, c.pos, q=x, q_out=y[0])
    for i in range(0, 64, 5):
        moved = x.clone()
        moved[:, i] += 1.0
        step = moved[:, i].double() - x[:, i].double()
        gdn.gdn_rope(c.d, c.table, c.pos, q=moved, q_out=y[1])
        diff = ((y[1].double() - y[0].double()) * u.double()).sum(1) / step
        tol = 2.0 ** -21 * ((y[0].abs() + y[1].abs() + 2.0) * u.abs()).double().max(1).values * 4
        assert ((diff - g[:, i].double()).abs() <= tol).all(), i


def test_what_is_not_finite_stays_in_its_pair():
    c = Case(9, 2, 1, 1, 64, 32, "f32", True)
    x = c.q.clone()
    x[0, 5], x[1, 40] = float("nan"), float("inf")  # pair 2; past the rotated part
    y, z = c.empty(2, 1), c.empty(2, 1)
    gdn.gdn_rope(c.d, c.table, c.pos, q=x, q_out=y)
    gdn.gdn_rope(c.d, c.table, c.pos, q=c.q, q_out=z)
    assert torch.isnan(y[0, 4:6]).all() and y[1, 40] == float("inf")
    y[0, 4:6] = z[0, 4:6]
    y[1, 40] = z[1, 40]
    assert torch.equal(y, z)


def test_other_stream_and_graph():
    c = Case(10, 40, 8, 2, 128, 128)
    want, qo = c.empty(40, 8), c.empty(40, 8)
    gdn.gdn_rope(c.d, c.table, c.pos, q=c.q, q_out=want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    gdn.gdn_rope(c.d, c.table, c.pos, q=c.q, q_out=qo, stream=s)
    s.synchronize()
    assert torch.equal(qo, want)
    qo.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_rope(c.d, c.table, c.pos, q=c.q, q_out=qo)
    g.replay()
    c.pos += 17
    g.replay()
    torch.cuda.synchronize()
    c.check(qo, c.q, "replayed at other positions")


def test_no_tokens():
    c = Case(11, 1, 2, 1, 64, 64)
    e = torch.empty((0, 128), device="cuda", dtype=torch.bfloat16)
    gdn.gdn_rope(c.d, c.table, torch.empty(0, dtype=torch.int32, device="cuda"), q=e, q_out=torch.empty_like(e))


def test_rows_past_32_bit_offsets():
    """A cache of more than 2^31 elements."""
    rows, D, hk = (1 << 31) // 1024 + 3, 128, 8
    kc = torch.zeros((rows, hk * D), device="cuda", dtype=torch.bfloat16)
    c = Case(12, 2, 8, hk, D, 128)
    at = torch.tensor([rows - 1, 0], dtype=torch.int32, device="cuda")
    gdn.gdn_rope(c.d, c.table, c.pos, k=c.k, k_out=kc, cache_rows=at)
    c.check(kc[at.long()], c.k, "k")
    assert not kc[1:rows - 1].any()
