"""gdn_attn_prefill and gdn_attn_shared against fp64 in every row of long sequences, fp32's accuracy there, cumulated
lengths outside of the tokens, and a cache whose rows hold keys and values side by side."""

import numpy as np
import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from tests import attn_reference as ref
from tests.test_gpu_attn import Case, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    yield
    assert gdn.gdn_device_error() == 0


def every_row(c, scale):
    """For each sequence and head: the rows' outputs and lse in fp64, and what their bounds (attn_reference) are made of:
    the weights' mean of the values' magnitudes, and the largest error of an exponent."""
    at = 0
    for n, m, start in zip(c.lengths, c.keys, c.start):
        K, V = (x[start:start + m].double().reshape(m, c.hk, c.D) for x in (c.k, c.v))
        see = torch.arange(m, device="cuda")[None, :] <= (m - n + torch.arange(n, device="cuda"))[:, None]
        for h in range(c.hq):
            kh = ref.head_of(h, c.hq, c.hk, c.tiled)
            q, k, v = c.q[at:at + n].double().reshape(n, c.hq, c.D)[:, h], K[:, kh], V[:, kh]
            s = (scale * (q @ k.T)).masked_fill(~see, -np.inf)
            e = scale * (q.abs() @ k.abs().T) * (c.D + 4) * 2.0 ** -23
            top = s.amax(1, keepdim=True)
            e = (e + 4 * 2.0 ** -24 * (s.abs() + top.abs())).masked_fill(~see, 0.0).amax(1)
            w = torch.exp(s - top)
            total = w.sum(1)
            w /= total[:, None]
            yield at, n, m, h, w @ v, w @ v.abs(), e, (top[:, 0] + torch.log(total))
        at += n


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lengths,keys,hq,hk,D", [
    ([4133], None, 4, 2, 128), ([3001, 5, 2500], None, 4, 1, 64), ([2111, 700], [2111, 5000], 3, 1, 96),
    ([300], [9000], 6, 1, 32)])
def test_every_row_of_long_sequences(dtype, lengths, keys, hq, hk, D):
    """The bounds of attn_reference; below fp16's normal range a weight is off by 2^-25 of a largest one of at least 1."""
    c = Case(31, lengths, keys, hq, hk, D, dtype, tiled=D == 128)
    c.run()
    u = ref.UNIT[dtype]
    for at, n, m, h, o, mag, e, lse in every_row(c, D ** -0.5):
        rel = 2 * e[:, None] + 2.0 ** -21 + (m + 4) * 2.0 ** -22 + (0 if dtype == "f32" else u)
        err = mag * rel + (0 if dtype == "f32" else 2 * ref.SMALLEST[dtype] * m * 6)  # |v| below 6
        tol = err + u * (o.abs() + err) + ref.SMALLEST[dtype]
        got = c.out[at:at + n, h].double()
        assert ((got - o).abs() <= tol).all(), (at, h, float(((got - o).abs() - tol).max()))
        ltol = e + (m + 4) * 2.0 ** -23 + 4 * 2.0 ** -24 * (lse.abs() + 8) + 2.0 ** -21
        assert ((c.lse[at:at + n, h].double() - lse).abs() <= ltol).all(), (at, h)


@pytest.mark.parametrize("lengths,keys,workspace,limit", [
    ([2066], None, "auto", 2.0 ** -18), ([300], [9000], "auto", 2.0 ** -18),
    ([1, 1, 1], [20000, 3, 9001], "auto", 2.0 ** -18), ([1, 1], [20000, 9001], None, 2.0 ** -17)])
def test_f32_is_fp32_throughout(lengths, keys, workspace, limit):
    """The error's norm relative to the outputs'. A rounding is off by 0.4 2^-24 of the value on average (rms). A score
    is a chain of D of them on partial sums that grow with their root: 0.4 2^-24 1.5 D / sqrt(2) for queries of 1.5,
    times the scale 4.8 2^-24 at D = 128; with the exponent's (scores of up to 10) and the exponential's own about
    6 2^-24, relative in a weight and, the errors of different keys being independent, in the output. A sum of m keys in
    one go adds at most 0.4 sqrt(m) 2^-24: 18 for 2066, 57 for 20,000 (without a workspace). So 20 and 58, below a third
    and a half of the limits, where a rounding to 16 bits anywhere would be 2^-13 and more."""
    c = Case(32, lengths, keys, 4, 1, 128, "f32")
    c.run(workspace=workspace)
    off = size = 0.0
    for at, n, m, h, o, mag, e, lse in every_row(c, 128 ** -0.5):
        off += float(((c.out[at:at + n, h].double() - o) ** 2).sum())
        size += float((o ** 2).sum())
        # lse: the factor of the scores, their product, the logarithm's sum, the way back, and the exponentials'
        assert ((c.lse[at:at + n, h].double() - lse).abs() <= 4 * 2.0 ** -24 * (lse.abs() + 8) + 2.0 ** -20).all()
    assert (off / size) ** 0.5 <= limit, (off / size) ** 0.5 * 2 ** 24


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_cu_seqlens_past_the_tokens(dtype):
    """A sequence whose end lies before its start has no tokens; the next one, that ends past the last token, has the
    tokens that there are. Rows before it are left alone."""
    c = Case(33, [4, 4], [40, 50], 4, 2, 64, dtype)
    c.cu = ints([8, 4, 2 ** 31 - 1])
    c.run()
    k, v = (ref.f64(x[c.start[1]:c.start[1] + 50]).reshape(50, 2, 64) for x in (c.k, c.v))
    o, tol, l, ltol = ref.attention(ref.f64(c.q[4:]).reshape(4, 4, 64), k, v, ref.causal(4, 50), 64 ** -0.5, dtype)
    ref.check(ref.f64(c.out[4:]), o, tol, "out")
    ref.check(ref.f64(c.lse[4:]), l, ltol, "lse")
    assert (c.out[:4] == 7.25).all() and (c.lse[:4] == 7.25).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_keys_and_values_side_by_side_in_a_cache(dtype):
    """gdn_rope writes keys and values to column slices of one row, the attention call reads them there."""
    hq, hk, D, rows = 6, 2, 96, 90
    io, gen = ref.DT[dtype], torch.Generator().manual_seed(34)
    cache = torch.full((rows, 2 * hk * D + 24), 7.25, device="cuda", dtype=io)
    kc, vc = cache[:, 8:8 + hk * D], cache[:, 16 + hk * D:16 + 2 * hk * D]
    T, first = 70, 11
    act = torch.randn((T, (hq + 2 * hk) * D), generator=gen).to(io).cuda()
    q, k, v = act[:, :hq * D], act[:, hq * D:(hq + hk) * D], act[:, (hq + hk) * D:]
    d, table, pos = gdn.dims(hk, hq, D, io_dtype=io), gdn.rope_spec(D), torch.arange(T, dtype=torch.int32, device="cuda")
    gdn.gdn_rope(d, table, pos, k=k, k_out=kc, v=v, v_out=vc, cache_rows=pos + first)
    want, tol = ref.rotate(ref.f64(k).reshape(T, hk, D), np.arange(T), ref.frequencies(D, 10000.0), False, 1.0, dtype)
    ref.check(ref.f64(kc[first:first + T]).reshape(T, hk, D), want, tol, "k")
    assert torch.equal(vc[first:first + T], v)
    rest = torch.ones_like(cache, dtype=torch.bool)
    rest[first:first + T, 8:8 + hk * D] = rest[first:first + T, 16 + hk * D:16 + 2 * hk * D] = False
    assert (cache[rest] == 7.25).all()
    out = torch.empty((T, hq, D), device="cuda", dtype=io)
    gdn.gdn_attn_prefill(d, ints([0, T]), q, kc, vc, out, kv_start=ints([first]), kv_len=ints([T]))
    K, V = (ref.f64(x[first:first + T]).reshape(T, hk, D) for x in (kc, vc))
    o, tol, _, _ = ref.attention(ref.f64(q).reshape(T, hq, D), K, V, ref.causal(T, T), D ** -0.5, dtype)
    ref.check(ref.f64(out), o, tol, "out")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("hq,hk,D,each", [(8, 2, 64, 8), (12, 4, 96, 5), (16, 1, 128, 7), (3, 3, 32, 40)])
def test_groups_of_several_items(dtype, hq, hk, D, each):
    """More query rows of a group than one item holds, groups that end within one, and sequences behind the last."""
    keys = [each + 7 * i % 61 for i in range(23)]
    c = Case(35, [each] * 23, keys, hq, hk, D, dtype, tiled=D == 96, prefixes=[(300, 11), (129, 2), (40, 9)], extra=2)
    c.run_shared()
    c.check(shared=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_calls_side_by_side(dtype):
    """Two captured calls with a workspace each, replayed on two streams at once."""
    cs = [Case(36 + i, [2] * 9, [40 * j + 2 for j in range(9)], 8, 2, 64, dtype, prefixes=[(1500, 5), (64, 4)])
          for i in range(2)]
    streams, graphs, keep = [torch.cuda.Stream() for _ in cs], [], []
    for c, s in zip(cs, streams):
        ws = torch.empty(gdn.gdn_attn_shared_workspace_size(c.d, 9, 18, 2), dtype=torch.uint8, device="cuda")
        groups = (ints([0, 10, 18]), ints([p for p, _, _ in c.prefix]), ints([n for _, n, _ in c.prefix]))
        keep.append((ws, groups))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            gdn.gdn_attn_shared(c.d, c.cu, c.q, c.k, c.v, c.kv["kv_start"], c.kv["kv_len"], *groups, c.out, lse=c.lse,
                                workspace=ws)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c in cs:
        c.check(shared=True)
