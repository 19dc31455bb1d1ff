"""gdn_attn_prefill and gdn_attn_shared against softmax attention in fp64, within bounds made of the inputs' magnitudes
(attn_reference)."""

import numpy as np
import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    yield
    assert gdn.gdn_device_error() == 0


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def before(lengths):
    return [0] + list(np.cumsum(lengths))


class Case:
    """lengths: new tokens of each sequence; keys: how many it sees (None: its new tokens, whose q, k and v then are
    slices of one row); prefixes: (keys, sequences) of each group."""

    def __init__(self, seed, lengths, keys, hq, hk, D, dtype="bf16", tiled=False, std=1.5, extra=0, prefixes=()):
        gen = torch.Generator().manual_seed(seed)
        io = ref.DT[dtype]
        n = lambda *s: torch.randn(s, generator=gen)
        self.lengths, self.keys, self.hq, self.hk, self.D, self.dtype, self.tiled = lengths, keys, hq, hk, D, dtype, tiled
        self.tokens = T = sum(lengths)
        self.d = gdn.dims(hk, hq, D, map=gdn.GDN_MAP_TILED if tiled else gdn.GDN_MAP_GROUPED, io_dtype=io)
        self.cu = ints(before(lengths))
        self.own = keys is None
        if self.own:
            act = n(T + extra, (hq + 2 * hk) * D + 8)
            act[:, :hq * D] *= std
            self.act = act.to(io).cuda()
            self.q, self.k = self.act[:, :hq * D], self.act[:, hq * D:(hq + hk) * D]
            self.v = self.act[:, (hq + hk) * D:(hq + 2 * hk) * D]
            self.start, self.keys = before(lengths)[:-1], list(lengths)
            self.kv = {}
        else:
            self.q = (n(T + extra, hq * D) * std).to(io).cuda()
            stretches = list(keys) + [p for p, _ in prefixes]
            order = torch.randperm(len(stretches), generator=gen).tolist()
            at, start = 3, [0] * len(stretches)
            for i in order:
                start[i] = at
                at += stretches[i] + 1 + i % 3  # rows that no token sees lie between
            pool = n(at + 2, 2 * hk * D + 16).to(io).cuda()
            self.k, self.v = pool[:, :hk * D], pool[:, hk * D + 16:]
            self.start = start[:len(keys)]
            self.kv = {"kv_start": ints(self.start), "kv_len": ints(list(keys))}
            self.prefix = [(start[len(keys) + j], p, c) for j, (p, c) in enumerate(prefixes)]
        self.fresh()

    def fresh(self):
        T = self.q.shape[0]
        self.out = torch.full((T, self.hq, self.D), 7.25, device="cuda", dtype=ref.DT[self.dtype])
        self.lse = torch.full((T, self.hq), 7.25, device="cuda")

    def run(self, scale=None, lse=True, **kw):
        gdn.gdn_attn_prefill(self.d, self.cu, self.q, self.k, self.v, self.out, lse=self.lse if lse else None, scale=scale,
                             **self.kv, **kw)

    def run_shared(self, scale=None, **kw):
        members = [c for _, _, c in self.prefix]
        at = before(self.lengths)
        cuts = ints([at[i] for i in before(members)])
        gdn.gdn_attn_shared(self.d, self.cu, self.q, self.k, self.v, self.kv["kv_start"], self.kv["kv_len"], cuts,
                            ints([s for s, _, _ in self.prefix]), ints([p for _, p, _ in self.prefix]), self.out,
                            lse=self.lse, scale=scale, **kw)

    def check(self, scale=None, lse=True, shared=False, only=None):
        scale = self.D ** -0.5 if scale is None else scale
        k, v = (ref.f64(x).reshape(x.shape[0], self.hk, self.D) for x in (self.k, self.v))
        q = ref.f64(self.q).reshape(-1, self.hq, self.D)
        group = [p for p in self.prefix for _ in range(p[2])] if shared else []
        at = 0
        for i, (n, m) in enumerate(zip(self.lengths, self.keys)):
            if n and (only is None or i in only):
                rows = np.arange(self.start[i], self.start[i] + m)
                see = ref.causal(n, m)
                if i < len(group):
                    rows = np.concatenate([np.arange(group[i][0], group[i][0] + group[i][1]), rows])
                    see = np.concatenate([np.ones((n, group[i][1]), bool), see], 1)
                o, tol, l, ltol = ref.attention(q[at:at + n], k[rows], v[rows], see, scale, self.dtype, self.tiled)
                ref.check(ref.f64(self.out[at:at + n]), o, tol, f"out of sequence {i}")
                if lse:
                    ref.check(ref.f64(self.lse[at:at + n]), l, ltol, f"lse of sequence {i}")
            at += n
        assert (self.out[at:] == 7.25).all() and (self.lse[at:] == 7.25).all()  # behind the last sequence
        assert lse or (self.lse == 7.25).all()


SHAPES = [(1, 1, 128), (4, 1, 128), (8, 2, 64), (3, 3, 96), (6, 2, 32), (10, 2, 96), (64, 1, 128)]
OWN = [[1], [2, 1, 3], [5, 0, 130], [128, 129], [300], [0, 7, 0, 64, 257, 0]]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("hq,hk,D", SHAPES)
@pytest.mark.parametrize("i", range(len(OWN)))
def test_prompts(dtype, hq, hk, D, i):
    c = Case(10 * i + D, OWN[i], None, hq, hk, D, dtype, tiled=i % 2 == 1, extra=i % 3)
    c.run(lse=i != 2)
    c.check(lse=i != 2)


CACHED = [([1], [1]), ([1, 1, 1], [700, 1, 129]), ([1] * 9, [128 * j for j in range(9)]), ([5, 17, 130], [2, 500, 130]),
          ([300, 1], [1111, 4000]), ([3, 0, 4], [0, 50, 1]), ([64], [1000])]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("hq,hk,D", SHAPES)
@pytest.mark.parametrize("i", range(len(CACHED)))
def test_cached_keys(dtype, hq, hk, D, i):
    """Single tokens, chunks and prompts on keys of a cache, fewer keys than tokens (rows that see nothing) among them."""
    c = Case(20 * i + D, *CACHED[i], hq, hk, D, dtype, tiled=i % 2 == 0, extra=i % 2)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("hq,hk,D", SHAPES[:5])
@pytest.mark.parametrize("each,keys,prefixes", [
    (1, [5, 1, 300, 64], [(1000, 4)]), (1, [1], [(1, 1)]), (3, [40, 3, 129, 7, 500], [(257, 2), (0, 1), (1300, 1)]),
    (2, [2, 0, 1, 90], [(100, 2), (31, 2)]), (1, [20] * 40, [(2000, 39)])])
def test_shared_prefixes(dtype, hq, hk, D, each, keys, prefixes):
    """One token each and several, an empty prefix, no keys of one's own, sequences outside of all groups."""
    c = Case(D + len(keys), [each] * len(keys), keys, hq, hk, D, dtype, tiled=D == 64, prefixes=prefixes, extra=1)
    c.run_shared()
    c.check(shared=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lengths,keys,hq,hk,D", [
    ([4133], None, 8, 2, 128), ([3001, 5, 2500], None, 8, 1, 64), ([2111, 700], [2111, 5000], 3, 1, 96),
    ([300], [9000], 16, 2, 32), ([1, 1, 1], [20000, 3, 9001], 4, 1, 128)])
def test_long_sequences(dtype, lengths, keys, hq, hk, D):
    """Many tiles in one item and many items in one CTA, twice over; every 97th token and the ends against fp64, the others
    against the second run."""
    if dtype == "f32" and keys is None:
        lengths = [n // 2 for n in lengths]
    c = Case(21, lengths, keys, hq, hk, D, dtype)
    c.run()
    first = c.out.clone(), c.lse.clone()
    c.fresh()
    c.run()
    assert torch.equal(first[0], c.out) and torch.equal(first[1], c.lse)
    at = 0
    for n, m, start in zip(c.lengths, c.keys, c.start):
        some = sorted(set(range(0, n, 97)) | {n - 1, n // 2, max(n - 65, 0)})
        rows = [at + i for i in some]
        k, v = (ref.f64(x[start:start + m]).reshape(m, hk, D) for x in (c.k, c.v))
        o, tol, l, ltol = ref.attention(ref.f64(c.q[rows]).reshape(-1, hq, D), k, v, ref.causal(n, m)[some], D ** -0.5,
                                        dtype)
        ref.check(ref.f64(c.out[rows]), o, tol, "out")
        ref.check(ref.f64(c.lse[rows]), l, ltol, "lse")
        at += n


def test_sequences_that_share_their_keys():
    """The same rows of the cache for several sequences, as forked ones have them."""
    c = Case(22, [1, 1, 4], [500, 500, 500], 8, 2, 64)
    c.start = [c.start[0], c.start[0] + 100, c.start[0]]
    c.keys = [500, 300, 400]
    c.kv = {"kv_start": ints(c.start), "kv_len": ints(c.keys)}
    c.run()
    c.check()


def test_shared_without_groups_is_the_plain_call():
    c = Case(3, [1, 2], [9, 300], 4, 2, 64, prefixes=[])
    z = torch.empty(0, dtype=torch.int32, device="cuda")
    gdn.gdn_attn_shared(c.d, c.cu, c.q, c.k, c.v, c.kv["kv_start"], c.kv["kv_len"], ints([0]), z, z, c.out, lse=c.lse)
    c.check()
    a = c.out.clone()
    c.fresh()
    c.run()
    assert torch.equal(a, c.out)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale", [1e-3, 1.0, 8.0])
def test_scales(dtype, scale):
    """Nearly even weights to nearly a single one."""
    c = Case(4, [200, 33], None, 4, 2, 64, dtype)
    c.run(scale=scale)
    c.check(scale=scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_running_maximum(dtype, order):
    """Scores that rise or fall by hundreds over the keys: every tile moves the maximum, or none after the first."""
    n = 700
    c = Case(5, [n], None, 2, 1, 64, dtype, std=1.0)
    lift = torch.linspace(0, 60, n, device="cuda") * (1 if order == "rising" else -1)
    c.q[:, 0], c.q[:, 64] = 8.0, 8.0
    c.k[:, 0] = lift.to(c.k.dtype)
    c.run()
    c.check()


def test_one_visible_key_gives_its_value():
    """The first token's output is its value, but for the weight's rounding."""
    for dtype in ("f32", "bf16", "f16"):
        c = Case(6, [1, 1, 1], None, 4, 2, 128, dtype)
        c.run()
        want = c.v.reshape(3, 2, 1, 128).expand(3, 2, 2, 128).reshape(3, 4, 128).double()
        assert ((c.out.double() - want).abs() <= 2.1 * ref.UNIT[dtype] * want.abs()).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [32, 64, 96, 128])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("what", ["k", "v"])
def test_not_finite_reaches_only_who_sees_it(dtype, D, bad, what):
    """One key or value of a long sequence, at the start, within and at the end of a tile, and in rows between the
    sequences: tokens before it and other sequences are as without it, bit for bit; in v, tokens from it on have what is
    not finite in its column."""
    n, hq, hk = 450, 6, 2
    for at in (0, 127, 128, 200, 449):
        c = Case(7, [n, 60], [n, 90], hq, hk, D, dtype, prefixes=[(5, 0)])
        c.run()
        clean, clse = c.out.clone(), c.lse.clone()
        t = getattr(c, what)
        t[c.start[0] + at, D + 3] = bad  # key head 1
        for s, m in zip(c.start, c.keys):
            t[s - 1] = bad  # rows that no token sees
            if s + m not in c.start:
                t[s + m] = bad
        c.fresh()
        c.run()
        assert torch.equal(c.out[:at], clean[:at]) and torch.equal(c.lse[:at], clse[:at]), at
        assert torch.equal(c.out[n:], clean[n:])
        assert torch.equal(c.out[:n, :hq // hk], clean[:n, :hq // hk])  # the other key head
        hit = c.out[at:n, hq // hk:].float()
        if what == "v":
            assert not torch.isfinite(hit[:, :, 3]).any()
            hit[:, :, 3] = clean[at:n, hq // hk:, 3].float()
            assert torch.equal(hit, clean[at:n, hq // hk:].float())
        elif bad != bad:
            assert torch.isnan(hit).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("what", ["k", "v"])
def test_not_finite_prefix_reaches_its_group(dtype, what):
    """And a sequence's own keys that are not finite its own tokens, prefix or not."""
    c = Case(7, [1] * 6, [40, 300, 1, 5, 129, 64], 4, 2, 64, dtype, prefixes=[(500, 2), (200, 2)])
    c.run_shared()
    clean = c.out.clone()
    t = getattr(c, what)
    t[c.prefix[0][0] + 321, 64:] = NAN  # key head 1
    t[c.start[3] + 2, :64] = NAN        # key head 0
    t[c.start[4] + 128, :64] = NAN
    for s, m, _ in c.prefix:
        t[s - 1] = t[s + m] = NAN
    c.fresh()
    c.run_shared()
    hit = torch.zeros((6, 4), dtype=torch.bool, device="cuda")
    hit[:2, 2:] = hit[3, :2] = hit[4, :2] = True
    assert torch.isnan(c.out[hit]).all() and torch.equal(c.out[~hit], clean[~hit])


def test_not_finite_query_stays_in_its_row():
    c = Case(8, [200], None, 4, 2, 64)
    c.run()
    clean = c.out.clone()
    c.q[77, 64:128] = NAN
    c.fresh()
    c.run()
    assert torch.isnan(c.out[77, 1]).all()
    c.out[77, 1] = clean[77, 1]
    assert torch.equal(c.out, clean)


def test_lengths_outside_of_the_rows_are_clamped():
    c = Case(9, [4, 4, 4], [8, 8, 8], 2, 1, 64)
    rows = c.k.shape[0]
    c.kv = {"kv_start": ints([-5, rows - 3, rows + 9]), "kv_len": ints([7, 2 ** 31 - 1, 5])}
    c.run()
    torch.cuda.synchronize()
    c.start, c.keys = [0, rows - 3, rows], [7, 3, 0]
    c.check()
    c.kv = {"kv_start": ints([0, 5, 5]), "kv_len": ints([-2, 4, -2 ** 31])}
    c.start, c.keys = [0, 5, 5], [0, 4, 0]
    c.fresh()
    c.run()
    c.check()


def test_cu_seqlens_outside_of_the_tokens_are_clamped():
    c = Case(10, [4, 4], [40, 50], 2, 1, 64)
    c.cu = ints([-3, 4, 100])
    c.run()
    c.check()
    c.cu = ints([8, 4, 2 ** 31 - 1])  # a sequence of no tokens, then one of the rest
    c.lengths, c.start, c.keys = [4], [c.start[1]], [c.keys[1]]
    c.fresh()
    c.run()
    assert (c.out[4:8] != 7.25).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_a_workspace(dtype):
    for lengths, keys in (([1, 1], [3000, 5]), ([70, 300], None)):
        c = Case(11, lengths, keys, 4, 2, 64, dtype)
        c.run(workspace=None)
        c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_workspace_contents_do_not_matter(dtype):
    """And a larger one is as good; the same call twice gives the same bits."""
    c = Case(12, [1, 40, 1], [2500, 700, 3], 8, 2, 128, dtype)
    need = gdn.gdn_attn_prefill_workspace_size(c.d, 3, c.tokens)
    got = []
    for fill in (0, 255):
        c.fresh()
        c.run(workspace=torch.full((need + 512,), fill, dtype=torch.uint8, device="cuda"))
        got.append((c.out, c.lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    c.check()
    with pytest.raises(gdn.GdnError):
        c.run(workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_streams_and_graphs(dtype):
    """Two captured calls with their own workspaces replayed side by side, lengths changed between replays."""
    cs = [Case(13 + i, [1] * 6, [900 + 100 * j for j in range(6)], 8, 2, 128, dtype) for i in range(2)]
    graphs, streams, ws = [], [torch.cuda.Stream() for _ in cs], []
    for c, s in zip(cs, streams):
        ws.append(torch.empty(gdn.gdn_attn_prefill_workspace_size(c.d, 6, 6), dtype=torch.uint8, device="cuda"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.run(workspace=ws[-1])
        graphs.append(g)
    for c in cs:
        c.keys = [1 + 150 * j for j in range(6)]
        c.kv["kv_len"].copy_(ints(c.keys))
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c in cs:
        c.check()
        c.fresh()
    c = cs[0]
    c.run(stream=streams[1])  # scratch of that stream's
    streams[1].synchronize()
    c.check()


def test_shared_captured():
    c = Case(15, [2] * 5, [30, 2, 400, 5, 77], 4, 1, 128, prefixes=[(900, 3), (64, 2)])
    need = gdn.gdn_attn_shared_workspace_size(c.d, 5, 10, 2)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    members, at = [3, 2], before(c.lengths)
    a = (ints([at[i] for i in before(members)]), ints([s for s, _, _ in c.prefix]), ints([p for _, p, _ in c.prefix]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_attn_shared(c.d, c.cu, c.q, c.k, c.v, c.kv["kv_start"], c.kv["kv_len"], *a, c.out, lse=c.lse, workspace=ws)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    c.check(shared=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_many_sequences(dtype):
    """More sequences than threads of a CTA, most of them short."""
    gen = np.random.default_rng(1)
    lengths = [int(x) for x in gen.integers(0, 3, 1500)]
    keys = [int(x) for x in gen.integers(0, 40, 1500)]
    keys[700] = 2000
    c = Case(16, lengths, keys, 2, 1, 32, dtype)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_past_32_bit_offsets(dtype):
    """Keys behind 2^31 elements of a cache."""
    D, hk = 128, 8 if dtype == "bf16" else 4
    rows = (1 << 31) // (hk * D) + 700
    k = torch.zeros((rows, hk * D), device="cuda", dtype=ref.DT[dtype])
    v = torch.zeros_like(k)
    c = Case(17, [3, 1], [300, 200], 16, hk, D, dtype)
    for i in range(2):
        m = c.keys[i]
        to = rows - 310 * (i + 1)
        k[to:to + m], v[to:to + m] = c.k[c.start[i]:c.start[i] + m], c.v[c.start[i]:c.start[i] + m]
        c.kv["kv_start"][i] = to
    small = (c.k, c.v)
    c.k, c.v = k, v
    c.run()
    c.k, c.v = small
    c.check()


def test_empty_calls():
    d = gdn.dims(1, 2, 64)
    e = lambda w: torch.empty((0, w), device="cuda", dtype=torch.bfloat16)
    gdn.gdn_attn_prefill(d, ints([0, 0]), e(128), e(64), e(64), torch.empty((0, 2, 64), device="cuda", dtype=torch.bfloat16))
    # a cache of no rows: every token sees nothing
    q = torch.ones((3, 128), device="cuda", dtype=torch.bfloat16)
    out, lse = torch.full((3, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16), torch.zeros((3, 2), device="cuda")
    gdn.gdn_attn_prefill(d, ints([0, 3]), q, e(64), e(64), out, lse=lse, kv_start=ints([0]), kv_len=ints([9]))
    assert (out == 0).all() and (lse == -INF).all()
