"""gdn_decay_step and gdn_decay_prefill against the recurrence in fp64, token
by token, within bounds made of the inputs' magnitudes (decay_reference)."""

import math

import numpy as np
import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from tests import decay_reference as ref

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# the tensor-core prefill (bf16, head_dim 128) holds fp32 factors as sums of bf16 parts: two parts leave 2^-17
# of a factor, two such factors never meet in one product, and its fp32 sums run over at most 128 tokens and
# 128 columns at a time
SPLIT = 2.0 ** -16

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


class Case:
    """Inputs of `tokens` rows inside one wide activation [q | k | v | z], as a projection leaves them."""

    def __init__(self, seed, hk, hv, D, dtype, tokens, states, token_decay=True, rate=0.2, tiled=False, gated=True,
                 pad=0):
        gen = torch.Generator().manual_seed(seed)
        io = DT[dtype]
        self.hk, self.hv, self.D, self.dtype, self.tiled, self.gated = hk, hv, D, dtype, tiled, gated
        n = lambda *s: torch.randn(s, generator=gen)
        act = n(tokens, (2 * hk + 2 * hv) * D + pad)
        act[:, hk * D:2 * hk * D] *= D ** -0.5
        act = act.to(io).cuda()
        self.act = act
        self.q, self.k = act[:, :hk * D], act[:, hk * D:2 * hk * D]
        self.v, self.z = act[:, 2 * hk * D:(2 * hk + hv) * D], act[:, (2 * hk + hv) * D:(2 * hk + 2 * hv) * D]
        g = -torch.nn.functional.softplus(n(*((tokens, hv) if token_decay else (hv,)))) * rate
        self.g = g.float().cuda()
        self.w = (1 + 0.2 * n(D)).float().cuda()
        self.state = (0.1 * n(states, hv, D, D)).float().cuda()
        self.out = torch.full((tokens, hv, D), 7.25, device="cuda", dtype=io)
        self.core = torch.full((tokens, hv, D), 7.25, device="cuda")
        self.d = gdn.dims(hk, hv, D, map=gdn.GDN_MAP_TILED if tiled else gdn.GDN_MAP_GROUPED, io_dtype=io)

    def gate(self):
        return {"z": self.z, "norm_w": self.w} if self.gated else {}

    def reference(self, a, b, S0, scale=None):
        """Tokens a..b as one sequence from S0."""
        scale = self.D ** -0.5 if scale is None else scale
        g = f64(self.g)
        g = g[a:b] if g.ndim == 2 else np.broadcast_to(g, (b - a, self.hv))
        r = lambda t, h: f64(t[a:b]).reshape(b - a, h, self.D)
        return ref.recurrence(r(self.q, self.hk), r(self.k, self.hk), r(self.v, self.hv), g, S0, scale, self.tiled)

    def check(self, a, b, S0, S, what, split=0.0, scale=None):
        o, S1, do, mag, dS, A = self.reference(a, b, S0, scale)
        do = do + split * mag
        ref.check(f64(S), S1, dS * 1.02 + split * A, what + " state")
        ref.check(f64(self.core[a:b]), o, do * 1.02 + 1e-38, what + " core_out")
        if self.gated:
            y, dy = ref.gated(o, f64(self.z[a:b]).reshape(o.shape), f64(self.w), 1e-6, self.dtype, do)
        else:
            y, dy = o, ref.rounded(o, self.dtype, do)
        ref.check(f64(self.out[a:b]), y, dy, what + " out")


SHAPES = [(1, 1, 128), (2, 4, 128), (4, 4, 64), (1, 3, 96), (2, 8, 32), (16, 32, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hk,hv,D", SHAPES)
@pytest.mark.parametrize("gated,tiled,token_decay", [(True, True, True), (False, False, False)])
def test_step_matches_the_recurrence(dtype, hk, hv, D, gated, tiled, token_decay):
    B = 3
    c = Case(hk * 100 + D, hk, hv, D, dtype, B, B, token_decay, tiled=tiled, gated=gated, pad=8)
    S0 = f64(c.state)
    gdn.gdn_decay_step(c.d, c.q, c.k, c.v, c.g, c.state, core_out=c.core, out=c.out, **c.gate())
    for b in range(B):
        c.check(b, b + 1, S0[b], c.state[b], f"row {b}")
    assert gdn.gdn_device_error() == 0


def test_step_outputs_one_at_a_time_are_the_same():
    c = Case(5, 2, 4, 128, "bf16", 4, 4)
    S0 = c.state.clone()
    gdn.gdn_decay_step(c.d, c.q, c.k, c.v, c.g, c.state, core_out=c.core, out=c.out, **c.gate())
    for kw in ({"core_out": torch.empty_like(c.core)}, {"out": torch.empty_like(c.out), **c.gate()}):
        S = S0.clone()
        gdn.gdn_decay_step(c.d, c.q, c.k, c.v, c.g, S, **kw)
        assert torch.equal(S, c.state)
        for name, full in (("core_out", c.core), ("out", c.out)):
            if name in kw:
                assert torch.equal(kw[name], full)


def test_step_slots_padding_and_out_of_range():
    B, P = 6, 9
    c = Case(6, 2, 4, 64, "bf16", B, P, gated=True)
    S0 = c.state.clone()
    slots = torch.tensor([8, -1, 3, P, 0, -(2 ** 31)], dtype=torch.int32, device="cuda")
    gdn.gdn_decay_step(c.d, c.q, c.k, c.v, c.g, c.state, core_out=c.core, out=c.out, state_slots=slots, **c.gate())
    for b, s in enumerate(slots.tolist()):
        if 0 <= s < P:
            c.check(b, b + 1, f64(S0[s]), c.state[s], f"row {b}")
        else:
            assert not c.core[b].any() and not c.out[b].any()
    untouched = [s for s in range(P) if s not in (8, 3, 0)]
    assert torch.equal(c.state[untouched], S0[untouched])
    assert gdn.gdn_device_error() == 2  # GDN_ERR_EXTENT, for the entry past the pool
    assert gdn.gdn_device_error() == 0


def test_step_scale_and_extreme_decays():
    """A reset (-inf), a decay past fp32's range, none, and a growing one; a given scale."""
    c = Case(7, 1, 4, 128, "f32", 2, 2, token_decay=False, gated=False)
    c.g.copy_(torch.tensor([-math.inf, -1e30, 0.0, 0.5]))
    S0 = f64(c.state)
    gdn.gdn_decay_step(c.d, c.q, c.k, c.v, c.g, c.state, core_out=c.core, out=c.out, scale=0.75)
    for b in range(2):
        c.check(b, b + 1, S0[b], c.state[b], f"row {b}", scale=0.75)


def test_step_nan_stays_in_its_row():
    c = Case(8, 2, 4, 64, "bf16", 3, 3)
    c.act[1, :] = float("nan")
    S0 = f64(c.state)
    gdn.gdn_decay_step(c.d, c.q, c.k, c.v, c.g, c.state, core_out=c.core, out=c.out, **c.gate())
    assert torch.isnan(c.state[1]).all() and torch.isnan(c.core[1]).all() and torch.isnan(c.out[1].float()).all()
    for b in (0, 2):
        c.check(b, b + 1, S0[b], c.state[b], f"row {b}")


def test_step_pool_past_32_bit_offsets():
    """A pool whose last slot starts past 2^31 elements (and 2^33 bytes)."""
    hv, D = 64, 128
    P = 2 ** 31 // (hv * D * D) + 3
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 9 GB of device memory")
    c = Case(9, 16, hv, D, "bf16", 2, 1)
    pool = torch.empty((P, hv, D, D), device="cuda")
    slots = [P - 1, 1]
    first = torch.randn((2, hv, D, D), device="cuda") * 0.1
    for s, f in zip(slots, first):
        pool[s].copy_(f)
    gdn.gdn_decay_step(c.d, c.q, c.k, c.v, c.g, pool, core_out=c.core, out=c.out,
                       state_slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), **c.gate())
    for b, s in enumerate(slots):
        c.check(b, b + 1, f64(first[b]), pool[s], f"row {b}")


def test_step_empty_batch():
    c = Case(10, 2, 4, 64, "bf16", 1, 1)
    S0 = c.state.clone()
    gdn.gdn_decay_step(c.d, c.q[:0], c.k[:0], c.v[:0], c.g[:0], c.state[:0], out=c.out[:0])
    assert torch.equal(S0, c.state)


# --------------------------------------------------------------------- prefill


def run_prefill(c, lengths, total=None, workspace="auto", what=""):
    cu = np.concatenate([[0], np.cumsum(lengths)])
    S0 = f64(c.state)
    gdn.gdn_decay_prefill(c.d, torch.tensor(cu, dtype=torch.int32, device="cuda"), c.q, c.k, c.v, c.g, c.state,
                          core_out=c.core, out=c.out, workspace=workspace, **c.gate())
    split = SPLIT if c.dtype == "bf16" and c.D == 128 else 0.0
    for n, length in enumerate(lengths):
        if length == 0:
            assert np.array_equal(f64(c.state[n]), S0[n])
        else:
            c.check(cu[n], cu[n + 1], S0[n], c.state[n], f"{what} sequence {n} ({length} tokens)", split)
    rest = slice(int(cu[-1]), None)
    assert (c.core[rest] == 7.25).all() and (c.out[rest].float() == 7.25).all()  # rows behind the last sequence
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hk,hv,D", [(1, 1, 128), (2, 4, 128), (4, 4, 64), (1, 3, 96), (2, 8, 32)])
@pytest.mark.parametrize("gated,tiled,token_decay", [(True, True, True), (False, False, False)])
def test_prefill_matches_the_recurrence(dtype, hk, hv, D, gated, tiled, token_decay):
    lengths = [1, 0, 7, 8, 9, 63, 64, 65, 0, 127, 128, 129, 200, 2, 0]
    T = sum(lengths)
    c = Case(hk * 10 + D, hk, hv, D, dtype, T + 5, len(lengths), token_decay, tiled=tiled, gated=gated, pad=8)
    run_prefill(c, lengths)


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("lengths", [[1, 0, 63, 64, 65, 130, 193], [700, 3]])
def test_prefill_outputs_one_at_a_time(gated, lengths):
    """out alone: the tensor-core kernel then rounds S and P to bf16, each 2^-8 of a factor of one product, so o is off
    by at most 2^-8 of the magnitudes; the state is the same to the bit. core_out alone is the same as beside out."""
    T = sum(lengths)
    cu = np.concatenate([[0], np.cumsum(lengths)])
    c = Case(31, 2, 4, 128, "bf16", T, len(lengths), gated=gated)
    dcu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    S0 = c.state.clone()
    gdn.gdn_decay_prefill(c.d, dcu, c.q, c.k, c.v, c.g, c.state, core_out=c.core, out=c.out, **c.gate())
    S, core = S0.clone(), torch.empty_like(c.core)
    gdn.gdn_decay_prefill(c.d, dcu, c.q, c.k, c.v, c.g, S, core_out=core)
    assert torch.equal(S, c.state) and torch.equal(core, c.core)
    S = S0.clone()
    c.out.fill_(7.25)
    gdn.gdn_decay_prefill(c.d, dcu, c.q, c.k, c.v, c.g, S, out=c.out, **c.gate())
    assert torch.equal(S, c.state)
    for n, length in enumerate(lengths):
        if length:
            a, b = cu[n], cu[n + 1]
            o, _, do, mag, _, _ = c.reference(a, b, f64(S0[n]))
            do = do + (2.0 ** -8 + SPLIT) * mag
            y, dy = (ref.gated(o, f64(c.z[a:b]).reshape(o.shape), f64(c.w), 1e-6, c.dtype, do) if gated
                     else (o, ref.rounded(o, c.dtype, do)))
            ref.check(f64(c.out[a:b]), y, dy, f"sequence {n}")


def test_prefill_state_aligned_to_16_bytes_alone():
    """The tensor-core kernel wants 32; the call takes 16."""
    lengths = [100, 60]
    c = Case(32, 1, 2, 128, "bf16", 160, 2)
    n = c.state.numel()
    buf = torch.empty(n + 8, device="cuda")
    at = 4 if buf.data_ptr() % 32 == 0 else 0
    shifted = buf[at:at + n].view(c.state.shape)
    shifted.copy_(c.state)
    assert shifted.data_ptr() % 32 == 16
    c.state = shifted
    run_prefill(c, lengths)


@pytest.mark.parametrize("N,L", [(40, 1), (40, 3), (33, 16), (20, 17), (70, 40)])
def test_prefill_several_tokens_of_many_sequences(N, L):
    """Both sides of the length from which chunks are used: several tokens of a decode step, short prompts."""
    c = Case(33 + L, 2, 2, 128, "bf16", N * L, N)
    run_prefill(c, [L] * N)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64), ("f16", 128)])
@pytest.mark.parametrize("workspace", ["auto", None])
def test_prefill_long_sequences(dtype, D, workspace):
    """Segments with and without a workspace: lengths at, below and above their multiples."""
    lengths = [1300, 1, 0, 512, 449, 448]
    c = Case(11, 1, 2, D, dtype, sum(lengths), len(lengths), rate=0.05)
    if workspace == "auto":
        assert gdn.gdn_decay_prefill_workspace_size(c.d, len(lengths), sum(lengths)) > 0
    run_prefill(c, lengths, workspace=workspace)


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f16", 64), ("bf16", 96), ("f32", 128)])
def test_prefill_one_long_sequence_among_many(dtype, D):
    """More (sequence, head) pairs than SMs, and one sequence that outlasts the rest: it alone is cut."""
    lengths = [3, 0, 9, 700] + [5, 1, 40, 0, 72, 2] * 6
    c = Case(35, 4, 16, D, dtype, sum(lengths) + 3, len(lengths), rate=0.05)
    assert gdn.gdn_decay_prefill_workspace_size(c.d, len(lengths), sum(lengths) + 3) > 0
    run_prefill(c, lengths)
    run_prefill(c, lengths, workspace=None)


def test_prefill_many_sequences():
    """More sequences than one probe of the search covers, most of them short or empty."""
    rng = np.random.default_rng(3)
    lengths = [int(x) for x in rng.integers(0, 4, size=1100)]
    c = Case(12, 1, 1, 32, "bf16", sum(lengths), len(lengths))
    run_prefill(c, lengths)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 128), ("bf16", 64)])
def test_prefill_strong_and_mixed_decays(dtype, D):
    """Decays from none to resets inside one chunk: the sums of log decays reach far below fp32's exponents, what
    they multiply must not suffer."""
    T = 300
    c = Case(13, 1, 2, D, dtype, T, 1)
    g = -torch.rand((T, 2), generator=torch.Generator().manual_seed(1)).cuda() * 12
    g[::7] = 0.0
    g[::31] = -math.inf
    g[5::53] = -1e4
    g[250:] = 0.0
    c.g.copy_(g)
    run_prefill(c, [T])


def test_prefill_continues_steps_and_splits():
    """Prefill 70 tokens, three steps, prefill the rest: the same as one prefill, within both bounds."""
    T = 150
    c = Case(14, 2, 4, 128, "bf16", T, 1)
    whole = c.state.clone()
    S0 = f64(whole)
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")
    sl = lambda a, b: dict(q=c.q[a:b], k=c.k[a:b], v=c.v[a:b], g=c.g[a:b])
    rest = lambda a, b: dict(core_out=c.core[a:b], out=c.out[a:b], z=c.z[a:b], norm_w=c.w)
    gdn.gdn_decay_prefill(c.d, cu(70), **sl(0, 70), state=c.state, **rest(0, 70))
    for t in range(70, 73):
        gdn.gdn_decay_step(c.d, **sl(t, t + 1), state=c.state, **rest(t, t + 1))
    gdn.gdn_decay_prefill(c.d, cu(T - 73), **sl(73, T), state=c.state, **rest(73, T))
    c.check(0, T, S0[0], c.state[0], "split", 3 * SPLIT)


def test_prefill_nan_stays_behind_its_token():
    """A NaN token spoils its own sequence from there on and nothing before it or beside it."""
    lengths = [100, 90, 60]
    c = Case(15, 1, 2, 128, "bf16", 250, 3, gated=False)
    c.act[140, :] = float("nan")  # token 40 of sequence 1
    S0 = f64(c.state)
    cu = torch.tensor([0, 100, 190, 250], dtype=torch.int32, device="cuda")
    gdn.gdn_decay_prefill(c.d, cu, c.q, c.k, c.v, c.g, c.state, core_out=c.core, out=c.out)
    c.check(0, 100, S0[0], c.state[0], "before", SPLIT)
    c.check(190, 250, S0[2], c.state[2], "after", SPLIT)
    o, _, do, mag, _, _ = c.reference(100, 140, S0[1])  # its own tokens before, most of them in the same chunk
    ref.check(f64(c.core[100:140]), o, do * 1.02 + SPLIT * mag, "own tokens before")
    assert torch.isnan(c.core[140]).all() and torch.isnan(c.state[1]).all()


@pytest.mark.parametrize("dtype,D,workspace", [("bf16", 128, "auto"), ("bf16", 128, None), ("f16", 128, "auto"),
                                               ("f32", 64, "auto"), ("bf16", 96, None)])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_prefill_bad_neighbours(dtype, D, workspace, what):
    """Every other sequence and the rows behind the last one hold nothing finite, their decays included: what a tile
    reads past a sequence's end must not reach it."""
    lengths = [100, 40, 65, 3, 1, 70, 300, 20, 5]
    cu = np.concatenate([[0], np.cumsum(lengths)])
    T = int(cu[-1]) + 40
    c = Case(23, 1, 2, D, dtype, T, len(lengths))
    for n in range(1, len(lengths), 2):
        c.act[cu[n]:cu[n + 1]] = what
        c.g[cu[n]:cu[n + 1]] = float("nan")
    c.act[cu[-1]:] = what
    c.g[cu[-1]:] = float("nan")
    S0 = f64(c.state)
    gdn.gdn_decay_prefill(c.d, torch.tensor(cu, dtype=torch.int32, device="cuda"), c.q, c.k, c.v, c.g, c.state,
                          core_out=c.core, out=c.out, workspace=workspace, **c.gate())
    for n in range(0, len(lengths), 2):
        c.check(cu[n], cu[n + 1], S0[n], c.state[n], f"sequence {n}", SPLIT if dtype == "bf16" and D == 128 else 0.0)
    assert (c.core[cu[-1]:] == 7.25).all() and (c.out[cu[-1]:].float() == 7.25).all()
    assert gdn.gdn_device_error() == 0


def test_prefill_infinite_value_spoils_its_value_row_alone():
    """An infinity in one element of v makes that value row non-finite from its token on, and nothing else."""
    T = 140
    c = Case(22, 1, 2, 128, "bf16", T, 1, gated=False)
    c.v[75, 128 + 9] = float("inf")  # V head 1, value row 9
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    gdn.gdn_decay_prefill(c.d, cu, c.q, c.k, c.v, c.g, c.state, core_out=c.core, out=c.out)
    spoilt = torch.zeros((T, 2, 128), dtype=torch.bool)
    spoilt[75:, 1, 9] = True
    assert torch.equal(~torch.isfinite(c.core).cpu(), spoilt)
    rows = torch.zeros((2, 128, 128), dtype=torch.bool)
    rows[1, 9] = True
    assert torch.equal(~torch.isfinite(c.state[0]).cpu(), rows)


def test_prefill_nothing_to_do():
    c = Case(16, 1, 2, 64, "bf16", 4, 2)
    S0 = c.state.clone()
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    gdn.gdn_decay_prefill(c.d, cu, c.q, c.k, c.v, c.g, c.state, core_out=c.core, out=c.out, **c.gate())
    gdn.gdn_decay_prefill(c.d, cu, c.q[:0], c.k[:0], c.v[:0], c.g[:0], c.state, out=c.out[:0])
    assert torch.equal(S0, c.state) and (c.core == 7.25).all() and (c.out.float() == 7.25).all()


@pytest.mark.parametrize("call", ["step", "prefill"])
def test_graph_replay_and_another_stream(call):
    """Captured on a side stream and replayed: every replay continues from the state the last one left."""
    lengths = [130, 40]
    rows = sum(lengths) if call == "prefill" else 4
    c = Case(17, 1, 2, 128, "bf16", rows, 2 if call == "prefill" else 4, rate=0.5)
    cu = torch.tensor([0, 130, 170], dtype=torch.int32, device="cuda")
    S0 = c.state.clone()

    def go(state, core, out, stream=None):
        kw = dict(core_out=core, out=out, stream=stream, **c.gate())
        if call == "step":
            gdn.gdn_decay_step(c.d, c.q, c.k, c.v, c.g, state, **kw)
        else:
            gdn.gdn_decay_prefill(c.d, cu, c.q, c.k, c.v, c.g, state, **kw)

    ref_state, ref_core, ref_out = S0.clone(), torch.empty_like(c.core), torch.empty_like(c.out)
    for _ in range(3):
        go(ref_state, ref_core, ref_out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go(c.state, c.core, c.out)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(c.state, c.core, c.out)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.state, ref_state) and torch.equal(c.core, ref_core) and torch.equal(c.out, ref_out)
    state, core, out = S0.clone(), torch.empty_like(c.core), torch.empty_like(c.out)
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        go(state, core, out, stream=s)
    s.synchronize()
    assert torch.equal(state, ref_state) and torch.equal(core, ref_core) and torch.equal(out, ref_out)


def test_two_calls_side_by_side():
    """Two prefills on two streams at once, each with its own workspace, give what they give alone."""
    cs = [Case(18 + i, 1, 2, 128, "bf16", 1500, 1, rate=0.05) for i in range(2)]
    cu = torch.tensor([0, 1500], dtype=torch.int32, device="cuda")
    alone = []
    for c in cs:
        S, out = c.state.clone(), torch.empty_like(c.out)
        gdn.gdn_decay_prefill(c.d, cu, c.q, c.k, c.v, c.g, S, out=out, **c.gate())
        alone.append((S, out))
    need = gdn.gdn_decay_prefill_workspace_size(cs[0].d, 1, 1500)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for c, w, s in zip(cs, ws, streams):
        gdn.gdn_decay_prefill(c.d, cu, c.q, c.k, c.v, c.g, c.state, out=c.out, workspace=w, stream=s, **c.gate())
    torch.cuda.synchronize()
    for c, (S, out) in zip(cs, alone):
        assert torch.equal(c.state, S) and torch.equal(c.out, out)


def test_refusals_of_the_binding():
    c = Case(20, 2, 4, 64, "bf16", 3, 3)
    ok = dict(q=c.q, k=c.k, v=c.v, g=c.g, state=c.state, out=c.out)
    bad = [dict(q=c.q.cpu()), dict(q=c.q.float()), dict(k=c.k[:, :-1]), dict(v=c.v[:2]), dict(g=c.g.half()),
           dict(g=c.g[:, :3]), dict(state=c.state[:2]), dict(state=c.state.half()), dict(out=c.out[:2]),
           dict(out=c.out.float()), dict(state_slots=torch.zeros(2, dtype=torch.int32, device="cuda")),
           dict(state_slots=torch.zeros(3, dtype=torch.int64, device="cuda")), dict(z=c.z), dict(norm_w=c.w),
           dict(scale=math.inf), dict(out=None), dict(q=c.q[:, 1:].contiguous()), dict(v=c.act[:, 1:1 + 256])]
    S0 = c.state.clone()
    for kw in bad:
        with pytest.raises((ValueError, TypeError, gdn.GdnError)):
            gdn.gdn_decay_step(c.d, **(ok | kw))
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_decay_step(c.d, **(ok | {"out": c.act.view(-1)[:3 * 4 * 64].view(3, 4, 64)}))  # over q
    assert e.value.status == 4
    assert torch.equal(S0, c.state)
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    for kw in (dict(cu_seqlens=cu.long()), dict(cu_seqlens=cu[:3]), dict(workspace="none"),
               dict(workspace=torch.empty(4, device="cuda"))):
        with pytest.raises((ValueError, TypeError, gdn.GdnError)):
            gdn.gdn_decay_prefill(c.d, **({"cu_seqlens": cu} | ok | kw))
    big = Case(21, 1, 2, 64, "bf16", 1500, 1)
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_decay_prefill(big.d, torch.tensor([0, 1500], dtype=torch.int32, device="cuda"), big.q, big.k, big.v,
                              big.g, big.state, out=big.out,
                              workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 1
