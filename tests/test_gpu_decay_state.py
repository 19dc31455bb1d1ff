"""The state that the tensor-core prefill keeps (bf16, head_dim 128): bounds of
its own arithmetic, far below those of a token-by-token sum.

A chunk of 64 tokens adds dS = sum_s w_s v_s k_s, w_s = e^(G_n - G_s), and
multiplies the state by e^(G_n). w_s is off by 2^-22 (two steps of the
exponential) and, for exponents below 1, 2^-23 through the difference, the
product w k by 2^-24; that product goes to the MMAs as three bf16 parts of
eight bits, which hold all of its 24, and v is exact; the twelve MMAs of 16
tokens that add up dS are allowed a step, 2^-23, each. Together below DS =
2^-19 of the sum of magnitudes M. The update takes two roundings of the sum
and the factor's own error: 4 u of the magnitudes A at most; joining segments
as much again. All terms here are positive, so that what a lost part leaves
out adds up instead of cancelling."""

import numpy as np
import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from tests.decay_reference import U, check
from tests.test_gpu_decay import Case, f64

DS = 2.0 ** -19
HK, HV, D = 1, 2, 128


def inputs(T, N, seed=61):
    """Positive k, v and states, decays of 0.0007 to 0.0014 a token."""
    gen = torch.Generator().manual_seed(seed)
    k = torch.rand((T, HK * D), generator=gen) + 0.5
    v = torch.rand((T, HV * D), generator=gen) + 0.5
    g = -0.0007 * (1 + torch.rand((T, HV), generator=gen))
    return k.to(torch.bfloat16), v.to(torch.bfloat16), g.float(), torch.rand((N, HV, D, D), generator=gen) * 10


def chunk(S, k, v, g, cut=None):
    """The state after up to 64 tokens and the chunk's sum of magnitudes, in fp64; cut: K' cut to that many bf16 parts."""
    G = np.cumsum(g, axis=0)
    out, add = np.empty_like(S), np.empty_like(S)
    for h in range(HV):
        w = np.exp(G[-1, h] - G[:, h])[:, None]
        kp = w * k
        if cut is not None:
            kp, left = 0.0, (w.astype(np.float32) * k.astype(np.float32)).astype(np.float32)
            for _ in range(cut):
                part = (left.view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)
                kp, left = kp + part.astype(np.float64), left - part
        add[h] = v[:, h * D:(h + 1) * D].T @ kp
        out[h] = np.exp(G[-1, h]) * S[h] + add[h]
    return out, add


def run(S, k, v, g, cut=None):
    """(state, bound) of one sequence."""
    E = np.zeros_like(S)
    for a in range(0, len(k), 64):
        S, M = chunk(S, k[a:a + 64], v[a:a + 64], g[a:a + 64], cut)
        E = np.exp(g[a:a + 64].sum(0))[:, None, None] * E + 8 * U * S + DS * M
    return S, E


def test_the_bound_tells_two_parts_from_three():
    k, v, g, S0 = (f64(t) for t in inputs(512, 1))
    want, bound = run(S0[0], k, v, g)
    assert (np.abs(run(S0[0], k, v, g, 3)[0] - want) < bound / 4).all()
    assert (np.abs(run(S0[0], k, v, g, 2)[0] - want) > bound).mean() > 0.9


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,workspace", [([512], None), ([512], "auto"), ([200, 64, 130, 1], None), ([1100], "auto")])
def test_state(lengths, workspace):
    T, N = sum(lengths), len(lengths)
    c = Case(62, HK, HV, D, "bf16", T, N, gated=False)
    k, v, g, S0 = inputs(T, N)
    c.k.copy_(k), c.v.copy_(v), c.g.copy_(g), c.state.copy_(S0)
    cu = np.concatenate([[0], np.cumsum(lengths)])
    if workspace == "auto":
        assert gdn.gdn_decay_prefill_workspace_size(c.d, N, T) > 0
    gdn.gdn_decay_prefill(c.d, torch.tensor(cu, dtype=torch.int32, device="cuda"), c.q, c.k, c.v, c.g, c.state, out=c.out,
                          workspace=workspace)
    for n in range(N):
        a, b = cu[n], cu[n + 1]
        want, bound = run(f64(S0[n]), f64(k)[a:b], f64(v)[a:b], f64(g)[a:b])
        check(f64(c.state[n]), want, bound, f"sequence {n} ({lengths[n]} tokens) state")
