"""gdn_decay_prefill with out alone, as a serving loop calls it: as near to the
recurrence as where core_out is asked for too, and the same bits."""

import numpy as np
import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from tests import decay_reference as ref
from tests.test_gpu_decay import SPLIT, Case, f64

pytestmark = pytest.mark.gpu


def prefill_out(c, lengths, seqs=None, workspace="auto"):
    """out alone, checked for the given sequences (all if None) within the bounds of a call that has core_out; the
    outputs and states of the two calls are the same."""
    cu = np.concatenate([[0], np.cumsum(lengths)])
    dcu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    S0 = c.state.clone()
    gdn.gdn_decay_prefill(c.d, dcu, c.q, c.k, c.v, c.g, c.state, out=c.out, workspace=workspace, **c.gate())
    S, out = S0.clone(), torch.full_like(c.out, 7.25)
    gdn.gdn_decay_prefill(c.d, dcu, c.q, c.k, c.v, c.g, S, core_out=c.core, out=out, workspace=workspace, **c.gate())
    bits = lambda t: t.view(torch.int16 if t.element_size() == 2 else torch.int32)
    for n in range(len(lengths)) if seqs is None else seqs:
        a, b = int(cu[n]), int(cu[n + 1])
        if a == b:
            assert torch.equal(c.state[n], S0[n])
            continue
        c.check(a, b, f64(S0[n]), c.state[n], f"sequence {n} ({lengths[n]} tokens)",
                SPLIT if c.dtype == "bf16" and c.D == 128 else 0.0)
        assert torch.equal(bits(c.out[a:b]), bits(out[a:b])) and torch.equal(bits(c.state[n]), bits(S[n]))
    assert (c.out[int(cu[-1]):].float() == 7.25).all()
    assert gdn.gdn_device_error() == 0
    return cu


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("where", ["state", "tokens"])
def test_cancelling_terms(gated, where):
    """Outputs far smaller than their terms. state: columns i and i + 64 of the state nearly alike and of q opposite, so
    that what is left of S q is their difference. tokens: every second v is the last one's opposite at the same k, so that
    P v leaves what the decay between the two takes. A factor held in one bf16 part would be off by 2^-9 of each term,
    several times what is allowed here."""
    T, hk, hv, D = 40, 2, 4, 128
    c = Case(41, hk, hv, D, "bf16", T, 1, rate=0.003, gated=gated)
    q, k, v = (t.view(T, -1, D) for t in (c.q, c.k, c.v))
    if where == "state":
        q[:, :, 64:] = -q[:, :, :64]
        k[:, :, 64:] = k[:, :, :64]
        c.state.mul_(10.0)
        c.state[..., 64:] = c.state[..., :64] + 0.002 * c.state[..., 64:]
    else:
        q.abs_(), k.abs_()
        k[1::2], v[1::2] = k[::2], -v[::2]
        c.state.zero_()
    prefill_out(c, [T])


@pytest.mark.parametrize("workspace", ["auto", None])
def test_long_sequences(workspace):
    lengths = [1300, 1, 0, 512, 449, 448]
    c = Case(42, 1, 2, 128, "bf16", sum(lengths) + 3, len(lengths), rate=0.05)
    prefill_out(c, lengths, workspace=workspace)


@pytest.mark.parametrize("gated", [True, False])
def test_strong_and_mixed_decays(gated):
    T = 300
    c = Case(43, 1, 2, 128, "bf16", T, 1, gated=gated)
    g = -torch.rand((T, 2), generator=torch.Generator().manual_seed(1)).cuda() * 12
    g[::7] = 0.0
    g[::31] = -float("inf")
    g[5::53] = -1e4
    g[250:] = 0.0
    c.g.copy_(g)
    prefill_out(c, [T])


@pytest.mark.parametrize("workspace", ["auto", None])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_bad_neighbours(workspace, what):
    lengths = [100, 40, 65, 3, 1, 70, 300, 20, 5]
    cu = np.concatenate([[0], np.cumsum(lengths)])
    c = Case(44, 1, 2, 128, "bf16", int(cu[-1]) + 40, len(lengths))
    for n in range(1, len(lengths), 2):
        c.act[cu[n]:cu[n + 1]] = what
        c.g[cu[n]:cu[n + 1]] = float("nan")
    c.act[cu[-1]:] = what
    c.g[cu[-1]:] = float("nan")
    prefill_out(c, lengths, seqs=range(0, len(lengths), 2), workspace=workspace)


def test_infinite_value_spoils_its_value_row_alone():
    T = 140
    c = Case(45, 1, 2, 128, "bf16", T, 1, gated=False)
    c.v[75, 128 + 9] = float("inf")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    gdn.gdn_decay_prefill(c.d, cu, c.q, c.k, c.v, c.g, c.state, out=c.out)
    spoilt = torch.zeros((T, 2, 128), dtype=torch.bool)
    spoilt[75:, 1, 9] = True
    assert torch.equal(~torch.isfinite(c.out.float()).cpu(), spoilt)
