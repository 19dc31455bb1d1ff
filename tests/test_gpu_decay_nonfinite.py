"""Where one entry that is not finite reaches, through gdn_decay_prefill: of q
or z the outputs of its token alone, of v its value row, of k or g every row,
from its token on; earlier tokens and other sequences never. The exact set of
entries that are not finite is that of the recurrence in fp64."""

import numpy as np
import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from tests import decay_reference as ref
from tests.test_gpu_decay import Case, f64

pytestmark = pytest.mark.gpu
HK, HV = 2, 4
# (lengths, sequence, token in it): in the middle of a chunk of one segment, and of the third of several
PLACES = [([37, 300, 20], 1, 139), ([700], 0, 330)]


@pytest.mark.parametrize("dtype,D,workspace", [("bf16", 128, "auto"), ("bf16", 128, None), ("f32", 64, "auto"),
                                               ("f16", 128, "auto"), ("bf16", 96, None)])
@pytest.mark.parametrize("name", ["q", "k", "v", "z", "g"])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("lengths,seq,token", PLACES)
def test_reach(dtype, D, workspace, name, what, lengths, seq, token):
    T, N = sum(lengths), len(lengths)
    cu = np.concatenate([[0], np.cumsum(lengths)])
    # a gated row mixes its head's value rows, so v is looked at without the gate
    c = Case(71, HK, HV, D, dtype, T, N, rate=0.02, gated=name != "v")
    at, head = int(cu[seq]) + token, 1  # K head or V head
    if name == "g":
        c.g[at, head] = what
    else:
        getattr(c, name)[at, head * D + 9] = what
    S0 = f64(c.state)
    dcu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if len(lengths) == 1 and workspace == "auto":
        assert gdn.gdn_decay_prefill_workspace_size(c.d, N, T) > 0
    gdn.gdn_decay_prefill(c.d, dcu, c.q, c.k, c.v, c.g, c.state, core_out=c.core, out=c.out, workspace=workspace, **c.gate())
    only = torch.empty_like(c.out)
    S1 = torch.tensor(S0, dtype=torch.float32, device="cuda")
    gdn.gdn_decay_prefill(c.d, dcu, c.q, c.k, c.v, c.g, S1, out=only, workspace=workspace, **c.gate())
    for n in range(N):
        a, b = int(cu[n]), int(cu[n + 1])
        with np.errstate(all="ignore"):
            o, S, do, *_ = c.reference(a, b, S0[n])
            y = ref.gated(o, f64(c.z[a:b]).reshape(o.shape), f64(c.w), 1e-6, dtype, do)[0] if c.gated else o
        bad = lambda t: ~np.isfinite(f64(t))
        assert np.array_equal(bad(c.core[a:b]), ~np.isfinite(o)), "core_out"
        for got in (c.out, only):
            assert np.array_equal(bad(got[a:b]), ~np.isfinite(y)), "out"
        for got in (c.state, S1):
            assert np.array_equal(bad(got[n]), ~np.isfinite(S)), "state"
        if n == seq:
            assert np.isfinite(o[:token]).all() and (name == "z") == np.isfinite(o[token]).all()
            assert np.isfinite(o[token + 1:]).all() == (name in "qz")
            assert np.isfinite(S).all() == (name in "qz")
        else:
            assert np.isfinite(o).all()
    assert gdn.gdn_device_error() == 0
