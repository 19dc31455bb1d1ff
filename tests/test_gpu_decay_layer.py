"""The calls together, as a serving loop uses them for one layer of linear
attention on 8-bit weights: residual norm -> 8-bit input projection (q | k |
v | z) -> prefill or decode step with the gated norm over slices of the
projection -> quantiser -> 8-bit output projection. Every call is checked
against its formula in fp64 on the very tensors that it was given."""

import numpy as np
import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from tests import decay_reference as ref
from tests import test_gpu_add_rmsnorm as norm
from tests import test_gpu_decay as decay
from tests import test_gpu_linear_fp8 as linear

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Layer:
    def __init__(self, hidden, hk, hv, D):
        gen = torch.Generator().manual_seed(3)
        self.hk, self.hv, self.D, self.hidden = hk, hv, D, hidden
        n_in = (2 * hk + 2 * hv) * D
        self.d = gdn.dims(hk, hv, D, io_dtype=BF)
        self.norm_in = (1 + 0.2 * torch.randn(hidden, generator=gen)).cuda()
        self.norm_w = (1 + 0.2 * torch.randn(D, generator=gen)).cuda()
        self.g = -torch.rand(hv, generator=gen).cuda() * 0.3
        self.w_in = self.quantise((torch.randn((n_in, hidden), generator=gen) * hidden ** -0.5).to(BF).cuda())
        self.w_out = self.quantise((torch.randn((hidden, hv * D), generator=gen) * (hv * D) ** -0.5).to(BF).cuda())

    def quantise(self, t):
        q, s = torch.empty(t.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(t.shape[0], device="cuda")
        gdn.gdn_add_rmsnorm(t, None, out_q=q, out_scale=s)
        norm.verify(t, None, None, 0, "bf16", None, None, q, s)
        return q, s

    def __call__(self, x, residual, state, cu=None, slots=None):
        """One layer over rows of x; the tensors between its calls."""
        M, (hk, hv, D) = x.shape[0], (self.hk, self.hv, self.D)
        t = {"q8": torch.empty((M, self.hidden), dtype=torch.float8_e4m3fn, device="cuda"),
             "s8": torch.empty(M, device="cuda"), "sum": torch.empty_like(x),
             "proj": torch.empty((M, self.w_in[0].shape[0]), dtype=BF, device="cuda"),
             "out": torch.empty((M, hv, D), dtype=BF, device="cuda"),
             "core": torch.empty((M, hv, D), device="cuda"), "y": torch.empty_like(x)}
        gdn.gdn_add_rmsnorm(x, self.norm_in, residual=residual, sum_out=t["sum"], out_q=t["q8"], out_scale=t["s8"])
        gdn.gdn_linear_fp8(t["q8"], t["s8"], *self.w_in, t["proj"])
        q, k, v, z = t["proj"].split([hk * D, hk * D, hv * D, hv * D], dim=1)
        kw = dict(core_out=t["core"], z=z, norm_w=self.norm_w, out=t["out"])
        if cu is None:
            gdn.gdn_decay_step(self.d, q, k, v, self.g, state, state_slots=slots, **kw)
        else:
            gdn.gdn_decay_prefill(self.d, cu, q, k, v, self.g, state, **kw)
        t["o8"], t["os"] = self.quantise_row(t["out"].view(M, hv * D))
        gdn.gdn_linear_fp8(t["o8"], t["os"], *self.w_out, t["y"])
        return t

    def quantise_row(self, t):
        q, s = torch.empty(t.shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(t.shape[0], device="cuda")
        gdn.gdn_add_rmsnorm(t, None, out_q=q, out_scale=s)
        return q, s

    def verify(self, t, x, residual, spans, S0, S, split):
        """spans: the rows of each sequence; S0, S its state before and after."""
        norm.verify(x, residual, self.norm_in, 1e-6, "bf16", t["sum"], None, t["q8"], t["s8"])
        linear.verify(t["q8"], t["s8"], *self.w_in, None, t["proj"], "bf16")
        c = decay.Case.__new__(decay.Case)
        c.hk, c.hv, c.D, c.dtype, c.tiled, c.gated = self.hk, self.hv, self.D, "bf16", False, True
        c.q, c.k, c.v, c.z = t["proj"].split([self.hk * self.D] * 2 + [self.hv * self.D] * 2, dim=1)
        c.g, c.w, c.core, c.out = self.g, self.norm_w, t["core"], t["out"]
        for (a, b), s0, s1 in zip(spans, S0, S):
            c.check(a, b, s0, s1, f"rows {a}..{b}", split)
        norm.verify(t["out"].view(x.shape[0], -1), None, None, 0, "bf16", None, None, t["o8"], t["os"])
        linear.verify(t["o8"], t["os"], *self.w_out, None, t["y"], "bf16")


@pytest.mark.parametrize("D,lengths", [(128, [70, 1, 133]), (64, [20, 5, 150])])
def test_prompt_then_decode(D, lengths):
    hidden, hk, hv = 512, 2, 4
    layer = Layer(hidden, hk, hv, D)
    gen = torch.Generator().manual_seed(4)
    T, N = sum(lengths), len(lengths)
    cu = np.concatenate([[0], np.cumsum(lengths)])
    x = torch.randn((T, hidden), generator=gen).to(BF).cuda()
    res = (3 * torch.randn((T, hidden), generator=gen)).to(BF).cuda()
    state = torch.zeros((N, hv, D, D), device="cuda")
    t = layer(x, res, state, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    spans = [(int(cu[n]), int(cu[n + 1])) for n in range(N)]
    layer.verify(t, x, res, spans, [np.zeros((hv, D, D))] * N, state, decay.SPLIT)

    # two decode steps over a pool that holds the states at other slots, one row padded
    pool = torch.randn((6, hv, D, D), device="cuda")
    slots = torch.tensor([4, 0, 5, -1], dtype=torch.int32, device="cuda")
    pool[slots[:3].long()] = state
    others = pool[1:4].clone()
    for _ in range(2):
        x = torch.randn((4, hidden), generator=gen).to(BF).cuda()
        res = (3 * torch.randn((4, hidden), generator=gen)).to(BF).cuda()
        before = pool.clone()
        t = layer(x, res, pool, slots=slots)
        layer.verify({k: v[:3] for k, v in t.items()}, x[:3], res[:3], [(0, 1), (1, 2), (2, 3)],
                     [decay.f64(before[s]) for s in (4, 0, 5)], [pool[s] for s in (4, 0, 5)], 0.0)
        assert not t["out"][3].any() and not t["y"][3].any()
    assert torch.equal(pool[1:4], others)
    assert gdn.gdn_device_error() == 0
