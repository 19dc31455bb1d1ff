"""The calls of a layer on 8-bit weights with an empty batch: nothing happens, nothing is refused."""

import pytest
import torch

import gated_delta_net_causal_gb300 as gdn

pytestmark = pytest.mark.gpu


def test_a_layer_of_no_rows():
    BF, F8 = torch.bfloat16, torch.float8_e4m3fn
    hidden, hk, hv, D = 64, 1, 2, 64
    e = lambda *s, dtype=BF: torch.empty(s, dtype=dtype, device="cuda")
    d = gdn.dims(hk, hv, D, io_dtype=BF)
    x, x8, s8, act, y = e(0, hidden), e(0, hidden, dtype=F8), e(0, dtype=torch.float32), e(0, 384), e(0, hidden)
    w_in = torch.ones((384, hidden), device="cuda").to(F8)
    w_out = torch.ones((hidden, hv * D), device="cuda").to(F8)
    o, o8 = e(0, hv, D), e(0, hv * D, dtype=F8)
    state, g = torch.ones((3, hv, D, D), device="cuda"), torch.zeros(hv, device="cuda")
    norm = torch.ones(hidden, device="cuda")
    one = lambda n: torch.ones(n, device="cuda")
    gdn.gdn_add_rmsnorm(x, norm, residual=x.clone(), sum_out=x.clone(), out_q=x8, out_scale=s8)
    assert gdn.gdn_linear_fp8(x8, s8, w_in, one(384), act) is act
    q, k, v, z = act.split([hk * D, hk * D, hv * D, hv * D], dim=1)
    gate = dict(z=z, norm_w=one(D), out=o)
    gdn.gdn_decay_step(d, q, k, v, g, state, state_slots=e(0, dtype=torch.int32), **gate)
    gdn.gdn_decay_prefill(d, torch.zeros(4, dtype=torch.int32, device="cuda"), q, k, v, g, state, **gate)
    gdn.gdn_add_rmsnorm(o.view(0, hv * D), None, out_q=o8, out_scale=s8)
    gdn.gdn_linear_fp8(o8, s8, w_out, one(hidden), y, bias=one(hidden))
    assert (state == 1).all() and gdn.gdn_device_error() == 0
    with pytest.raises((ValueError, TypeError)):  # still looked at
        gdn.gdn_linear_fp8(x8, s8, w_in, one(383), act)
