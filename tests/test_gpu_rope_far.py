"""gdn_rope at the ends of the positions' range against angles that are reduced in 60 digits."""

import numpy as np
import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from tests import attn_reference as ref, rope_exact

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1e7])
def test_far_positions_are_as_right_as_near_ones(interleaved, base):
    """The bound is that of a position of 1 (ref.rotate, at an angle of at most half a turn): a step is off by at most
    2^-65 of a turn, which 2^31 positions make 2^-34 of one, 2 pi 2^-34 radians; the bound has 2^-22 for the sine's own
    error, of which sincospif takes at most half."""
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 1 << 30, -1999999973, 1, 0]
    T, heads, D = len(pos), 2, 128
    x = torch.randn((T, heads * D), generator=torch.Generator().manual_seed(1)).cuda()
    y = torch.empty_like(x)
    d = gdn.dims(1, heads, D, io_dtype=torch.float32)
    table = gdn.rope_spec(D, layout=int(interleaved), base=base)
    gdn.gdn_rope(d, table, torch.tensor(pos, dtype=torch.int32, device="cuda"), q=x, q_out=y)
    turns = rope_exact.turns(D, base)
    for t, p in enumerate(pos):
        angles = np.array([rope_exact.angle(p, f) for f in turns])
        want, tol = ref.rotate(ref.f64(x[t:t + 1]).reshape(1, heads, D), np.array([1]), angles, interleaved, 1.0, "f32")
        ref.check(ref.f64(y[t:t + 1]).reshape(want.shape), want, tol, f"position {p}")
