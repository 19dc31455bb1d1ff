"""gdn_decay_step of an empty batch over a pool, through the C ABI."""

import ctypes

import gated_delta_net_causal_gb300 as gdn
from gated_delta_net_causal_gb300 import _build


def test_no_rows_of_a_pool():
    _build.build()
    lib, d = gdn.library(), gdn.dims(2, 4, 64)
    call = lambda batch, num: lib.gdn_decay_step(ctypes.byref(d), batch, None, num, None, 128, None, 128, None, 256, None,
                                                 0, 0.1, None, None, None, 0, None, None, None)
    assert call(0, 3) == 0 and call(0, 0) == 0  # no table: that of no rows may have no address
    assert call(0, -1) == 1 and call(-1, 3) == 1 and call(2, 3) == 1
