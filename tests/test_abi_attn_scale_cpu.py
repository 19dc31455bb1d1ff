"""The largest and smallest scales of the attention calls, with addresses that are never used."""

import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from gated_delta_net_causal_gb300 import _build
from tests.test_abi_attn_cpu import ALIGN, ATTN, INVALID, SHARED, attn, shared

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer validation runs only without a GPU")


@no_gpu
@pytest.mark.parametrize("call,base", [(attn, ATTN), (shared, SHARED)])
def test_scale_whose_base_2_form_overflows(call, base):
    """The kernels take exponentials to base 2: 3.4e38 log2 e is not finite. (A workspace off its alignment, which is
    looked at later, stands for a scale that is taken.)"""
    _build.build()
    lib, d = gdn.library(), gdn.dims(8, 32, 128)
    off = base["ws"] + 128
    for s in (3.4e38, 2.36e38):
        assert call(lib, d, scale=s, ws=off) == INVALID, s
    for s in (2.35e38, 1.0, 1e-45):
        assert call(lib, d, scale=s, ws=off) == ALIGN, s
