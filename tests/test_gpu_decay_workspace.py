"""Scratch of gdn_decay_prefill: no more than the sequences that can be cut
need, and their segments in it apart."""

import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from gated_delta_net_causal_gb300 import _build
from tests.test_gpu_decay import Case, run_prefill


@pytest.mark.parametrize("io,D,hv,N,L", [(torch.float32, 128, 64, 128, 200), (torch.float16, 64, 32, 100, 300),
                                         (torch.bfloat16, 96, 64, 500, 40)])
def test_many_short_sequences_ask_for_little(io, D, hv, N, L):
    """Sequences of which few can outlast the rest: far less than the states themselves."""
    _build.build()
    need = gdn.gdn_decay_prefill_workspace_size(gdn.dims(hv, hv, D, io_dtype=io), N, N * L)
    assert need < N * hv * D * D * 4 / 4


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,hv,lengths", [
    ("f32", 32, 16, [300, 5, 0, 400, 176, 175, 174, 3] + [1, 20, 0, 7] * 8 + [500]),
    ("f16", 64, 16, [400, 399, 1, 2] + [3, 0, 9, 30] * 10),
    ("bf16", 128, 8, [1, 1200, 30, 20, 1500, 40, 0, 17, 25, 33, 1100]),
    ("bf16", 96, 16, [0, 0, 700] + [11] * 40 + [650, 0])])
def test_several_long_sequences_among_many(dtype, D, hv, lengths):
    T = sum(lengths)
    c = Case(81, hv // 2, hv, D, dtype, T + 4, len(lengths), rate=0.05)
    need = gdn.gdn_decay_prefill_workspace_size(c.d, len(lengths), T + 4)
    assert need > 0
    # a workspace of just that size, with a guard behind it
    buf = torch.full((need + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
    run_prefill(c, lengths, workspace=buf[:need])
    assert (buf[need:] == 0xa5).all()
