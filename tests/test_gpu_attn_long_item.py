"""A single token whose keys take one CTA several seconds, longer than any one wait of the kernel may last."""

import time

import pytest
import torch

import gated_delta_net_causal_gb300 as gdn

pytestmark = pytest.mark.gpu


def test_one_token_on_a_cache_of_seconds():
    """Without a workspace the keys are one CTA's, and the half of it that has no row waits for all of them. Keys are
    zeros, but for the last one, whose score of 1024 / sqrt(32) leaves every other weight at 0: the output is its value,
    lse its score but for four roundings of 2^-24 of it (the factor of the scores, the product, and back)."""
    n, D = 800_000_000, 32
    d = gdn.dims(1, 1, D)
    kv = torch.zeros((n, D), device="cuda", dtype=torch.bfloat16)
    kv[-1] = 32.0
    q = torch.ones((1, D), device="cuda", dtype=torch.bfloat16)
    out, lse = torch.empty((1, 1, D), device="cuda", dtype=torch.bfloat16), torch.empty((1, 1), device="cuda")
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    args = d, i(0, 1), q, kv, kv, out
    stretch = {"kv_start": i(0), "kv_len": i(n)}
    torch.cuda.synchronize()
    start = time.monotonic()
    gdn.gdn_attn_prefill(*args, lse=lse, workspace=None, **stretch)
    torch.cuda.synchronize()
    took = time.monotonic() - start
    del kv, args
    torch.cuda.empty_cache()
    assert gdn.gdn_device_error() == 0
    assert (out == 32.0).all()
    assert abs(float(lse) - 1024 * D ** -0.5) <= 4 * 2.0 ** -24 * 182
    print(f"{took:.2f} s")
    assert took > 2.5  # else the case does not show what it is for
