"""A softmax attention layer of a hybrid model as it is used: prompts whose queries and keys are rotated and whose keys and
values go into a cache, then single tokens, then tokens behind a shared prefix, each against fp64."""

import numpy as np
import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hq,hk,D,rotary,interleaved", [(8, 2, 128, 64, False), (4, 4, 64, 64, True)])
def test_prompt_then_tokens(dtype, hq, hk, D, rotary, interleaved):
    """The checks take the rotated queries and keys as the call rounded them, after checking those themselves."""
    gen = torch.Generator().manual_seed(D)
    io, capacity = ref.DT[dtype], 400
    lengths = [200, 1, 77]
    n = len(lengths)
    d = gdn.dims(hk, hq, D, io_dtype=io)
    table = gdn.rope_spec(rotary, layout=int(interleaved), base=1e5)
    freq = ref.frequencies(rotary, 1e5)
    kc = torch.full((n * capacity, hk * D), float("nan"), device="cuda", dtype=io)  # rows not written yet
    vc = kc.clone()
    start = torch.arange(n, dtype=torch.int32, device="cuda") * capacity
    have = [0] * n
    for new in (lengths, [1] * n, [1] * n, [5, 2, 1]):
        T = sum(new)
        act = torch.randn((T, (hq + 2 * hk) * D), generator=gen).to(io).cuda()
        pos = torch.cat([torch.arange(h, h + m) for h, m in zip(have, new)]).to(torch.int32).cuda()
        rows = torch.cat([torch.arange(h, h + m) + i * capacity for i, (h, m) in enumerate(zip(have, new))])
        q, k, v = act[:, :hq * D], act[:, hq * D:(hq + hk) * D], act[:, (hq + hk) * D:]
        k_before = k.clone()
        qr = torch.empty((T, hq * D), device="cuda", dtype=io)
        gdn.gdn_rope(d, table, pos, q=q, q_out=qr, k=k, k_out=kc, v=v, v_out=vc, cache_rows=rows.to(torch.int32).cuda())
        have = [h + m for h, m in zip(have, new)]
        out = torch.empty((T, hq, D), device="cuda", dtype=io)
        cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
        gdn.gdn_attn_prefill(d, cu, qr, kc, vc, out, kv_start=start,
                             kv_len=torch.tensor(have, dtype=torch.int32, device="cuda"))
        p = ref.f64(pos)
        for x, got in ((q, qr), (k_before, kc[rows.cuda()])):
            y, tol = ref.rotate(ref.f64(x).reshape(T, -1, D), p, freq, interleaved, 1.0, dtype)
            ref.check(ref.f64(got).reshape(y.shape), y, tol, "rotated")
        at = 0
        for i, m in enumerate(new):
            keep = slice(i * capacity, i * capacity + have[i])
            o, tol, _, _ = ref.attention(ref.f64(qr[at:at + m]).reshape(m, hq, D), ref.f64(kc[keep]).reshape(-1, hk, D),
                                         ref.f64(vc[keep]).reshape(-1, hk, D), ref.causal(m, have[i]), D ** -0.5, dtype)
            ref.check(ref.f64(out[at:at + m]), o, tol, f"sequence {i}")
            at += m
    # the first sequence's first 128 keys as a prefix that all of them share
    q = torch.randn((n, hq * D), generator=gen).to(io).cuda()
    out = torch.empty((n, hq, D), device="cuda", dtype=io)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    gdn.gdn_attn_shared(d, i32([0, 1, 2, 3]), q, kc, vc, start, i32(have), i32([0, n]), i32([0]), i32([128]), out)
    for i in range(n):
        rows = np.concatenate([np.arange(128), np.arange(i * capacity, i * capacity + have[i])])
        k, v = (ref.f64(t)[rows].reshape(-1, hk, D) for t in (kc, vc))
        o, tol, _, _ = ref.attention(ref.f64(q[i:i + 1]).reshape(1, hq, D), k, v, np.ones((1, len(rows)), bool), D ** -0.5,
                                     dtype)
        ref.check(ref.f64(out[i:i + 1]), o, tol, f"shared, sequence {i}")
