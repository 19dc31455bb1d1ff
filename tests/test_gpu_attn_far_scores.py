"""Softmax attention where scores are large: queries and keys of small whole numbers and scales that are powers of two, so
that scores are exact, and either tie or differ by so much that one of them takes all."""

import numpy as np
import pytest
import torch

import gated_delta_net_causal_gb300 as gdn
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def inputs(seed, tokens, rows, hq, hk, D, dtype):
    gen = torch.Generator().manual_seed(seed)
    io = ref.DT[dtype]
    q = torch.randint(-4, 5, (tokens, hq * D), generator=gen).to(io).cuda()
    k = torch.randint(-4, 5, (rows, hk * D), generator=gen).to(io).cuda()  # |q . k| <= 16 D: exact in fp32
    v = torch.randn((rows, hk * D), generator=gen).to(io).cuda()
    return q, k, v


def check(c, q, k, v, out, lse, visible, scale):
    """Each row's output is the mean of the values whose scores tie for the largest. Bound: the weights are equal, but may
    be off a power of two, so that their rounding to 16 bits counts (their sum is taken before it); then the fp32 sums
    and the division, (n + 4) 2^-23 of the values' mean magnitude for n of them, and the output's rounding. lse: 2^-24 of
    itself for the scores' factor, their product, the sum of both logarithms, and the way back from log2, of up to 8 more
    than itself (7 of which the f16 kernel lifts the weights by)."""
    hq, hk, D, dtype = c
    Q, K, V = (ref.f64(x).reshape(x.shape[0], -1, D) for x in (q, k, v))
    o, l = ref.f64(out), ref.f64(lse)
    for h in range(hq):
        kh = h // (hq // hk)
        s = np.where(visible, Q[:, h] @ K[:, kh].T, -np.inf)
        top = s.max(1)
        tie = s == top[:, None]
        n = tie.sum(1)
        want = (tie @ V[:, kh]) / n[:, None]
        mag = (tie @ np.abs(V[:, kh])) / n[:, None]
        err = ((n[:, None] + 4) * 2.0 ** -23 + (ref.UNIT[dtype] if dtype != "f32" else 0.0)) * mag
        ref.check(o[:, h], want, err + ref.UNIT[dtype] * (np.abs(want) + err) + ref.SMALLEST[dtype], f"head {h}")
        w = scale * top + np.log(n)
        ref.check(l[:, h], w, 4 * 2.0 ** -24 * (np.abs(w) + 8), f"lse of head {h}")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("hq,hk,D", [(4, 2, 64), (2, 1, 128), (6, 1, 32)])
@pytest.mark.parametrize("power", [10, 15, 20, 24, 30, 60, 110])
def test_prompts(dtype, hq, hk, D, power):
    T = 333
    q, k, v = inputs(power, T, T, hq, hk, D, dtype)
    out, lse = torch.empty((T, hq, D), device="cuda", dtype=ref.DT[dtype]), torch.empty((T, hq), device="cuda")
    gdn.gdn_attn_prefill(gdn.dims(hk, hq, D, io_dtype=ref.DT[dtype]), ints(0, T), q, k, v, out, lse=lse,
                         scale=2.0 ** power)
    check((hq, hk, D, dtype), q, k, v, out, lse, ref.causal(T, T), 2.0 ** power)
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("workspace", ["auto", None])
@pytest.mark.parametrize("power", [12, 24, 40, 100])
def test_long_caches(dtype, workspace, power):
    """Parts of several CTAs, rising maxima, ties across parts, negative scores only."""
    hq, hk, D, m = 4, 1, 64, 6000
    q, k, v = inputs(power, 3, m, hq, hk, D, dtype)
    q[2] = -q[2].abs() - 1  # the last token's scores
    k[:, :] = k.abs() + 1   # are all negative
    d = gdn.dims(hk, hq, D, io_dtype=ref.DT[dtype])
    out, lse = torch.empty((3, hq, D), device="cuda", dtype=ref.DT[dtype]), torch.empty((3, hq), device="cuda")
    gdn.gdn_attn_prefill(d, ints(0, 1, 3), q, k, v, out, lse=lse, scale=2.0 ** power, kv_start=ints(0, 0),
                         kv_len=ints(m, m), workspace=workspace)
    see = np.concatenate([ref.causal(1, m), ref.causal(2, m)])
    check((hq, hk, D, dtype), q, k, v, out, lse, see, 2.0 ** power)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("steep", [0.25, 4.0, 64.0, 1024.0])
def test_scores_that_move_by_hundreds(dtype, order, steep):
    """Scores that rise or fall by up to a million over the keys in exact steps (a quarter and more of a key's): rising,
    every token's last visible key leads; falling, the first one. Against fp64, with the bound of exact scores: the
    exponents' differences are off by 2^-23 of themselves where they matter (up to 110; the rounding of the maximum is
    the same for all of a row); a sum's terms shrink by exp(-1/4) at least from one key to the next, so that after the
    67th they are below its roundings: 72 of 2^-23, less than 2^-16; weights and outputs as in attn_reference."""
    n, D = 1000, 64
    io = ref.DT[dtype]
    q = torch.zeros((n, D), device="cuda", dtype=io)
    k = torch.zeros((n, D), device="cuda", dtype=io)
    v = torch.randn((n, D), generator=torch.Generator().manual_seed(3)).to(io).cuda()
    i = torch.arange(n, device="cuda")
    q[:, 0], q[:, 1] = 32.0, 1.0
    k[:, 0], k[:, 1] = (i // 32).to(io), (i % 32).to(io)  # q . k = the key's index
    out, lse = torch.empty((n, 1, D), device="cuda", dtype=io), torch.empty((n, 1), device="cuda")
    scale = steep
    if order < 0:
        q = -q
    gdn.gdn_attn_prefill(gdn.dims(1, 1, D, io_dtype=io), ints(0, n), q, k, v, out, lse=lse, scale=scale)
    s = np.where(ref.causal(n, n), order * scale * np.arange(n)[None, :], -np.inf)
    top = s.max(1, keepdims=True)
    w = np.exp(s - top)
    total = w.sum(1, keepdims=True)
    V = ref.f64(v)
    want, mag = (w / total) @ V, (w / total) @ np.abs(V)
    off = 110 * 2.0 ** -23
    rel = 2 * off + 2.0 ** -21 + 2.0 ** -16 + (ref.UNIT[dtype] if dtype != "f32" else 0.0)
    err = mag * rel + 2 * ref.SMALLEST[dtype] * np.abs(V).sum(0)
    ref.check(ref.f64(out[:, 0]), want, err + ref.UNIT[dtype] * (np.abs(want) + err) + ref.SMALLEST[dtype], "out")
    want_lse = (top + np.log(total))[:, 0]
    ref.check(ref.f64(lse[:, 0]), want_lse, off + 2.0 ** -16 + 4 * 2.0 ** -24 * (np.abs(want_lse) + 8),
              "lse")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("power", [12, 24, 40, 100])
def test_shared_prefixes(dtype, power):
    """Odd scores over the prefix, even ones over the sequences' own keys, so that no tie lies across the two."""
    hq, hk, D, p, own = 4, 2, 64, 700, [5, 300, 40]
    n, rows = len(own), 700 + sum(own)
    q, k, v = inputs(power, n, rows, hq, hk, D, dtype)
    q[:, ::D] = 1.0  # each head's first element
    k *= 2
    k[:p, ::D] = 1.0
    start = [p, p + own[0], p + own[0] + own[1]]
    d = gdn.dims(hk, hq, D, io_dtype=ref.DT[dtype])
    out, lse = torch.empty((n, hq, D), device="cuda", dtype=ref.DT[dtype]), torch.empty((n, hq), device="cuda")
    gdn.gdn_attn_shared(d, ints(0, 1, 2, 3), q, k, v, ints(*start), ints(*own), ints(0, 2), ints(0), ints(p), out, lse=lse,
                        scale=2.0 ** power)
    see = np.zeros((n, rows), bool)
    for i in range(n):
        see[i, start[i]:start[i] + own[i]] = True
        see[i, :p] = i < 2  # the last sequence is outside of the group
    check((hq, hk, D, dtype), q, k, v, out, lse, see, 2.0 ** power)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_that_see_nothing_beside_far_ones(dtype):
    """Tokens without a key have zeros and -inf, whatever their neighbours' scores are."""
    hq, hk, D, power = 4, 2, 64, 30
    q, k, v = inputs(1, 9, 40, hq, hk, D, dtype)
    out, lse = torch.empty((9, hq, D), device="cuda", dtype=ref.DT[dtype]), torch.empty((9, hq), device="cuda")
    gdn.gdn_attn_prefill(gdn.dims(hk, hq, D, io_dtype=ref.DT[dtype]), ints(0, 5, 9), q, k, v, out, lse=lse,
                         scale=2.0 ** power, kv_start=ints(0, 2), kv_len=ints(2, 38))
    assert (out[:3] == 0).all() and (lse[:3] == -float("inf")).all()
    see = np.zeros((9, 40), bool)
    see[3, :1] = see[4, :2] = True
    see[5:, 2:] = ref.causal(4, 38)
    rows = slice(3, 9)
    check((hq, hk, D, dtype), q[rows], k, v, out[rows], lse[rows], see[rows], 2.0 ** power)
