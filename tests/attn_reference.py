"""Softmax attention and rotary positions from their definitions in fp64, with bounds on what the kernels' roundings can
add, made of the inputs' magnitudes."""

import math

import numpy as np
import torch

UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # half a step, relative to the value
SMALLEST = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half the smallest step
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def head_of(h, hq, hk, tiled):
    return h % hk if tiled else h // (hq // hk)


def attention(q, keys, values, visible, scale, dtype, tiled=False):
    """q [n][hq][D]; keys, values: a list of [m][hk][D] for each token, or one for all; visible [n][m] bool. Returns
    out, its bound, lse, its bound. The bound:

    a score is a sum of D products, each exact (16-bit inputs) or off by 2^-24 of itself, added in fp32 with sums that
    may be cut off instead of rounded: (D + 4) 2^-23 of the sum of magnitudes; scaling and taking the maximum off adds
    2 2^-24 of the scaled score's and maximum's magnitude. That error e of the exponents is one of e relative in a
    weight, at most 2 e after the division by the sum. An exponential is off by 2^-22 of itself, the sums over m keys by
    (m + 4) 2^-23, a weight rounded to 16 bits by half a step (its sum is taken before that), relative to the weights'
    magnitudes times the values'; the output's own rounding comes last. Weights below fp16's normal range are off by
    half its smallest step at worst, of a largest weight of at least 2^-1 (the fp16 kernel scales by more)."""
    n, hq, D = q.shape
    hk = keys.shape[-2]
    u = UNIT[dtype]
    out, tol = np.zeros((n, hq, D)), np.zeros((n, hq, D))
    lse, ltol = np.full((n, hq), -np.inf), np.zeros((n, hq))
    m = visible.shape[1]
    for h in range(hq):
        kh = head_of(h, hq, hk, tiled)
        k, v = keys[:, kh], values[:, kh]
        s = scale * (q[:, h] @ k.T)
        e = scale * (np.abs(q[:, h]) @ np.abs(k).T) * (D + 4) * 2.0 ** -23 + 4 * 2.0 ** -24 * np.abs(s)
        s = np.where(visible, s, -np.inf)
        some = visible.any(1)
        if not some.any():
            continue
        top = s.max(1, keepdims=True, initial=-np.inf, where=visible)
        top = np.where(np.isfinite(top), top, 0.0)
        e = np.where(visible, e + 4 * 2.0 ** -24 * np.abs(top), 0.0).max(1, keepdims=True)
        w = np.where(visible, np.exp(s - top), 0.0)
        total = w.sum(1, keepdims=True)
        safe = np.where(total > 0, total, 1.0)
        w = w / safe
        vz = np.where(np.isfinite(v), v, 0.0)
        o = w @ vz
        mag = w @ np.abs(vz)
        rel = 2 * e + 2.0 ** -21 + (m + 4) * 2.0 ** -22
        if dtype != "f32":
            rel = rel + u
            mag_small = 2 * SMALLEST[dtype] * (visible @ np.abs(vz)) / np.maximum(safe, 1.0)
        else:
            mag_small = 0.0
        err = mag * rel + mag_small
        out[:, h] = np.where(some[:, None], o, 0.0)
        tol[:, h] = err + u * (np.abs(o) + err) + SMALLEST[dtype]
        lse[:, h] = np.where(some, (top + np.log(safe))[:, 0], -np.inf)
        ltol[:, h] = (e[:, 0] + (m + 4) * 2.0 ** -23 + 4 * 2.0 ** -24 * (np.abs(np.where(some, lse[:, h], 0.0)) + 1) + 2.0 ** -21)
    return out, tol, lse, ltol


def causal(n, m):
    """What token i of n new ones sees of m keys."""
    return np.arange(m)[None, :] <= (m - n + np.arange(n))[:, None]


def check(got, want, tol, what):
    assert got.shape == want.shape, (what, got.shape, want.shape)
    with np.errstate(invalid="ignore"):  # -inf less -inf, where they are equal
        same = (got == want) | (np.abs(got - want) <= tol)
    assert same.all(), (f"{what}: {int((~same).sum())} of {same.size} beyond the bound, at "
                        f"{[tuple(int(i) for i in x) for x in np.argwhere(~same)[:4]]}: got {got[~same][:4]}, "
                        f"want {want[~same][:4]}, bound {np.broadcast_to(tol, got.shape)[~same][:4]}")


def frequencies(rotary, base, scaling="plain", factor=1.0, length=0.0, low=0.0, high=0.0):
    f = []
    for i in range(rotary // 2):
        b = base ** (-2.0 * i / rotary)
        if scaling == "linear":
            b /= factor
        elif scaling == "bands":
            n = length * b / (2 * math.pi)
            w = min(max((n - low) / (high - low), 0.0), 1.0)
            b *= w + (1 - w) / factor
        elif scaling == "ramp":
            at = lambda n: rotary * math.log(length / (2 * math.pi * n)) / (2 * math.log(base))
            first, last = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rotary - 1)
            w = 1 - min(max((i - first) / max(last - first, 0.001), 0.0), 1.0)
            b *= w + (1 - w) / factor
        f.append(b)
    return np.array(f)


def rotate(x, pos, freq, interleaved, amplitude, dtype, inverse=False):
    """x [T][h][D] rotated, and its bound: the angle is off by 2^-53 of itself (its own step in fp64) and, as a fraction
    of a turn in fp32, by 2^-24 of at most half a turn, pi 2^-24; sine and cosine by 2^-22 more, the amplitude, the two
    products and their sum by 2^-24 each; then the output's rounding."""
    R = 2 * len(freq)
    t = pos.astype(np.float64)[:, None, None] * freq
    c, s = amplitude * np.cos(t), amplitude * np.sin(t) * (-1 if inverse else 1)
    i1, i2 = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y, tol = x.copy(), np.zeros_like(x)
    x1, x2 = x[..., i1], x[..., i2]
    y[..., i1], y[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
    mag = abs(amplitude) * (np.abs(x1) + np.abs(x2))
    err = mag * (np.abs(t) * 2.0 ** -50 + math.pi * 2.0 ** -24 + 2.0 ** -22 + 4 * 2.0 ** -24)
    for i in (i1, i2):
        tol[..., i] = err + UNIT[dtype] * (np.abs(y[..., i]) + err) + SMALLEST[dtype]
    return y, tol
