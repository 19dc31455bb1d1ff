"""Plain fp64 references of linear attention with a decay for each head, of
the residual RMS norm with 8-bit output and of the 8-bit linear layer, with
the magnitudes that their error bounds are made of.

u = 2^-24 is half an fp32 step relative to the value. For the recurrence
S_t = a_t S_{t-1} + v_t k_t^T let A_t = a_t A_{t-1} + |v_t| |k_t|^T be the same
with magnitudes, and B_t = a_t B_{t-1} + A_t. A token's update in fp32 is off
by at most 6 u A_t: four u for exp (CUDA's expf is within 2 ulp; g is an
input, so exact), one for a S, one for the sum. So the state is off by at
most 6 u B_t at token t. An output, a sum of D products in fp32, adds at most
(D + 2) u times the sum of magnitudes.

Kernels that keep their operands as sums of 16-bit parts are allowed `split`
more, relative to those same sums of magnitudes.
"""

from __future__ import annotations

import numpy as np

U = 2.0 ** -24
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}  # half the smallest step


def k_head(h, hk, hv, tiled):
    return h % hk if tiled else h // (hv // hk)


def recurrence(q, k, v, g, S0, scale, tiled):
    """One sequence: q, k [T][Hk][D], v [T][Hv][D], g [T][Hv], S0 [Hv][D][D]
    (all fp64). Returns o [T][Hv][D], the state, and their error scales: for o
    the fp32 bound and the sum of magnitudes, for the state the same."""
    T, hk, D = k.shape
    hv = v.shape[1]
    heads = np.array([k_head(h, hk, hv, tiled) for h in range(hv)])
    S, A, B = S0.copy(), np.abs(S0), np.zeros_like(S0)
    o = np.zeros((T, hv, D))
    bound, mag = np.zeros_like(o), np.zeros_like(o)
    for t in range(T):
        with np.errstate(invalid="ignore"):
            a = np.exp(g[t])[:, None, None]
        kt, qt = k[t][heads], q[t][heads]
        S = a * S + v[t][:, :, None] * kt[:, None, :]
        A = a * A + np.abs(v[t])[:, :, None] * np.abs(kt)[:, None, :]
        B = a * B + A
        aq = np.abs(qt)[:, :, None]
        o[t] = (S @ qt[:, :, None])[..., 0] * scale
        mag[t] = (A @ aq)[..., 0] * abs(scale)
        bound[t] = 6 * U * (B @ aq)[..., 0] * abs(scale) + (D + 2) * U * mag[t]
    return o, S, bound, mag, 6 * U * B, A


def gated(o, z, w, eps, dtype, do):
    """The gated norm of o and its bound: o off by do moves y_j through o_j and
    through the root; rounding is half a step; the fp32 arithmetic of the
    norm and of silu is allowed 64 u."""
    r = 1.0 / np.sqrt(np.mean(o * o, axis=-1, keepdims=True) + eps)
    gate = w * z / (1.0 + np.exp(-z))
    y = o * r * gate
    through_root = np.minimum(1.0, r * np.sqrt(np.mean(do * do, axis=-1, keepdims=True)))
    bound = (np.abs(gate) * r * do + np.abs(y) * 2 * through_root) * (1 + 2 ** -6)
    return y, bound + (HALF_STEP[dtype] * (1 + 2 ** -6) + 64 * U) * np.abs(y) + TINY[dtype]


def rounded(o, dtype, do):
    return do * (1 + 2 ** -6) + HALF_STEP[dtype] * np.abs(o) + TINY[dtype]


def check(got, ref, bound, what):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), f"{what}: values that are not finite"
    err = np.abs(got - ref)
    over = err - bound
    assert over.max(initial=-1.0) <= 0, (
        f"{what}: {int((over > 0).sum())} of {err.size} beyond the bound; worst error {err.flat[over.argmax()]:.3e}, "
        f"allowed {np.broadcast_to(bound, err.shape).flat[over.argmax()]:.3e} "
        f"at {np.unravel_index(over.argmax(), err.shape)}")
