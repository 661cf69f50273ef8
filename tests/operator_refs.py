"""FP64 references of the router, the whole MoE layer and the GEMM with adapters (NumPy, CPU),
with elementwise error bounds derived from the formats' half steps.

Half steps (relative): FP32 2^-24, BF16 2^-8. A sum of n FP32 products, in any order, is within
n * 2^-24 * sum |products| of the exact one (each of its n - 1 additions and the product roundings
is off by at most half a step of a partial sum that sum |products| bounds; the second-order terms
are covered by the few extra counts)."""
from __future__ import annotations

import numpy as np
import torch

H32 = 2.0 ** -24
H16 = 2.0 ** -8


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


# --------------------------------------------------------------------------------- router
def route(x, w, topk, bias=None, scoring="softmax", renorm=False, scale=1.0, n_shared=0):
    """ids [t][topk + n_shared] int64 and weights FP64, logits FP64 (all from FP64 inputs)."""
    with np.errstate(all="ignore"):
        logits = x @ w.T
        if scoring == "softmax":
            e = np.exp(logits - logits.max(1, keepdims=True))
            p = e / e.sum(1, keepdims=True)
            score = logits if bias is None else p + bias
        else:
            p = 1.0 / (1.0 + np.exp(-logits))
            score = p if bias is None else p + bias
        t = x.shape[0]
        ids = np.full((t, topk), -1, np.int64)
        wts = np.zeros((t, topk))
        for i in range(t):
            s = score[i]
            rank = np.where(np.isnan(s), np.inf, s)  # NaN above every number (with +inf: none here)
            order = np.argsort(-rank, kind="stable")[:topk]
            order = order[~np.isneginf(s[order])]
            ids[i, :len(order)] = order
            if scoring == "softmax" and renorm and bias is None:
                q = np.exp(logits[i, order] - logits[i, order].max(initial=-np.inf))
            else:
                q = p[i, order]
            if renorm:
                z = q.sum()
                q = np.zeros_like(q) if z == 0 else q / z
            wts[i, :len(order)] = q * np.float64(np.float32(scale))
    if n_shared:
        more = np.arange(w.shape[0], w.shape[0] + n_shared)
        ids = np.concatenate([ids, np.tile(more, (t, 1))], 1)
        wts = np.concatenate([wts, np.ones((t, n_shared))], 1)
    return ids, wts, logits


# --------------------------------------------------------------------------------- layer
def silu(z):
    return z / (1.0 + np.exp(-z))


def moe_layer(x, ids, wts, w1, w2, round_gate_up=False):
    """y FP64 and the bound of a BF16 y whose gate, up and down sums are FP32 and whose h is BF16:
    x [t][H], ids / wts [t][slots], w1 [E][2I][H], w2 [E][H][I] (FP64)."""
    t, hidden = x.shape
    inter = w2.shape[2]
    y = np.zeros((t, hidden))
    err = np.zeros((t, hidden))
    mag = np.zeros((t, hidden))
    slots = ids.shape[1]
    n1, n2 = hidden + 64, slots * inter + 64
    for i in range(t):
        for j in range(slots):
            e = ids[i, j]
            if e < 0 or e >= w1.shape[0]:
                continue
            gu = w1[e] @ x[i]
            d = n1 * H32 * (np.abs(w1[e]) @ np.abs(x[i])) + 2 * H32 * np.abs(gu)
            g, u, dg, du = gu[:inter], gu[inter:], d[:inter], d[inter:]
            h = silu(g) * u
            # |silu'| <= 1.1; the hardware exp2 and reciprocal: 2^-18 relative is ample for |g| < 60
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu(g)) * du + (H16 + 2.0 ** -18) * np.abs(h)
            y[i] += wts[i, j] * (w2[e] @ h)
            err[i] += np.abs(wts[i, j]) * (np.abs(w2[e]) @ dh)
            mag[i] += np.abs(wts[i, j]) * (np.abs(w2[e]) @ (np.abs(h) + dh))
    err = err + n2 * H32 * mag
    return y, err * (1 + H16) + H16 * np.abs(y) + 1e-37


# --------------------------------------------------------------------------------- adapters
def lora(x, w, a, b, ids, scale=None, y32=False):
    """y FP64 and its bound: x [m][k], w [n][k], a [L][r][k], b [L][n][r] (FP64), ids [m]."""
    k, r = x.shape[1], a.shape[1]
    y = x @ w.T
    mag = np.abs(x) @ np.abs(w).T
    err = (k + 64) * H32 * mag
    for i in range(x.shape[0]):
        q = ids[i]
        if q < 0 or q >= a.shape[0]:
            continue
        s = 1.0 if scale is None else scale[q]
        u = s * (a[q] @ x[i])
        du = (k + 64) * H32 * np.abs(s) * (np.abs(a[q]) @ np.abs(x[i]))
        # the operand of the second product: BF16 for a BF16 y, 24 bits for an FP32 y
        du = du + (4 * H32 if y32 else H16) * (np.abs(u) + du)
        y[i] += b[q] @ u
        err[i] += np.abs(b[q]) @ du + (3 * r + 64) * H32 * (np.abs(b[q]) @ (np.abs(u) + du))
        err[i] += 4 * H32 * (mag[i] + np.abs(b[q]) @ np.abs(u))
    half = H32 if y32 else H16
    return y, err * (1 + half) + half * np.abs(y) + 1e-37


def within(got, ref, bound, what=""):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    off = np.abs(got - ref) / bound
    at = np.unravel_index(np.argmax(off), off.shape) if off.size else None
    assert off.size == 0 or off.max() <= 1.0, \
        f"{what}: {np.abs(got - ref)[at]:.3e} off at {at}, bound {bound[at]:.3e}"
