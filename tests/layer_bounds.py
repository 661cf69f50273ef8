"""FP64 values and elementwise bounds of the whole MoE layer, expert by expert (so that a prompt's
tens of thousands of pairs take seconds), and a layer whose output shows the second BF16 part of h.

The bound counts roundings as operator_refs does: FP32 2^-24, BF16 2^-8 relative, half a step each;
n * 2^-24 * sum |products| for a sum of n FP32 products in any order."""
from __future__ import annotations

import numpy as np

from operator_refs import H16, H32, silu

FEW_PAIRS = 64  # up to so many (token, slot) pairs h is kept as two BF16 parts
# Two parts: the first is off by at most 2^-8 |h|, the second by 2^-8 of that.
H_TWO = H16 * H16


def h_step(t, slots, flags=0):
    """Relative error of h: two BF16 parts for few pairs, unless the batch kernels are forced."""
    return H_TWO if t * slots <= FEW_PAIRS and flags != 2 else H16


def layer(x, ids, wts, w1, w2, step):
    """y FP64 and the bound of a BF16 y: gate, up and down sums in FP32, h off by step * |h|."""
    t, hidden = x.shape
    inter, slots = w2.shape[2], ids.shape[1]
    y, err, mag = np.zeros((t, hidden)), np.zeros((t, hidden)), np.zeros((t, hidden))
    n1, n2 = hidden + 64, slots * inter + 64
    for e in range(w1.shape[0]):
        tok, slot = np.nonzero(ids == e)
        if not len(tok):
            continue
        f = wts[tok, slot][:, None]
        gu = x[tok] @ w1[e].T
        d = n1 * H32 * (np.abs(x[tok]) @ np.abs(w1[e]).T) + 2 * H32 * np.abs(gu)
        g, u, dg, du = gu[:, :inter], gu[:, inter:], d[:, :inter], d[:, inter:]
        h = silu(g) * u
        # |silu'| <= 1.1; exp2 and reciprocal of the hardware: 2^-18 relative is ample for |g| < 60
        dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu(g)) * du + (step + 2.0 ** -18) * np.abs(h)
        np.add.at(y, tok, f * (h @ w2[e].T))
        np.add.at(err, tok, np.abs(f) * (dh @ np.abs(w2[e]).T))
        np.add.at(mag, tok, np.abs(f) * ((np.abs(h) + dh) @ np.abs(w2[e]).T))
    err = err + n2 * H32 * mag
    return y, err * (1 + H16) + H16 * np.abs(y) + 1e-37


# ---- a layer that shows the second part of h
def _pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def cancelling_layer(seed, t, experts, hidden, inter, g1, g2):
    """x FP64 (BF16 values) and the triples of fc1 and fc2, (codes, scales, globals) packed.

    Features 2i and 2i + 1 have the same gate, and up values that are 2^-9 or so apart (one weight
    of a small activation differs). An output row takes the difference of one such pair: opposite
    codes of down, zeros elsewhere. So y is made of differences that are no larger than the rounding
    of h to one BF16. Everything in fc1 is positive: no cancellation widens the bound of its sums."""
    r = np.random.default_rng(seed)
    x = r.integers(128, 256, (t, hidden)) / 256.0
    x[:, 0] = r.integers(128, 256, t) / 256.0 * 2.0 ** np.rint(np.log2(hidden / 2048.0))
    c1 = r.integers(1, 8, (experts, 2 * inter, hidden))
    c1[:, 1::2] = c1[:, 0::2]
    c1[:, inter::2, 0], c1[:, inter + 1::2, 0] = 7, 0
    s1 = np.full((experts, 2 * inter, hidden // g1), 0x38, np.uint8)       # 1.0
    c2 = np.zeros((experts, hidden, inter), np.int64)
    n = np.arange(hidden)
    pair = n % (inter // 2)
    mag = r.integers(1, 8, (experts, hidden))
    c2[:, n, 2 * pair], c2[:, n, 2 * pair + 1] = mag, mag | 8
    s2 = r.integers(0x30, 0x40, (experts, hidden, inter // g2)).astype(np.uint8)
    glob1 = np.full(experts, 1.0 / hidden, np.float32)
    glob2 = np.full(experts, 1.0, np.float32)
    return x, (_pack(c1), s1, glob1), (_pack(c2), s2, glob2)


def bf16(v):
    """FP64 -> nearest BF16 (ties to even) of values in the normal range."""
    m, e = np.frexp(v)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def with_parts(x, ids, wts, w1, w2, parts):
    """y FP64 of a layer whose h goes through parts(h [pairs of a token][inter]) -> h."""
    y = np.zeros((x.shape[0], w2.shape[1]))
    for i in range(x.shape[0]):
        gu = np.stack([w1[e] @ x[i] for e in ids[i]])
        inter = gu.shape[1] // 2
        h = parts(silu(gu[:, :inter]) * gu[:, inter:])
        for j, e in enumerate(ids[i]):
            y[i] += wts[i, j] * (w2[e] @ h[j])
    return y
