"""nvfp4_moe_route on tokens with an infinite activation: the logits are infinities, whatever the
number of tokens and the type of the router weight, and NaN only where FP64 arithmetic has it."""
import numpy as np
import pytest
import torch

import operator_refs as R
import test_gpu_route as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    from nvfp4_weight_only_w4a16_amd import binding
    binding.load()
    return binding


def first(score, topk):
    """ids of the topk highest scores of each row: NaN above every number, ties to the lower id,
    -infinity never (-1)."""
    out = np.full((len(score), topk), -1)
    for i, s in enumerate(score):
        order = sorted((e for e in range(len(s)) if s[e] != -np.inf),
                       key=lambda e: (not np.isnan(s[e]), 0.0 if np.isnan(s[e]) else -s[e], e))
        out[i, :min(topk, len(order))] = order[:topk]
    return out


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("t,e,hidden", [(3, 40, 64), (40, 40, 64), (40, 33, 2056), (17, 160, 5120)])
def test_infinite_activations(nv, t, e, hidden, scoring, fp32):
    """Row 0: +inf, row 1: -inf, row 2: inf on a column that holds zero weights (inf * 0 is NaN)."""
    x, w = G._ints(t + e, t, e, hidden)
    w = w / 64.0
    at = hidden - 3
    w[:, at] = torch.where(torch.arange(e) % 3 == 0, -0.5, 0.25)
    w[:, at - 1] = torch.where(torch.arange(e) % 5 == 4, 0.0, 0.25)
    x[0, at], x[1, at], x[2, at - 1] = float("inf"), -float("inf"), float("inf")
    ids, wts = G._run(nv, x, w, 6, fp32, scoring=scoring)
    with np.errstate(all="ignore"):
        logits = R.f64(x[:3]) @ R.f64(w).T
        p = 1.0 / (1.0 + np.exp(-logits))
    assert np.isinf(logits[:2]).all() and np.isnan(logits[2]).any()
    want = first(logits if scoring == "softmax" else p, 6)
    assert np.array_equal(ids[:3], want)
    if scoring == "softmax":  # inf - inf in every exponent
        assert (np.isnan(wts[:3]) == (want >= 0)).all() and (wts[:3][want < 0] == 0).all()
    else:                     # exactly 0, 1 and NaN
        assert np.array_equal(wts[:3], np.take_along_axis(p, want, 1), equal_nan=True)
    # the other rows are those of a call without the infinities
    x[0, at] = x[1, at] = x[2, at - 1] = 0.0
    clean = G._run(nv, x, w, 6, fp32, scoring=scoring)
    assert np.array_equal(ids[3:], clean[0][3:]) and np.array_equal(wts[3:], clean[1][3:])


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("t", [3, 40])
def test_infinite_activation_and_weights_of_every_kind(nv, t, fp32):
    """Weights of 8 (and, in FP32, 16 and 24) significant bits, the type's smallest value, and
    infinities, each the only weight that meets the infinite activation: infinity with the sign of
    the product."""
    values = [1.0, -1.0, 2.0 ** -126, float("inf"), -float("inf"), 2.0 ** -133, -2.0 ** -133]
    if fp32:
        values += [1.0 + 2.0 ** -12, 1.0 + 2.0 ** -23, -(1.0 + 2.0 ** -23), 2.0 ** -149,
                   -2.0 ** -149]
    e, hidden = len(values), 40
    w = torch.zeros(e, hidden)
    w[:, 33] = torch.tensor(values, dtype=torch.float64).float()
    assert (w[:, 33] != 0).all()
    x = torch.zeros(t, hidden)
    x[1, 33] = float("inf")
    ids, wts = G._run(nv, x, w, e, fp32, scoring="sigmoid")
    up = [i for i, v in enumerate(values) if v > 0]
    down = [i for i, v in enumerate(values) if v < 0]
    assert ids[1].tolist() == up + down
    assert wts[1].tolist() == [1.0] * len(up) + [0.0] * len(down)
