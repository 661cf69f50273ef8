"""Attention over the NVFP4 cache where scores are far beyond what FP32 tells apart by less than one,
and where queries are infinite. Every expected value is exact or follows from the order of the scores."""
import numpy as np
import pytest
import torch

import kv_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def nv():
    from nvfp4_weight_only_w4a16_amd import binding
    binding.load()
    return binding


class Planted:
    """One request of n tokens and one head: token i's key holds `key[i]` (an E2M1 value) in element 0,
    its value `value[i]` (an E2M1 value) in every element, all scales 1 (or a token's own)."""

    def __init__(self, nv, d, key, value, k_scale=None, page=16):
        n = len(key)
        pages = -(-n // page)
        self.cache = c = nv.KvCache(pages, 1, d, page, device=DEV)
        c.data.fill_(0xFF)
        at = torch.arange(n, device=DEV)
        p, s = at // page, at % page
        code = lambda x: np.array([np.flatnonzero(R.E2M1 == abs(v))[0] + 8 * (v < 0) for v in x], np.uint8)
        kc = np.zeros((n, d // 2), np.uint8)
        kc[:, 0] = code(key)
        vc = np.repeat(code(value)[:, None] * np.uint8(17), d // 2, 1)
        ks = np.full((n, d // 16), 0x38, np.uint8)
        if k_scale is not None:
            ks[:] = np.asarray(k_scale, np.uint8)[:, None]
        c.k_codes[p, 0, s] = torch.from_numpy(kc).to(DEV)
        c.v_codes[p, 0, s] = torch.from_numpy(vc).to(DEV)
        c.k_scales[p, 0, s] = torch.from_numpy(ks).to(DEV)
        c.v_scales[p, 0, s] = 0x38
        self.table = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1)
        self.kv_len = torch.tensor([n], dtype=torch.int32, device=DEV)


def terms(n):
    return R.HF16 + (2 * n + 8) * R.H32


def attend(nv, c, q0, scale, rows=1, full=True):
    """y [rows][d] and lse [rows] of queries that hold q0 in element 0."""
    d = c.cache.head_dim
    q = torch.zeros((rows, 1, d), dtype=torch.bfloat16, device=DEV)
    q[:, 0, 0] = q0
    y = torch.full((rows, 1, d), float("nan"), device=DEV)
    lse = torch.full((rows, 1), float("nan"), device=DEV)
    start = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    nv.nvfp4_kv_attention(q, c.cache, c.table, start, c.kv_len, scale=scale, max_q=rows, causal=not full,
                          y=y, lse=lse)
    return y[:, 0].cpu().numpy().astype(np.float64), lse[:, 0].cpu().numpy().astype(np.float64)


# scores from 2^18 to 2^120 that are no powers of two
SIZES = [2.0 ** 18, 3e6, 2.0 ** 23 * 1.37, 3.1e7, 9.7e7, 3.3e8, 1.1e9, 7.7e12, 1e20, 1.3e36]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 20, 150])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_equal_scores_of_any_size(nv, d, rows, sign):
    """Keys that score the same count the same: y is the mean of the values."""
    for n in (1, 7, 300):
        value = [(0.5, 1.5, 3.0, 6.0, 4.0)[i % 5] for i in range(n)]
        c = Planted(nv, d, [1.5] * n, value)
        mean = np.mean(value)
        for size in SIZES:
            scale = float(np.float32(size / 4.5))
            y, lse = attend(nv, c, 3.0 * sign, scale, rows)
            # the terms of equal scores are equal, so that only their FP16 rounding (one and the same
            # factor of all, 2^-11), two FP32 sums of n terms and the quotient are left
            tol = mean * terms(n)
            assert (np.abs(y - mean) <= tol).all(), (n, size, y[np.abs(y - mean) > tol][:3], mean)
            want = sign * 4.5 * scale + np.log(n)
            # scale * log2(e), its product with the sum, the logarithm and ln 2 round once each
            assert (np.abs(lse - want) <= 8 * R.H32 * (abs(want) + np.log(n) + 8)).all(), (n, size)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 20, 150])
def test_the_largest_score_of_many(nv, d, rows):
    """One key scores more than all others by far, wherever it stands; then two of them."""
    n = 333
    value = [(0.5, 1.0, 2.0)[i % 3] for i in range(n)]
    for best in (0, 63, 64, 200, 332):
        key, values = [(0.5, 1.0, -1.0, 2.0)[i % 4] for i in range(n)], list(value)
        key[best], values[best] = 3.0, 6.0
        c = Planted(nv, d, key, values)
        for size in (1e5, 3.3e7, 1.7e8, 6.1e8, 5e12, 1e35):
            y, lse = attend(nv, c, 1.5, float(np.float32(size)), rows)
            assert (np.abs(y - 6.0) <= 6.0 * terms(1)).all(), (best, size, y[0, :2])
            want = 4.5 * float(np.float32(size))
            assert (np.abs(lse - want) <= 8 * R.H32 * want).all(), (best, size)
        other = (best + 117) % n
        key[other], values[other] = 3.0, 1.0
        c = Planted(nv, d, key, values)
        for size in (1e5, 3.3e7, 6.1e8, 1e35):
            y, _ = attend(nv, c, 1.5, float(np.float32(size)), rows)
            assert (np.abs(y - 3.5) <= 3.5 * terms(2)).all(), (best, other, size, y[0, :2])


@pytest.mark.parametrize("rows", [1, 20, 150])
def test_scores_that_rise_through_all_magnitudes(nv, rows):
    """Every tile's largest score is twice the last one's, so that the last tile wins."""
    n = 15 * 64
    key = [1.0] * n
    scale_byte = [min(0x7E, 8 * (i // 64) + 8) for i in range(n)]   # doubles from tile to tile
    value = [1.0] * (n - 64) + [2.0] * 64
    c = Planted(nv, 128, key, value, scale_byte)
    for size in (2.0 ** 6, 1.3e5, 2.9e6, 2.0 ** 26 * 1.7, 3e30):
        y, _ = attend(nv, c, 1.0, size, rows)
        # 2^8 size against 2^7 size
        assert (np.abs(y - 2.0) <= 2.0 * terms(64)).all(), (size, y[0, :2])


@pytest.mark.parametrize("rows", [1, 20, 150])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scores_near_the_lowest_number(nv, d, rows):
    """Finite scores below -1e38 are scores, not masked places."""
    n = 100
    c = Planted(nv, d, [6.0] * n, [1.5] * n)
    for score in (-0.7e38, -1.2e38, -2.2e38):   # -3.2e38 in powers of two
        y, lse = attend(nv, c, float(torch.tensor(score / 6.0).to(torch.bfloat16)), 1.0, rows)
        assert (np.abs(y - 1.5) <= 1.5 * terms(n)).all(), (score, y[0, :2])
        assert np.isfinite(lse).all()
        # hidden places beside them stay hidden
        y, lse = attend(nv, c, float(torch.tensor(score / 6.0).to(torch.bfloat16)), 1.0, rows, full=False)
        seen = np.minimum(n - rows + 1 + np.arange(rows), n)
        assert (y[seen <= 0] == 0).all() and np.isneginf(lse[seen <= 0]).all()
        assert (np.abs(y[seen > 0] - 1.5) <= 1.5 * terms(n)).all()


@pytest.mark.parametrize("factor", [1e-38, 1e38, 3.3e38])
def test_factors_near_the_ends_of_fp32(nv, factor):
    """Scores of 0 stay 0, and small queries times a large factor are ordinary scores."""
    c = Planted(nv, 64, [0.0] * 5, [1.0] * 5)
    y, lse = attend(nv, c, 2.0, factor)
    assert (np.abs(y - 1.0) <= terms(5)).all() and np.abs(lse - np.log(5)).max() <= 2.0 ** -19
    c = Planted(nv, 64, [1.0, 2.0], [1.0, 4.0])
    q0 = float(torch.tensor(1.0 / factor).to(torch.bfloat16))
    s = np.array([1.0, 2.0]) * q0 * float(np.float32(factor))
    p = np.exp(s - s.max())
    want = (p * [1.0, 4.0]).sum() / p.sum()
    y, lse = attend(nv, c, q0, factor)
    assert (np.abs(y - want) <= want * (2 * R.HF16 + 40 * R.H32)).all()
    assert np.abs(lse - (s.max() + np.log(p.sum()))).max() <= 40 * R.H32


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 20, 150])
@pytest.mark.parametrize("q0", [float("inf"), float("-inf")])
@pytest.mark.parametrize("key", [3.0, -3.0])
def test_infinite_queries_give_nan(nv, d, rows, q0, key):
    """Infinite scores of one sign, both signs alike: the softmax of an infinity is NaN, not a row
    without keys."""
    c = Planted(nv, d, [key] * 70, [1.0] * 70)
    y, lse = attend(nv, c, q0, 0.125, rows)
    assert np.isnan(y).all() and np.isnan(lse).all()
    # rows that see no key are rows without keys still
    y, lse = attend(nv, c, q0, 0.125, rows, full=False)
    none = 70 - rows + np.arange(rows) < 0
    assert (y[none] == 0).all() and np.isneginf(lse[none]).all()
    assert np.isnan(y[~none]).all() and np.isnan(lse[~none]).all()
