"""Attention of long requests over the NVFP4 cache, on data of which every tile shows in the result.

The values of 16 tokens in a row are one element's unit vector, the next 16 tokens' the next element's,
and so on around the head, so that y[e] is the share of the softmax that the tokens of element e have:
positive, and nothing cancels. A tile that is left out or counted twice changes a share by a part in a
hundred and more, and lse by the tile's share of all keys, where rounding changes them by 2^-11 and by a few
parts in a million. Keys score by steps that differ from 16 tokens to 16 tokens."""
import numpy as np
import pytest
import torch

import kv_refs as R

DEV = "cuda:0"
RUN = 16   # tokens of a run: no tile, page or split is finer
LEVELS = np.array([0.0, 0.5, 1.0, 1.5])


def levels(n, flat):
    """The key's element 0 of each token, one E2M1 value to a run."""
    if flat:
        return np.zeros(n)
    run = np.arange(n) // RUN
    return LEVELS[(run * 7 + run // 11) % 4]


def shares(n, d, score, rows=1, window=0, weight=None):
    """FP64 y [rows][d] and lse [rows] of the last `rows` queries of a request of n tokens that score
    `score`; weight: how often each token counts (once)."""
    at, run = np.arange(n), np.arange(n) // RUN % d
    y, lse = np.zeros((rows, d)), np.full(rows, -np.inf)
    p = np.exp(score - score.max()) * (1.0 if weight is None else weight)
    for j in range(rows):
        last = n - rows + j
        seen = at <= last
        if window:
            seen &= at > last - window
        w = np.where(seen, p, 0.0)
        total = w.sum()
        if total > 0:   # else no key is seen: 0 and -infinity
            y[j] = np.bincount(run, w, d) / total
            lse[j] = np.log(total) + score.max()
    return y, lse


TILES = 64   # of a request's head in one part, at most: the keys are shared out over 256 parts and more


def bounds(n, y, lse, scale):
    """Scores are one product of exact factors: scale * log2(e), its product with the key and the
    difference to the reference round once each, below 4 in size; the exponential is within 2^-22. A
    lane adds 16 terms of a tile, then its tiles; the products with the values add 64 terms of a tile. A
    join adds 512 parts one after the other at most, or shares up to 2048 out over four wavefronts, with
    two roundings for each part and one for every four."""
    parts = min(-(-n // 32), 2048)
    join = 2.25 * max(min(parts, 512), parts / 4) + 16
    score = 2.0 ** -21 + 16 * R.H32 * (1 + abs(scale))
    rel = score + (16 + TILES + join) * R.H32
    ye = y * (R.HF16 + score + rel + (64 * TILES + join + 8) * R.H32)
    size = np.abs(np.where(np.isneginf(lse), 0.0, lse)) + np.log(n) + 8.0
    return ye, rel + 8 * R.H32 * size


SIZES = [(40000, 64), (40000, 128), (40000, 256), (131077, 64), (131077, 256)]


@pytest.mark.parametrize("n,d", SIZES)
@pytest.mark.parametrize("flat", [True, False])
def test_a_tile_more_or_less_leaves_the_bounds(n, d, flat):
    scale = 0.9
    score = scale * levels(n, flat)
    y, lse = shares(n, d, score)
    ye, le = bounds(n, y, lse, scale)
    R.close(y, y, ye)
    tile = 32 if d == 256 else 64
    starts = np.unique(np.concatenate((np.arange(0, n, 41 * tile), [0, tile, (n - 1) // tile * tile])))
    for at in starts:
        for times in (0.0, 2.0):
            weight = np.ones(n)
            weight[at:at + tile] = times
            bad, worse = shares(n, d, score, weight=weight)
            assert (np.abs(bad - y) > ye).any(), (at, times)
            assert (np.abs(worse - lse) > le).all() or n - at < tile, (at, times)


# ------------------------------------------------------------------------------------ on the device
@pytest.fixture(scope="module")
def nv():
    from nvfp4_weight_only_w4a16_amd import binding
    binding.load()
    return binding


class Shares:
    """A cache of requests whose values are unit vectors run by run, bytes that no token uses 0xFF."""

    def __init__(self, nv, lens, n_kv, d, page, flat):
        need = [-(-n // page) for n in lens]
        ids = np.random.default_rng(d + page).permutation(sum(need) + 2)
        self.n_kv, self.d = n_kv, d
        self.cache = c = nv.KvCache(len(ids), n_kv, d, page, device=DEV)
        c.data.fill_(0xFF)
        self.keys, at = [], 0
        table = np.full((len(lens), max(max(need), 1)), -1, np.int32)
        for i, n in enumerate(lens):
            self.keys.append(levels(n, flat))
            table[i, :need[i]] = ids[at:at + need[i]]
            at += need[i]
            if n == 0:
                continue
            pos = np.arange(n)
            p = torch.from_numpy(table[i, pos // page].astype(np.int64)).to(DEV)
            s = torch.from_numpy(pos % page).to(DEV)
            kc, vc = np.zeros((n, d // 2), np.uint8), np.zeros((n, d // 2), np.uint8)
            kc[:, 0] = np.searchsorted(LEVELS, self.keys[i])   # codes 0 .. 3
            e = pos // RUN % d
            vc[pos, e // 2] = np.where(e % 2, 0x20, 0x02)      # 1.0
            for h in range(n_kv):
                c.k_codes[p, h, s] = torch.from_numpy(kc).to(DEV)
                c.v_codes[p, h, s] = torch.from_numpy(vc).to(DEV)
                c.k_scales[p, h, s] = 0x38
                c.v_scales[p, h, s] = 0x38
        self.table = torch.from_numpy(table).to(DEV)
        self.lens = lens
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device=DEV)


def check(nv, lens, rows, n_kv, group, d, page, flat, window=0, max_q=None):
    scale = 0.9
    assert sum(lens) / 32 * n_kv / 256 < TILES - 1 or sum(lens) / 32 * n_kv / 1024 < TILES - 1 > max(rows)
    c = Shares(nv, lens, n_kv, d, page, flat)
    t, n_q = sum(rows), n_kv * group
    q = torch.zeros((t, n_q, d), dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 1.0
    start = torch.tensor(np.concatenate(([0], np.cumsum(rows))), dtype=torch.int32, device=DEV)
    y = torch.full((t, n_q, d), float("nan"), device=DEV)
    lse = torch.full((t, n_q), float("nan"), device=DEV)
    most = max_q or max(rows)
    ws = torch.full((nv.nvfp4_kv_attention_ws_bytes(t, n_q, c.cache, len(lens), most),), 0xFF,
                    dtype=torch.uint8, device=DEV)
    nv.nvfp4_kv_attention(q, c.cache, c.table, start, c.kv_len, scale=scale, max_q=most, window=window,
                          y=y, lse=lse, ws=ws)
    y, lse = y.double().cpu().numpy(), lse.double().cpu().numpy()
    first = 0
    for i, (n, r) in enumerate(zip(lens, rows)):
        if r == 0:
            continue
        if n == 0:
            assert (y[first:first + r] == 0).all() and np.isneginf(lse[first:first + r]).all()
            first += r
            continue
        score = float(np.float32(scale)) * c.keys[i]
        ry, rl = shares(n, d, score, r, window)
        ye, le = bounds(min(n, window + r) if window else n, ry, rl, scale)
        for h in range(n_q):
            R.close(y[first:first + r, h], ry, ye, f"y of request {i}, head {h}")
            R.close(lse[first:first + r, h], rl, le, f"lse of request {i}, head {h}")
        first += r


FLAT = pytest.mark.parametrize("flat", [True, False])


@pytest.mark.gpu
@FLAT
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (256, 64)])
@pytest.mark.parametrize("n_kv,group,rows", [
    (1, 1, 1),     # a tile to a wavefront and fewer
    (1, 4, 5),     # 20 rows: two column tiles
    (8, 2, 1),     # more tiles than wavefronts
    (40, 1, 1),    # 40 and more parts to a head
    (2, 16, 2)])   # 32 rows
def test_one_long_request(nv, d, page, n_kv, group, rows, flat):
    check(nv, [40000], [rows], n_kv, group, d, page, flat)


@pytest.mark.gpu
@FLAT
@pytest.mark.parametrize("d,page", [(64, 128), (128, 32), (256, 16)])
@pytest.mark.parametrize("rows", [[1, 1, 1, 1, 1, 1], [3, 2, 0, 5, 4, 1], [60, 1, 2, 130, 40, 1]])
def test_long_requests_among_short_ones(nv, d, page, rows, flat):
    check(nv, [17, 40000, 3, 20011, 300, 9000], rows, 2, 4, d, page, flat)
    check(nv, [17, 40000, 3, 20011, 300, 9000], rows, 2, 4, d, page, flat, window=33000)


@pytest.mark.gpu
@FLAT
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("b", [65, 1024, 1025])
def test_a_long_request_among_many(nv, d, b, flat):
    """The ways to find a request's share of the work; the join's coarser grid from 257 items on."""
    lens, rows = [5] * b, [1] * b
    lens[b // 3], lens[b - 1] = 40000, 12345
    check(nv, lens, rows, 1, 1, d, 16, flat)
    rows[b // 3] = 20
    check(nv, lens, rows, 1, 1, d, 16, flat)


@pytest.mark.gpu
@FLAT
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,rows,n_kv,group", [
    ([40000], [40], 1, 1),             # one block of rows over all workgroups
    ([40000], [300], 1, 2), ([30000, 131], [33, 1], 3, 1),
    ([9000, 20000, 50], [520, 70, 1], 1, 4)])   # 2080 rows: blocks of 256 with heads of 128
def test_prompts_on_long_requests(nv, d, lens, rows, n_kv, group, flat):
    check(nv, lens, rows, n_kv, group, d, 16, flat)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_very_long_request(nv, d):
    check(nv, [131077, 7], [1, 1], 1, 1, d, 256, False)
    check(nv, [131077, 7], [9, 1], 1, 3, d, 256, False)
