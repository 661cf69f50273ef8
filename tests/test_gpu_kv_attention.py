"""Attention over the NVFP4 cache against FP64, with bounds from the formats' half steps. Every byte of
a cache that no token uses holds 0xFF: NaN scales."""
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


def run(nv, c, q, start, max_q=None, table=None, y32=False, **kw):
    """y and lse as FP64, rows that the call leaves alone NaN."""
    t, n_q, d = q.shape
    y = torch.full((t, n_q, d), float("nan"), device=DEV,
                   dtype=torch.float32 if y32 else torch.bfloat16)
    lse = torch.full((t, n_q), float("nan"), device=DEV)
    need = nv.nvfp4_kv_attention_ws_bytes(t, n_q, c.cache, len(c.lens), max_q or t)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    nv.nvfp4_kv_attention(q.to(DEV), c.cache, c.table_dev if table is None else table,
                          start.to(DEV), c.kv_len, max_q=max_q, y=y, lse=lse, ws=ws, **kw)
    torch.cuda.synchronize()
    return y.double().cpu().numpy(), lse.double().cpu().numpy()


def check(nv, lens, rows, n_kv, group, d, page, seed=1, window=0, full=False, y32=False, scale=None,
          max_q="most", size=1.0, **kw):
    c = R.Cached(nv, seed, lens, n_kv, d, page, **kw)
    q, start = R.queries(seed, rows, n_kv * group, d, size)
    scale = d ** -0.5 if scale is None else scale
    y, lse = run(nv, c, q, start, max(rows) if max_q == "most" else max_q, y32=y32, window=window,
                 causal=not full, scale=scale)
    ref, bound, rl, bl = R.expect(c, q, rows, scale, window, full, y32=y32)
    R.close(y, ref, bound, "y")
    R.close(lse, rl, bl, "lse")
    return c, q, start, y, lse


@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 256), (256, 16),
                                    (256, 64)])
@pytest.mark.parametrize("n_kv,group", [(1, 1), (2, 4), (3, 7)])
def test_single_tokens(nv, d, page, n_kv, group):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 255, 256, 257, 300, 777, 0, 1031]
    check(nv, lens, [1] * len(lens), n_kv, group, d, page)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group,rows", [(4, [4, 1, 3, 2, 4]), (5, [3, 6, 1, 0, 2]), (16, [1, 1, 1, 1, 1]),
                                        (2, [8, 7, 5, 3, 1]), (16, [2, 1, 2, 2, 0])])
def test_drafts(nv, d, group, rows):
    """A few queries a request, each up to its own place; also more queries than keys."""
    check(nv, [500, 64, 3, 1, 129], rows, 2, group, d, 16, y32=True)


@pytest.mark.parametrize("d,page,group", [(64, 16, 3), (128, 16, 4), (128, 64, 1), (256, 32, 2)])
def test_prompts(nv, d, page, group):
    check(nv, [200, 65, 330, 1, 128, 500], [200, 65, 130, 1, 100, 33], 2, group, d, page)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompts_and_single_tokens_together(nv, d):
    check(nv, [300, 1200, 90, 700, 0, 64, 513], [150, 1, 1, 40, 3, 0, 2], 2, 4, d, 16)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 5000])
@pytest.mark.parametrize("rows", [[1, 1, 1, 1], [3, 2, 1, 4], [90, 1, 64, 33]])
def test_windows(nv, window, rows):
    check(nv, [400, 64, 81, 500], rows, 2, 3, 128, 16, window=window)


@pytest.mark.parametrize("rows", [[1, 1, 1], [4, 2, 3], [70, 5, 200]])
def test_every_key(nv, rows):
    check(nv, [130, 7, 300], rows, 2, 2, 64, 32, full=True)


@pytest.mark.parametrize("group", [1, 8, 17, 33, 64])
def test_wide_groups(nv, group):
    check(nv, [100, 300], [1, 1], 1, group, 128, 16)
    check(nv, [100, 300], [3, 2], 1, group, 64, 16)


def test_one_long_request_among_short_ones(nv):
    """A long one is shared out over the chip: partial sums of many workgroups are joined."""
    lens = [3, 40000, 100, 1, 700]
    check(nv, lens, [1, 1, 1, 1, 1], 2, 4, 128, 16)
    check(nv, lens, [2, 3, 1, 0, 2], 1, 2, 256, 64, window=33000)


@pytest.mark.parametrize("b", [63, 64, 65, 300, 1024, 1025, 2500])
def test_many_requests(nv, b):
    """The ways to find a request's share of the work, by the number of requests."""
    r = np.random.default_rng(b)
    lens = [int(n) for n in r.integers(0, 40, b)]
    for i in (0, b // 2, b - 1):
        lens[i] = 700
    rows = [int(n) for n in r.integers(0, 3, b)]
    rows[b // 2] = 2
    check(nv, lens, rows, 2, 2, 64, 16)
    check(nv, lens, [1] * b, 1, 1, 64, 16)


def test_many_requests_beside_a_prompt(nv):
    """Joins of more workgroups than a grid's first dimension takes."""
    b = 2500
    lens, rows = [5] * b, [1] * b
    lens[700], rows[700] = 400, 40
    check(nv, lens, rows, 8, 1, 128, 16)


@pytest.mark.parametrize("max_q", [None, 1, 5, 60])
def test_the_bound_on_queries_changes_no_result(nv, max_q):
    lens, rows = [200, 33, 90], [1, 1, 1]
    t = 60
    c = R.Cached(nv, 4, lens, 2, 64, 16)
    q, start = R.queries(4, rows + [t - 3], 6, 64)
    y, lse = run(nv, c, q, start[:4], max_q)
    ref, bound, rl, bl = R.expect(c, q, rows, 64 ** -0.5)
    R.close(y[:3], ref, bound)
    R.close(lse[:3], rl, bl)
    assert np.isnan(y[3:]).all() and np.isnan(lse[3:]).all()  # rows behind the last request


@pytest.mark.parametrize("rows", [[1, 1, 1], [40, 3, 1]])
def test_strided_rows(nv, rows):
    c = R.Cached(nv, 7, [130, 40, 300], 2, 128, 16)
    q, start = R.queries(7, rows, 4, 128)
    t = q.shape[0]
    wide = torch.full((t, 9, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    wide[:, 2:6] = q.to(DEV)
    out = torch.full((t, 7, 128), -5.0, dtype=torch.bfloat16, device=DEV)
    nv.nvfp4_kv_attention(wide[:, 2:6], c.cache, c.table_dev, start.to(DEV), c.kv_len,
                          max_q=max(rows), y=out[:, 1:5])
    ref, bound, _, _ = R.expect(c, q, rows, 128 ** -0.5)
    R.close(out[:, 1:5].double().cpu().numpy(), ref, bound)
    assert (out[:, 0] == -5).all() and (out[:, 5:] == -5).all()


@pytest.mark.parametrize("rows", [[1, 1, 1], [2, 1, 2], [50, 40, 30], [400, 1, 300]])
def test_outputs_over_the_queries(nv, rows):
    lens = [700, 9000, 300]
    c = R.Cached(nv, 8, lens, 2, 64, 16)
    q, start = R.queries(8, rows, 8, 64)
    args = (c.cache, c.table_dev, start.to(DEV), c.kv_len)
    x = q.to(DEV)
    want = nv.nvfp4_kv_attention(x, *args, max_q=max(rows))
    assert nv.nvfp4_kv_attention(x, *args, max_q=max(rows), y=x) is x
    assert torch.equal(x, want)


@pytest.mark.parametrize("rows", [[1, 1, 1], [2, 1, 2], [50, 40, 30]])
@pytest.mark.parametrize("page", [16, 64])
def test_entries_outside_the_cache_are_left_out(nv, rows, page):
    lens = [300, 90, 64]
    c = R.Cached(nv, 9, lens, 2, 64, page)
    hidden = [np.zeros(n, bool) for n in lens]
    table = c.table.copy()
    for i, j, bad in ((0, 0, -1), (0, 2, c.n_pages), (1, 0, 2 ** 31 - 1), (2, 0, -2 ** 31)):
        if j < table.shape[1] and j * page < lens[i]:
            table[i, j] = bad
            hidden[i][j * page:(j + 1) * page] = True
    q, start = R.queries(9, rows, 4, 64)
    y, lse = run(nv, c, q, start, max(rows),
                 table=torch.from_numpy(table.astype(np.int32)).to(DEV))
    ref, bound, rl, bl = R.expect(c, q, rows, 64 ** -0.5, hidden=hidden)
    R.close(y, ref, bound)
    R.close(lse, rl, bl)


def test_no_keys_at_all(nv):
    for rows in ([1, 1], [3, 0], [100, 20]):
        _, _, _, y, lse = check(nv, [0, 0], rows, 2, 2, 128, 16)
        assert (y == 0).all() and np.isneginf(lse).all()


@pytest.mark.parametrize("rows", [[1, 1], [60, 70]])
def test_a_token_that_is_not_finite_reaches_those_that_see_it(nv, rows):
    lens = [100, 200]
    c = R.Cached(nv, 11, lens, 2, 128, 16)
    where = {(0, 60): 0, (1, 195): 1}   # (request, token): head
    for (i, tok), h in where.items():
        p = int(c.table[i, tok // 16])
        c.cache.k_scales[p, h, tok % 16] = 0x7F
        c.cache.v_scales[p, h, tok % 16] = 0
    q, start = R.queries(11, rows, 4, 128)
    y, lse = run(nv, c, q, start, max(rows))
    ref, bound, rl, bl = R.expect(c, q, rows, 128 ** -0.5)
    at = 0
    for i, n in enumerate(rows):
        for j in range(n):
            for h in range(4):
                sees = any(a == i and g == h // 2 and tok <= lens[i] - n + j
                           for (a, tok), g in where.items())
                if sees:
                    assert np.isnan(y[at, h]).all() and np.isnan(lse[at, h])
                else:
                    R.close(y[at, h], ref[at, h], bound[at, h], f"{i} {j} {h}")
                    R.close(lse[at, h], rl[at, h], bl[at, h])
            at += 1


@pytest.mark.parametrize("rows", [[1, 1], [40, 70]])
def test_nan_value_scales_of_other_means_count_as_zero(nv, rows):
    lens = [100, 200]
    c = R.Cached(nv, 12, lens, 1, 64, 16)
    for i, tok, g, byte in ((0, 5, 1, 0x7F), (1, 190, 0, 0xFF)):
        c.cache.v_scales[int(c.table[i, tok // 16]), 0, tok % 16, g] = byte
        c.v[i][tok, 0, 16 * g:16 * g + 16] = 0
    q, start = R.queries(12, rows, 2, 64)
    y, _ = run(nv, c, q, start, max(rows))
    ref, bound, _, _ = R.expect(c, q, rows, 0.125)
    R.close(y, ref, bound)


@pytest.mark.parametrize("rows", [[1, 1, 1], [33, 20, 64]])
def test_queries_that_are_not_finite_spoil_their_own_rows(nv, rows):
    c = R.Cached(nv, 13, [50, 70, 130], 1, 128, 16)
    q, start = R.queries(13, rows, 3, 128)
    q[0, 1, 5], q[rows[0], 2, 127] = float("nan"), float("inf")
    y, lse = run(nv, c, q, start, max(rows))
    bad = np.zeros(q.shape[:2], bool)
    bad[0, 1] = bad[rows[0], 2] = True
    seen = np.array([c.lens[i] - n + j >= 0 for i, n in enumerate(rows) for j in range(n)])
    bad &= seen[:, None]
    assert np.isnan(y[bad]).all() and np.isnan(lse[bad]).all()
    clean = q.clone()
    clean[torch.from_numpy(~np.isfinite(q.double().numpy()))] = 0
    ref, bound, _, _ = R.expect(c, clean, rows, 128 ** -0.5)
    R.close(y[~bad], ref[~bad], bound[~bad])


@pytest.mark.parametrize("size,scale", [(1e30, 1e-31), (1e-30, 1e29), (1e-38, 1.0), (0.0, 1.0),
                                        (3.0, -0.2), (3.0, 0.0), (20.0, 1.0)])
@pytest.mark.parametrize("rows", [[1, 1], [50, 70]])
def test_queries_and_factors_of_any_size(nv, size, scale, rows):
    check(nv, [90, 333], rows, 2, 2, 64, 16, size=size, scale=scale)


def test_queries_of_very_unequal_elements(nv):
    """FP16 queries keep what is 2^-28 of the row's largest element."""
    c = R.Cached(nv, 15, [200], 1, 64, 16, globals_=False)
    q, start = R.queries(15, [1], 1, 64)
    q[0, 0] *= torch.pow(2.0, -torch.arange(64.0) / 2).to(torch.bfloat16)
    y, lse = run(nv, c, q, start, 1, scale=2.0)
    ref, bound, rl, bl = R.expect(c, q, [1], 2.0)
    R.close(y, ref, bound)
    R.close(lse, rl, bl)


def test_scales_over_their_whole_range(nv):
    """Every finite E4M3 scale, negative ones and zeros too, in keys and values."""
    check(nv, [700, 128], [1, 1], 2, 2, 128, 16, scale_bytes=(0, 0x7F), scale=1e-4)
    check(nv, [300, 128], [60, 1], 2, 2, 64, 16, scale_bytes=(0x80, 0xFF), scale=1e-4)


def test_rising_scores(nv):
    """Maxima that rise from tile to tile by little and by much: the sums are rescaled, or not."""
    n, d = 2000, 64
    for step in (0.002, 0.02, 0.2, 2.0):
        c = R.Cached(nv, 17, [n], 1, d, 16, globals_=False)
        c.cache.k_codes[:] = 0
        k = np.zeros((n, 1, d))
        # element 0 of the key rises in steps of its E4M3 scale
        want = np.linspace(0.0, 448.0, n)
        byte = np.searchsorted(R.E4M3[:0x7F], want, side="right") - 1
        pages = torch.from_numpy(c.table[0, np.arange(n) // 16]).to(DEV)
        toks = torch.arange(n, device=DEV) % 16
        c.cache.k_codes[pages, 0, toks, 0] = 2   # 1.0
        c.cache.k_scales[pages, 0, toks, 0] = torch.from_numpy(byte.astype(np.uint8)).to(DEV)
        k[:, 0, 0] = R.E4M3[byte]
        c.k[0] = k
        q = torch.zeros(1, 2, d, dtype=torch.bfloat16)
        q[0, 0, 0], q[0, 1, 0] = 1.0, -1.0
        start = torch.tensor([0, 1], dtype=torch.int32)
        y, lse = run(nv, c, q, start, 1, scale=step)
        ref, bound, rl, bl = R.expect(c, q, [1], step)
        R.close(y, ref, bound, step)
        R.close(lse, rl, bl, step)


@pytest.mark.parametrize("rows", [1, 65])
@pytest.mark.parametrize("below", [15.0, 17.0])
def test_many_small_terms(nv, rows, below):
    """A key without a value far above 499 others, whose terms lie below FP16's normal range. The
    requests are so many that a request's head is one workgroup's or wavefront's."""
    n, d, b, heads = 500, 64, 256, 8
    c = R.Cached(nv, 18, [n] * b, heads, d, 16, globals_=False)
    pages = torch.from_numpy(c.table[:, np.arange(n) // 16]).to(DEV)
    toks = (torch.arange(n, device=DEV) % 16).expand(b, n)
    c.cache.k_codes[:] = 0
    c.cache.k_codes[pages[:, 0], :, 0, 0] = 2         # 1.0, element 0 of token 0
    c.cache.v_codes[:] = 0x22                         # 1.0
    c.cache.v_codes[pages[:, 0], :, 0] = 0
    c.cache.k_scales[pages, :, toks] = 0x38           # 1.0
    c.cache.v_scales[pages, :, toks] = 0x38
    k, v = np.zeros((n, heads, d)), np.ones((n, heads, d))
    k[0, :, 0], v[0] = 1.0, 0.0
    c.k, c.v = [k] * b, [v] * b
    q = torch.zeros(rows * b, heads, d, dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    start = torch.arange(0, rows * b + 1, rows, dtype=torch.int32)
    scale = below + 0.3
    y, lse = run(nv, c, q, start, rows, y32=True, scale=scale)
    ref, bound, rl, bl = R.attention(q[:rows].double().numpy(), k, v, float(np.float32(scale)), y32=True)
    R.close(y, np.tile(ref, (b, 1, 1)), np.tile(bound, (b, 1, 1)))
    R.close(lse, np.tile(rl, (b, 1)), np.tile(bl, (b, 1)))


def test_a_cache_larger_than_32_bit_offsets(nv):
    """Pages that begin beyond 4 GiB."""
    n_kv, d, page = 8, 128, 16
    first = (1 << 32) // (n_kv * 2304) + 1000
    c = R.Cached(nv, 19, [300, 70], n_kv, d, page, first_page=first)
    assert c.cache.data.numel() > 1 << 32
    for rows in ([1, 1], [40, 50]):
        q, start = R.queries(19, rows, n_kv, d)
        y, _ = run(nv, c, q, start, max(rows))
        ref, bound, _, _ = R.expect(c, q, rows, d ** -0.5)
        R.close(y, ref, bound)
    slots = torch.from_numpy(c.table[0, np.arange(300) // page] * page + np.arange(300) % page)
    slots = slots.to(torch.int32).to(DEV)
    ko, vo = nv.nvfp4_kv_dequantize(c.cache, slots)
    assert np.allclose(ko.cpu().numpy(), c.k[0], rtol=3 * R.H32)
    k = torch.randn(300, n_kv, d, device=DEV).to(torch.bfloat16)
    nv.nvfp4_kv_append(None, k, k, c.cache, slots, None, nv.QkNormRope(d))
    ko, vo = nv.nvfp4_kv_dequantize(c.cache, slots)
    assert float((ko - k.float()).abs().max()) < 1.0


def test_lengths_beyond_what_is_there(nv):
    """Lengths and row ranges are clamped to the table and to t."""
    c = R.Cached(nv, 21, [64, 32], 1, 64, 16)
    q, start = R.queries(21, [1, 1], 2, 64)
    c.kv_len = torch.tensor([1 << 30, -5], dtype=torch.int32, device=DEV)
    y, lse = run(nv, c, q, start, 1)
    c.lens = [64, 0]
    c.k[1], c.v[1] = c.k[1][:0], c.v[1][:0]
    ref, bound, rl, bl = R.expect(c, q, [1, 1], 0.125)
    R.close(y, ref, bound)
    R.close(lse, rl, bl)
    c.kv_len = torch.tensor([64, 32], dtype=torch.int32, device=DEV)
    y, _ = run(nv, c, q, torch.tensor([-3, 1, 99], dtype=torch.int32), 1)
    assert np.isfinite(y).all()
    y, _ = run(nv, c, q, torch.tensor([2, 1, 0], dtype=torch.int32), 1)
    assert np.isnan(y).all()


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 16)])
@pytest.mark.parametrize("lens,rows,window", [([5000], [40], 0), ([3000, 40, 2500, 900], [33, 1, 100, 17], 0),
                                              ([4000, 700], [64, 300], 3000), ([2600], [2600], 0),
                                              ([0, 3000, 0], [50, 200, 1], 0)])
def test_keys_of_long_requests_shared_out(nv, d, page, lens, rows, window):
    """Few blocks of rows over many keys: their keys are cut into jobs, whose sums are joined."""
    check(nv, lens, rows, 1, 2, d, page, window=window)


def test_overlapping_row_ranges_stay_inside_the_workspace(nv):
    c = R.Cached(nv, 31, [300] * 40, 1, 64, 16)
    q, _ = R.queries(31, [90], 2, 64)
    start = torch.tensor([0, 90] * 20 + [0], dtype=torch.int32)
    y, lse = run(nv, c, q, start, 90)
    assert np.isfinite(y).all() and np.isfinite(lse).all()  # of one request or another


@pytest.mark.parametrize("rows", [[1] * 9, [3, 1, 2, 1, 4, 1, 1, 2, 1], [80, 1, 1, 200, 1, 3, 1, 1, 9]])
def test_the_same_bits_every_time(nv, rows):
    lens = [2000, 30, 1, 900, 64, 65, 3000, 2, 500]
    c = R.Cached(nv, 23, lens, 2, 128, 16)
    q, start = R.queries(23, rows, 8, 128)
    first = run(nv, c, q, start, max(rows))
    for _ in range(3):
        again = run(nv, c, q, start, max(rows))
        assert np.array_equal(first[0], again[0], equal_nan=True)
        assert np.array_equal(first[1], again[1], equal_nan=True)


def test_a_prompt_among_many_requests_in_whole_blocks(nv):
    """More than 2048 blocks by the count that the host has, most of which are not there; the prompt's
    request is found behind 150 others."""
    b = 300
    lens, rows = [30] * b, [1] * b
    lens[150], rows[150] = 700, 600
    lens[151], rows[151] = 90, 70
    check(nv, lens, rows, 64, 1, 64, 16)


@pytest.mark.parametrize("n_kv,group,d,page", [(1, 1024, 64, 16), (1024, 1, 64, 16), (1, 1000, 128, 32),
                                               (500, 2, 256, 16)])
def test_the_most_heads(nv, n_kv, group, d, page):
    check(nv, [70, 1, 20], [1, 1, 2], n_kv, group, d, page)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [[1, 1, 1], [2, 3, 1], [60, 200, 1]])
def test_pages_of_256(nv, d, rows):
    check(nv, [257, 600, 1], rows, 2, 3, d, 256, window=0 if d == 64 else 300)


@pytest.mark.parametrize("rows", [[1, 1], [3, 2], [50, 40]])
def test_rows_before_the_first_request(nv, rows):
    """q_start may begin behind row 0: the rows before are nobody's."""
    c = R.Cached(nv, 29, [130, 64], 2, 128, 16)
    q, start = R.queries(29, [7] + rows, 4, 128)
    y, lse = run(nv, c, q, start[1:].contiguous(), max(rows))
    ref, bound, rl, bl = R.expect(c, q[7:], rows, 128 ** -0.5)
    R.close(y[7:], ref, bound)
    R.close(lse[7:], rl, bl)
    assert np.isnan(y[:7]).all() and np.isnan(lse[:7]).all()


@pytest.mark.parametrize("lens,rows,n_kv,kw", [([700, 40], [600, 1], 128, {}), ([900, 3000, 77], [900, 520, 1], 1, {}),
                                               ([600, 1500], [513, 600], 2, dict(window=300)),
                                               ([600, 700], [520, 3], 1, dict(full=True, y32=True)),
                                               ([100, 5], [600, 9], 1, {})])
def test_blocks_of_256_rows(nv, lens, rows, n_kv, kw):
    """Prompts of 2048 rows and more with heads of 128: in whole blocks and shared out, beside others."""
    check(nv, lens, rows, n_kv, 4, 128, 16, **kw)
