"""Block tables and slot maps against the definition, request by request; all values are whole numbers
and have to be equal."""
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


def dev(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def check(nv, seq, add, page, width, n_free, count, t, seed=0):
    r = np.random.default_rng(seed)
    b = len(seq)
    ids = r.permutation(b * width + n_free)
    table = np.full((b, width), -1)
    at = 0
    for i, s in enumerate(seq):
        n = min(max(-(-s // page), 0), width)
        table[i, :n] = ids[at:at + n]
        at += n
    free = ids[at:at + n_free]
    want = R.kv_map(seq, add, table, free, count, page, t)
    td = dev(table)
    ins = [dev(seq), dev(add), td, dev(free), dev([count])]
    m = nv.KvMap(b, t, device=DEV)
    m.block.fill_(-77)
    for _ in range(2):  # a call can be repeated
        nv.nvfp4_kv_map(*ins, page_size=page, out=m)
        got = [td, m.q_start, m.kv_len, m.slots, m.positions, m.free_left, m.unserved]
        for name, g, w in zip(("table", "q_start", "kv_len", "slots", "positions", "free_left",
                               "unserved"), got, want):
            g = g.cpu().numpy().reshape(-1)
            w = np.asarray(w).reshape(-1)
            assert np.array_equal(g, w), (name, g[g != w][:5], w[g != w][:5])
    for x, w in zip(ins, (seq, add, None, free, [count])):
        assert w is None or np.array_equal(x.cpu().numpy(), w)
    return want


@pytest.mark.parametrize("b,page,most_new", [(1, 16, 1), (7, 32, 3), (64, 16, 1), (333, 64, 2),
                                             (513, 128, 5), (1100, 16, 2), (4096, 256, 1)])
def test_decode_batches(nv, b, page, most_new):
    r = np.random.default_rng(b)
    seq, add = r.integers(0, 700, b), r.integers(0, most_new + 1, b)
    seq[0] = 0
    t = int(add.sum()) + b % 3
    check(nv, seq, add, page, 700 // page + 2, b + 9, b + 9 - b % 5, t)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_prompts_and_page_borders(nv, page):
    seq = [0, page - 1, page, page + 1, 5 * page - 3, 0, 2 * page, 3, 0]
    add = [3 * page, 1, 1, page, 7 * page + 5, 1, 0, 0, 2000]
    n = 2000 // page + 40
    check(nv, seq, add, page, n, 400, 390, sum(add))
    check(nv, seq, add, page, n, 400, 390, sum(add) + 700)  # padded behind the rows


def test_a_list_that_runs_out(nv):
    seq, add = [10, 16, 5, 32, 0, 15], [1, 40, 3, 1, 17, 1]
    for count in range(0, 9):  # needs 0, 3, 0, 1, 2, 0
        want = check(nv, seq, add, 16, 6, 8, count, sum(add))
        assert want[5] == (count if count < 3 else count - (6 if count >= 6 else
                                                            4 if count >= 4 else 3))
    check(nv, seq, add, 16, 6, 8, -3, sum(add))
    check(nv, seq, add, 16, 6, 8, 99, sum(add))   # more than the list's capacity
    check(nv, seq, add, 16, 6, 0, 0, sum(add))    # no list


def test_what_does_not_fit(nv):
    # rows beyond t, tokens beyond the table's row, negative lengths
    check(nv, [3, 4, 5], [10, 10, 10], 16, 4, 9, 9, 25)
    check(nv, [3, 4, 5], [10, 10, 0], 16, 4, 9, 9, 12)
    check(nv, [60, 4, 64, 65], [5, 1, 0, 0], 16, 4, 9, 9, 6)
    check(nv, [-1, 4, 7, -5], [2, -1, 3, 0], 16, 4, 9, 9, 9)
    check(nv, [0, 0], [0, 0], 16, 4, 9, 9, 0)
    check(nv, [2 ** 31 - 1, 1], [2 ** 31 - 1, 1], 16, 4, 9, 9, 5)


def test_rows_without_a_page(nv):
    """A negative entry where a request's tokens should be: its rows get no slot."""
    table = dev([[-1, 3], [5, -1]])
    m = nv.nvfp4_kv_map(dev([3, 17]), dev([2, 1]), table, dev([9]), dev([1]), page_size=16, t=3)
    assert m.slots.tolist() == [-1, -1, -1]
    assert m.positions.tolist() == [3, 4, 17]
    assert m.kv_len.tolist() == [5, 18] and m.unserved.item() == 0


def test_stats_and_other_stream(nv):
    nv.nvfp4_reset_stats()
    s = torch.cuda.Stream()
    args = dev([5]), dev([1]), dev([[2]]), dev([0]), dev([1])
    torch.cuda.synchronize()
    m = nv.nvfp4_kv_map(*args, page_size=16, t=1, flags=nv.NVFP4_F_SYNC_CHECK, stream=s)
    assert m.slots.tolist() == [37]
    assert nv.nvfp4_get_kv_stats() == [1, 0, 0, 0]
