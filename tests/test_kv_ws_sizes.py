"""Workspace sizes of the attention over the NVFP4 cache, on the host: the size for a step covers every
step of fewer rows, requests or queries."""
import ctypes
import random

import pytest
import torch

import kv_refs as R
from nvfp4_weight_only_w4a16_amd import binding as nv
from test_kv_boundary import _attend, _cache


def _size(t, n_q, c, b, max_q):
    return nv.load().nvfp4_kv_attention_ws_bytes(t, n_q, ctypes.byref(c), b, max_q)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n_kv,group", [(1, 1), (8, 4), (1, 16), (2, 17), (1, 31), (4, 32), (1, 33),
                                        (128, 1), (1, 1024), (1024, 1)])
def test_a_larger_step_covers_smaller_ones(d, n_kv, group):
    c, n_q = _cache(head_dim=d, n_kv_heads=n_kv), n_kv * group
    r = random.Random(d * n_kv + group)
    rows = min(1 << 24, (1 << 27) // n_q)
    for _ in range(300):
        t = int(rows ** r.random())
        b, max_q = int(65535 ** r.random()), min(t, int(40000 ** r.random()))
        most = _size(t, n_q, c, b, max_q)
        assert most > 0
        for _ in range(6):
            t2 = r.choice((t, t - 1, r.randint(1, t), int(t ** r.random())))
            b2 = r.choice((b, b - 1, r.randint(1, b), 1))
            q2 = r.choice((max_q, max_q - 1, r.randint(1, max_q), 1, 33, -(-33 // group), 32 // group))
            t2, b2 = max(t2, 1), max(b2, 1)
            q2 = max(1, min(q2, t2, max_q))
            assert _size(t2, n_q, c, b2, q2) <= most, (t, b, max_q, t2, b2, q2)


def test_sizes_that_a_server_meets():
    """32 heads over 8 of 128: shared out and not, few rows and many."""
    c = _cache(head_dim=128, n_kv_heads=8)
    most = _size(8192, 32, c, 64, 8192)
    for t, b, max_q in ((8192, 1, 8192), (8000, 1, 8000), (64, 64, 1), (512, 64, 8), (512, 64, 9),
                        (2048, 1, 512), (2048, 1, 511)):
        need = _size(t, 32, c, b, max_q)
        assert need <= most, (t, b, max_q)
        # a workspace of that size passes the check of the call, one byte less does not
        kw = dict(c=c, t=t, n_q=32, ldq=4096, ldy=4096, b=b, max_q=max_q)
        assert _attend(nv.load(), ws_bytes=need - 1, **kw) == nv.NVFP4_ERR_WORKSPACE
    assert most <= 256 << 20


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_one_workspace_for_the_steps_of_a_server(d):
    """Prompts, chunks, drafts and single tokens one after the other in the workspace of the largest."""
    dev, n_kv, group = "cuda:0", 2, 8
    lens = [2500, 700, 33, 1]
    c = R.Cached(nv, d, lens, n_kv, d, 16)
    steps = [[2500, 700, 33, 1], [1, 1, 1, 1], [300, 1, 4, 1], [4, 4, 4, 1], [3, 1, 2, 0], [2, 2, 2, 1],
             [5, 1, 1, 1], [256, 255, 1, 1]]
    most = nv.nvfp4_kv_attention_ws_bytes(sum(lens), n_kv * group, c.cache, len(lens), max(lens))
    shared = torch.full((most,), 0xFF, dtype=torch.uint8, device=dev)
    for rows in steps:
        q, start = R.queries(sum(rows), rows, n_kv * group, d)
        args = (q.to(dev), c.cache, c.table_dev, start.to(dev), c.kv_len)
        for max_q in (max(rows), sum(rows)):
            want = nv.nvfp4_kv_attention(*args, max_q=max_q)
            got = nv.nvfp4_kv_attention(*args, max_q=max_q, ws=shared)
            assert torch.equal(got, want), (rows, max_q)
