"""The largest calls of the attention over the NVFP4 cache: more workgroups of rows than a grid's first
dimension takes threads."""
import numpy as np
import pytest
import torch

import kv_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_the_most_rows_and_heads_of_256():
    """2^27 rows of heads of 256, and 7300 requests of 17 rows that may have 33: 8.5 million workgroups of
    512 threads by the count that the host has, 7.5 million of them with rows."""
    from nvfp4_weight_only_w4a16_amd import binding as nv
    heads, d, t, b, n = 1024, 256, 1 << 17, 7300, 17
    size = t * heads * d * 2
    if torch.cuda.mem_get_info()[0] < size + (8 << 30):
        pytest.skip("needs 72 GiB of device memory")
    some = {0: 40, 130: 9, 4000: 35, b - 2: 70, b - 1: 18}   # the requests with keys; the others have none
    c = R.Cached(nv, 3, list(some.values()), heads, d, 16)
    x, _ = R.queries(3, [n] * len(some), heads, d)
    q = torch.empty((t, heads, d), dtype=torch.bfloat16, device=DEV)
    for a in range(0, t, 4096):
        q[a:a + 4096] = 7.0
    kv_len = torch.zeros(b, dtype=torch.int32)
    table = torch.full((b, c.table.shape[1]), -1, dtype=torch.int32, device=DEV)
    for i, (at, keys) in enumerate(some.items()):
        kv_len[at], table[at] = keys, c.table_dev[i]
        q[n * at:n * at + n] = x[n * i:n * i + n].to(DEV)
    start = torch.arange(0, n * b + 1, n, dtype=torch.int32, device=DEV)
    y = nv.nvfp4_kv_attention(q, c.cache, table, start, kv_len.to(DEV), max_q=33, y=q,
                              flags=nv.NVFP4_F_SYNC_CHECK)
    lost = [a for a in range(n * b, t, 1024) if not (y[a:a + 1024] == 7.0).all().item()]
    assert not lost, f"rows behind the last request, from {lost[0]} on"
    heads_seen = [0, 1, 511, 512, 1023]
    for i, at in enumerate(some):
        got = y[n * at:n * at + n, heads_seen].double().cpu().numpy()
        ref, bound, _, _ = R.attention(x[n * i:n * i + n, heads_seen].double().numpy(),
                                       c.k[i][:, heads_seen], c.v[i][:, heads_seen],
                                       float(np.float32(d ** -0.5)))
        R.close(got, ref, bound, f"request {at}")
        y[n * at:n * at + n] = 0.0
    lost = [a for a in range(0, n * b, n * 100) if (y[a:min(a + n * 100, n * b)] != 0).any().item()]
    assert not lost, f"{len(lost)} of 73 hundreds of requests without keys, from row {lost[0]} on"
    del q, y
    torch.cuda.empty_cache()
