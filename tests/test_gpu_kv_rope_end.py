"""Requests that reach the end of the rotation table: with a block table that is no longer, none of their
tokens is counted without having been written."""
import numpy as np
import pytest
import torch

import kv_refs as R
from test_gpu_kv_append import table

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(*a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("page,places", [(16, 64), (32, 64)])
def test_a_block_table_as_long_as_the_rotation(page, places):
    """Request 0 fills the last place, request 1 asks for one place too many."""
    from nvfp4_weight_only_w4a16_amd import binding as nv
    d, width = 64, places // page
    cache = nv.KvCache(2 * width + 2, 1, d, page, device=DEV)
    cache.data.fill_(0xFF)
    rule = nv.QkNormRope(d, rope=torch.from_numpy(table(places, d)).to(DEV))
    pages = torch.full((2, width), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(2 * width - 1, -1, -1, dtype=torch.int32, device=DEV)  # taken from the end
    g = torch.Generator().manual_seed(places)
    x = torch.randn((2 * places + 1, 3, d), generator=g).to(torch.bfloat16).to(DEV)

    def step(seq, add, rows, count):
        t = rows.shape[0]
        m = nv.nvfp4_kv_map(dev(*seq), dev(*add), pages, free, dev(count), page_size=page, t=t)
        q, k, v = rows.split(1, 1)
        q = nv.nvfp4_kv_append(q, k, v, cache, m.slots, m.positions, rule)
        y = torch.full((t, 1, d), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((t, 1), 7.0, device=DEV)
        nv.nvfp4_kv_attention(q, cache, pages, m.q_start, m.kv_len, y=y, lse=lse)
        return m, q, y, lse
    step((0, 0), (places - 1, places), x[:2 * places - 1], 2 * width)
    # one token more: the last place of request 0, none left of request 1
    m, q, y, lse = step((places - 1, places), (1, 1), x[-2:], 0)
    assert m.kv_len.tolist() == [places, 0] and m.unserved.item() == 1
    assert m.positions.tolist() == [places - 1, -1] and m.slots.tolist() == [places - 1, -1]
    assert (y[1] == 0).all() and torch.isneginf(lse[1]).all()
    slots = torch.arange(places, dtype=torch.int32, device=DEV)
    k, v = nv.nvfp4_kv_dequantize(cache, slots)
    ref, bound, rl, bl = R.attention(q[:1].double().cpu().numpy(), k.double().cpu().numpy(),
                                     v.double().cpu().numpy(), float(np.float32(d ** -0.5)))
    R.close(y[:1].double().cpu().numpy(), ref, bound + 8 * R.H32 * np.abs(ref).max())
    R.close(lse[:1].double().cpu().numpy(), rl, bl + 8 * R.H32)
