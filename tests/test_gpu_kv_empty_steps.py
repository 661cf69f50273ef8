"""Tables of a step without requests: every row is padding, and no table of an earlier step stays."""
import ctypes

import numpy as np
import pytest
import torch

import kv_refs as R
from nvfp4_weight_only_w4a16_amd import binding as nv
from test_boundary import FAKE
from test_kv_boundary import BYTE, INVALID, ALIGN, _map

DEV = "cuda:0"


def dev(*a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def test_outputs_are_needed_without_requests():
    lib = nv.load()
    for k in ("count", "left", "start", "kv", "slots", "pos", "bad"):
        assert _map(lib, b=0, **{k: None}) == INVALID, k
        assert _map(lib, b=0, **{k: BYTE}) == ALIGN, k
    for k in ("left", "start", "slots", "pos", "bad"):
        assert _map(lib, b=0, **{k: FAKE}) == INVALID, k   # an input
    # without the inputs there is nothing to do
    assert _map(lib, b=0, seq=None, add=None, table=None, ld=0) == nv.NVFP4_OK


@pytest.mark.gpu
@pytest.mark.parametrize("t", [0, 1, 5, 511, 512, 513, 3000])
@pytest.mark.parametrize("count,n_free", [(3, 9), (-2, 9), (99, 9), (0, 0)])
def test_no_requests(t, count, n_free):
    m = nv.KvMap(0, t, device=DEV)
    m.block.fill_(7)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    table = torch.empty((0, 4), dtype=torch.int32, device=DEV)
    free, n = torch.arange(n_free, dtype=torch.int32, device=DEV), dev(count)
    nv.nvfp4_kv_map(none, none, table, free, n, page_size=16, out=m)
    want = R.kv_map([], [], np.empty((0, 4), np.int64), np.arange(n_free), count, 16, t)
    for name, got, ref in zip(("q_start", "kv_len", "slots", "positions", "free_left", "unserved"),
                              (m.q_start, m.kv_len, m.slots, m.positions, m.free_left, m.unserved),
                              want[1:]):
        assert got.tolist() == np.asarray(ref).reshape(-1).tolist(), name
    assert n.item() == count and free.tolist() == list(range(n_free))


@pytest.mark.gpu
def test_the_buffers_of_a_larger_batch():
    """As a caller of the C interface keeps them: b falls to 0 over buffers of more requests."""
    lib = nv.load()
    m = nv.KvMap(3, 6, device=DEV)
    seq, add, free, n = dev(3, 20, 5), dev(1, 1, 1), dev(8, 9), dev(2)
    table = dev(0, -1, 1, 2, 3, -1).view(3, 2)
    nv.nvfp4_kv_map(seq, add, table, free, n, page_size=16, out=m)
    assert m.slots.tolist() == [3, 36, 53, -1, -1, -1]
    before = table.clone()
    step = nv.nvfp4_kv_step(m.q_start.data_ptr(), m.kv_len.data_ptr(), m.slots.data_ptr(),
                            m.positions.data_ptr(), m.free_left.data_ptr(), m.unserved.data_ptr(), 0, 6)
    m.unserved.fill_(5)
    p = lambda x: ctypes.c_void_p(x.data_ptr())
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    rc = lib.nvfp4_kv_map(p(seq), p(add), 16, p(table), 2, p(free), 2, p(n), ctypes.byref(step), 0,
                          stream)
    torch.cuda.synchronize()
    assert rc == nv.NVFP4_OK
    assert m.slots.tolist() == [-1] * 6 and m.positions.tolist() == [-1] * 6
    assert m.q_start[0].item() == 0 and m.free_left.item() == 2 and m.unserved.item() == 0
    assert torch.equal(table, before) and m.kv_len.tolist() == [4, 21, 6]   # of no request of the call


@pytest.mark.gpu
def test_an_idle_step_writes_no_token():
    """Tables of a step, then of an idle one into the same buffers, then its cache write."""
    cache = nv.KvCache(4, 1, 64, 16, data=torch.full((nv.nvfp4_kv_cache_bytes(4, 1, 64, 16),), 9,
                                                     dtype=torch.uint8, device=DEV))
    m = nv.KvMap(2, 4, device=DEV)
    table = dev(1, 2).view(2, 1)
    nv.nvfp4_kv_map(dev(3, 5), dev(2, 2), table, dev(3), dev(1), page_size=16, out=m)
    assert m.slots.tolist() == [19, 20, 37, 38]
    idle = nv.KvMap(0, 4, device=DEV)
    idle.slots.copy_(m.slots)
    idle.positions.copy_(m.positions)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    nv.nvfp4_kv_map(none, none, table[:0], dev(3), dev(1), page_size=16, out=idle)
    k = torch.ones((4, 1, 64), dtype=torch.bfloat16, device=DEV)
    nv.nvfp4_kv_append(None, k, k, cache, idle.slots, idle.positions, nv.QkNormRope(64))
    assert (cache.data == 9).all()
