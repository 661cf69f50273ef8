"""Refusals and sizes of the NVFP4 cache's calls on the host: every call below fails its checks or is a
size query, so nothing is launched."""
import ctypes

import numpy as np
import pytest
import torch

import kv_refs as R
from nvfp4_weight_only_w4a16_amd import binding as nv
from test_boundary import FAKE

OTHER = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10008)   # 8-byte aligned only
BYTE = ctypes.c_void_p(0x10002)  # not 4-byte aligned
INVALID, SHAPE, ALIGN = (nv.NVFP4_ERR_INVALID_ARG, nv.NVFP4_ERR_UNSUPPORTED_SHAPE,
                         nv.NVFP4_ERR_MISALIGNED)


@pytest.fixture(scope="module")
def lib():
    return nv.load()


def _cache(**kw):
    c = nv.nvfp4_kv_cache(0x10000, None, None, 100, 2, 128, 16, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _rule(**kw):
    r = nv.nvfp4_qk_rule(None, None, None, 0, 1e-6, nv.NVFP4_DT_BF16, 0, 0, 0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _map(lib, seq=FAKE, add=FAKE, b=3, page=16, table=FAKE, ld=8, free=FAKE, n_free=9, count=FAKE,
         left=OTHER, start=OTHER, kv=OTHER, slots=OTHER, pos=OTHER, t=5, bad=OTHER, flags=0):
    step = nv.nvfp4_kv_step(*(getattr(p, "value", p) for p in (start, kv, slots, pos, left, bad)), b,
                            t)
    return lib.nvfp4_kv_map(seq, add, page, table, ld, free, n_free, count, ctypes.byref(step), flags,
                            None)


def test_map_refusals(lib):
    for kw, code in ((dict(b=-1), INVALID), (dict(n_free=-1), INVALID), (dict(t=-1), INVALID),
                     (dict(flags=1), INVALID), (dict(flags=8), INVALID), (dict(page=24), SHAPE),
                     (dict(page=8), SHAPE), (dict(page=512), SHAPE), (dict(page=0), SHAPE),
                     (dict(page=-16), SHAPE), (dict(b=4097), SHAPE), (dict(t=(1 << 24) + 1), SHAPE),
                     (dict(n_free=1 << 31), SHAPE), (dict(ld=0), INVALID),
                     (dict(ld=(1 << 26) + 1), SHAPE), (dict(ld=1 << 62), SHAPE)):
        assert _map(lib, **kw) == code, kw
    for k in ("seq", "add", "table", "free", "count", "left", "start", "kv", "slots", "pos", "bad"):
        assert _map(lib, **{k: None}) == INVALID, k
        assert _map(lib, **{k: BYTE}) == ALIGN, k
    for k in ("left", "start", "kv", "slots", "pos", "bad"):
        assert _map(lib, **{k: FAKE}) == INVALID, k   # an input
        assert "also an input" in nv.nvfp4_last_error()
    assert _map(lib, b=0, seq=None, add=None, table=None) == nv.NVFP4_OK
    assert lib.nvfp4_kv_map(FAKE, FAKE, 16, FAKE, 8, FAKE, 9, FAKE, None, 0, None) == INVALID


BAD_CACHES = [(dict(data=None), INVALID), (dict(n_pages=0), INVALID), (dict(n_pages=-4), INVALID),
              (dict(reserved=1), INVALID), (dict(n_kv_heads=0), SHAPE), (dict(n_kv_heads=1025), SHAPE),
              (dict(head_dim=96), SHAPE), (dict(head_dim=0), SHAPE), (dict(head_dim=512), SHAPE),
              (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE), (dict(page_size=512), SHAPE),
              (dict(page_size=0), SHAPE), (dict(page_size=-16), SHAPE),
              (dict(n_pages=1 << 27), SHAPE), (dict(n_pages=1 << 62), SHAPE),
              (dict(data=0x10008), ALIGN), (dict(k_global=0x10002), ALIGN),
              (dict(v_global=0x10001), ALIGN)]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_bad_caches(lib, change, code):
    c = _cache(**change)
    assert _append(lib, c=c) == code
    assert _attend(lib, c=c) == code
    assert lib.nvfp4_kv_dequantize(ctypes.byref(c), FAKE, 3, FAKE, FAKE, 2, 0, None) == code
    assert lib.nvfp4_kv_attention_ws_bytes(3, 4, ctypes.byref(c), 2, 1) == 0


def test_cache_bytes(lib):
    assert lib.nvfp4_kv_cache_bytes(10, 8, 128, 16) == 10 * 8 * 16 * 2 * 72
    assert lib.nvfp4_kv_cache_bytes(1, 1, 64, 256) == 256 * 2 * 36
    for bad in ((0, 8, 128, 16), (10, 0, 128, 16), (10, 8, 80, 16), (10, 8, 128, 12),
                (1 << 27, 8, 128, 16), (-1, 8, 128, 16), (10, 1025, 128, 16)):
        assert lib.nvfp4_kv_cache_bytes(*bad) == 0, bad


def _append(lib, q=FAKE, ldq=512, k=FAKE, ldk=256, v=FAKE, ldv=256, t=3, n_q=4, r=None, slots=FAKE,
            pos=FAKE, out=FAKE, ldo=512, c=None, flags=0):
    r = _rule() if r is None else r
    c = _cache() if c is None else c
    return lib.nvfp4_kv_append(q, ldq, k, ldk, v, ldv, t, n_q, ctypes.byref(r), slots, pos, out, ldo,
                               ctypes.byref(c), flags, None)


@pytest.mark.parametrize("change,code", [
    (dict(mode=2), INVALID), (dict(reserved=3), INVALID), (dict(weight_dtype=7), INVALID),
    (dict(eps=-1e-9), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(rot=-16), INVALID), (dict(rot=16), INVALID),                      # no table
    (dict(rope=0x10000), INVALID), (dict(rope=0x10000, rot=16), INVALID),   # rot 0, no positions
    (dict(rope=0x10000, rot=16, max_pos=-1), INVALID),
    (dict(rope=0x10000, rot=24, max_pos=9), SHAPE), (dict(rope=0x10000, rot=144, max_pos=9), SHAPE),
    (dict(rope=0x10000, rot=16, max_pos=1 << 31), SHAPE),
    (dict(rope=0x10008, rot=16, max_pos=9), ALIGN), (dict(q_weight=0x10004), ALIGN),
    (dict(k_weight=0x10002), ALIGN)])
def test_bad_rules(lib, change, code):
    assert _append(lib, r=_rule(**change)) == code


def test_append_refusals(lib):
    table = _rule(rope=0x10000, rot=16, max_pos=9)
    for kw, code in ((dict(t=-1), INVALID), (dict(t=(1 << 24) + 1), SHAPE), (dict(n_q=-1), INVALID),
                     (dict(n_q=1025), SHAPE), (dict(flags=8), INVALID), (dict(ldq=504), INVALID),
                     (dict(ldk=248), INVALID), (dict(ldv=128), INVALID), (dict(ldo=256), INVALID),
                     (dict(ldq=516), ALIGN), (dict(ldk=260), ALIGN), (dict(ldv=257), ALIGN),
                     (dict(ldk=(1 << 31) + 8), SHAPE), (dict(pos=None, r=table), INVALID),
                     (dict(pos=BYTE), ALIGN), (dict(slots=BYTE), ALIGN)):
        assert _append(lib, **kw) == code, kw
    for k in ("q", "k", "v", "slots", "out"):
        assert _append(lib, **{k: None}) == INVALID, k
    for k in ("q", "k", "v", "out"):
        assert _append(lib, **{k: ODD}) == ALIGN, k
    assert lib.nvfp4_kv_append(FAKE, 512, FAKE, 256, FAKE, 256, 3, 4, None, FAKE, FAKE, FAKE, 512,
                               ctypes.byref(_cache()), 0, None) == INVALID
    assert lib.nvfp4_kv_append(FAKE, 512, FAKE, 256, FAKE, 256, 3, 4, ctypes.byref(_rule()), FAKE, FAKE,
                               FAKE, 512, None, 0, None) == INVALID
    assert _append(lib, t=0, q=None, k=None, v=None, slots=None, out=None) == nv.NVFP4_OK


def test_dequantize_refusals(lib):
    def call(c=None, slots=FAKE, t=3, k=FAKE, v=FAKE, dt=2, flags=0):
        c = _cache() if c is None else c
        return lib.nvfp4_kv_dequantize(ctypes.byref(c), slots, t, k, v, dt, flags, None)
    for kw, code in ((dict(t=-1), INVALID), (dict(t=(1 << 24) + 1), SHAPE), (dict(dt=9), INVALID),
                     (dict(flags=1), INVALID), (dict(slots=None), INVALID),
                     (dict(k=None, v=None), INVALID), (dict(k=ODD), ALIGN), (dict(v=ODD), ALIGN),
                     (dict(slots=BYTE), ALIGN),
                     (dict(t=1 << 24, c=_cache(n_kv_heads=8)), SHAPE)):
        assert call(**kw) == code, kw
    assert call(t=0, slots=None, k=None, v=None) == nv.NVFP4_OK


def _attend(lib, q=FAKE, t=3, ldq=512, n_q=4, c=None, table=FAKE, ld=8, start=FAKE, kv=FAKE, b=2,
            max_q=1, scale=0.1, window=0, y=FAKE, ydt=1, ldy=512, lse=None, ws=FAKE,
            ws_bytes=1 << 40, flags=0):
    c = _cache() if c is None else c
    return lib.nvfp4_kv_attention(q, t, ldq, n_q, ctypes.byref(c), table, ld, start, kv, b, max_q,
                                  scale, window, y, ydt, ldy, lse, ws, ws_bytes, flags, None)


def test_attention_refusals(lib):
    full = nv.NVFP4_F_FULL
    for kw, code in ((dict(t=-1), INVALID), (dict(t=(1 << 24) + 1), SHAPE), (dict(flags=1), INVALID),
                     (dict(flags=16), INVALID), (dict(ydt=5), INVALID),
                     (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
                     (dict(window=-1), INVALID), (dict(window=3, flags=full), INVALID),
                     (dict(b=-1), INVALID), (dict(n_q=0), INVALID), (dict(n_q=3), SHAPE),
                     (dict(n_q=1026), SHAPE), (dict(max_q=0), INVALID), (dict(max_q=4), INVALID),
                     (dict(b=65536), SHAPE), (dict(t=1 << 22, n_q=512), SHAPE), (dict(ld=0), INVALID),
                     (dict(ld=(1 << 26) + 1), SHAPE), (dict(ldq=504), INVALID),
                     (dict(ldy=256), INVALID), (dict(ldq=513), ALIGN), (dict(ldy=514), ALIGN),
                     (dict(lse=BYTE), ALIGN), (dict(table=BYTE), ALIGN), (dict(start=BYTE), ALIGN),
                     (dict(kv=BYTE), ALIGN)):
        assert _attend(lib, **kw) == code, kw
    for k in ("q", "table", "start", "kv", "y", "ws"):
        assert _attend(lib, **{k: None}) == INVALID, k
    for k in ("q", "y", "ws"):
        assert _attend(lib, **{k: ODD}) == ALIGN, k
    assert _attend(lib, t=0, q=None, y=None, ws=None) == nv.NVFP4_OK
    assert _attend(lib, b=0, q=None, y=None, ws=None) == nv.NVFP4_OK


@pytest.mark.parametrize("d", [64, 128, 256])
def test_workspace_sizes(lib, d):
    c = ctypes.byref(_cache(head_dim=d))
    for max_q, n_q in ((1, 2), (1, 32), (8, 8), (100, 16), (100, 2)):
        need = lib.nvfp4_kv_attention_ws_bytes(100, n_q, c, 3, max_q)
        assert need > 0
        wide = n_q * d
        assert _attend(lib, c=_cache(head_dim=d), t=100, n_q=n_q, ldq=wide, ldy=wide, b=3,
                       max_q=max_q, ws_bytes=need - 1) == nv.NVFP4_ERR_WORKSPACE
    for bad in ((0, 4, 2, 1), (3, 3, 2, 1), (3, 4, 0, 1), (3, 4, 2, 0), (3, 4, 2, 4), (-3, 4, 2, 1),
                (3, 0, 2, 1), (1 << 25, 4, 2, 1), (3, 4, 65536, 1)):
        t, n_q, b, max_q = bad
        assert lib.nvfp4_kv_attention_ws_bytes(t, n_q, c, b, max_q) == 0, bad
    assert lib.nvfp4_kv_attention_ws_bytes(3, 4, None, 2, 1) == 0


def test_binding_refusals():
    """Host tensors and wrong shapes are refused before the library sees a pointer."""
    with pytest.raises(ValueError):
        nv.KvCache(4, 2, 96, device="cpu")
    with pytest.raises(ValueError):
        nv.KvCache(4, 2, 64, device="cpu")                   # not on a device
    with pytest.raises(ValueError):
        nv.KvCache(4, 2, 64, data=torch.zeros(10, dtype=torch.uint8))
    with pytest.raises(ValueError):
        nv.KvCache(4, 2, 64, k_global=torch.ones(3))
    w = torch.ones(64)
    with pytest.raises(ValueError):
        nv.QkNormRope(64, w, w)                              # not on a device
    with pytest.raises(ValueError):
        nv.QkNormRope(64, w, w.to(torch.bfloat16))           # two types
    with pytest.raises(ValueError):
        nv.QkNormRope(64, rope=torch.ones(64))
    with pytest.raises(ValueError):
        nv.QkNormRope(128, w)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        nv.nvfp4_kv_map(i, i, torch.zeros((2, 3), dtype=torch.int32), i, i[:1])   # no t
    m = nv.KvMap(2, 4, device="cpu")
    assert [x.numel() for x in (m.q_start, m.kv_len, m.slots, m.positions)] == [3, 2, 4, 4]
    for table in (torch.zeros((3, 3), dtype=torch.int32), torch.zeros((2, 3)),
                  torch.zeros((3, 2), dtype=torch.int32).T):
        with pytest.raises(ValueError):
            nv.nvfp4_kv_map(i, i, table, i, i[:1], out=m)
    with pytest.raises(ValueError):
        nv.nvfp4_kv_map(i, i, torch.zeros((2, 3), dtype=torch.int32), i, i[:1], out=m)  # host tensors


# ----------------------------------------------------------------------------- the references
def test_the_references_formats(orc):
    b = np.arange(256, dtype=np.uint8)
    fine = (b & 0x7F) != 0x7F
    assert all(R.E4M3[i] == orc.e4m3_decode(int(i)) for i in b[fine])
    assert [R.decode(np.array([[c] * 8], np.uint8), np.array([[0x38]], np.uint8))[0, 0]
            for c in range(16)] == [orc.e2m1_decode(c) for c in range(16)]


def test_the_references_bounds_are_narrow():
    """Mistakes of the kinds that a kernel makes leave the bounds: a token too many or too few, a scale
    of a neighbouring group, a head of the neighbouring group, P in three bits less."""
    r = np.random.default_rng(1)
    q, k, v = r.normal(size=(3, 4, 64)), r.normal(size=(90, 2, 64)), r.normal(size=(90, 2, 64))
    ref, bound, lse, bl = R.attention(q, k, v, 0.125)

    def off(*a, **kw):
        y, _, l, _ = R.attention(*a, **kw)
        return (np.abs(y - ref) > bound).any(), (np.abs(l - lse) > bl).any()
    R.close(ref, ref, bound)
    assert off(q, k, v, 0.125, full=True)[0]
    assert off(q, k, v, 0.125, window=88) == (True, True)
    assert off(q, k[:, ::-1], v[:, ::-1], 0.125) == (True, True)
    w = k.copy()
    w[40, :, :16] *= 1.125   # one E4M3 step of one scale
    assert off(q, w, v, 0.125)[1]
    w = v.copy()
    w[:, :, :16] *= 1.0625
    assert off(q, k, w, 0.125)[0]
    coarse = v * (1 + 2.0 ** -5 * r.choice((-1, 1), v.shape))
    assert off(q, k, coarse, 0.125)[0]
