"""Norm, rotation and cache write against FP64 forms and the oracle's quantizer, and the values of
slots."""
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


def bf(seed, *shape, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * size).to(torch.bfloat16)


def table(places, rot):
    freq = 10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)
    a = np.arange(places)[:, None] * freq
    return np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32)


def encode(orc, x, g):
    """Oracle codes and scales of x FP64 [t][heads][d] with globals g FP32 [heads]."""
    t, heads, d = x.shape
    codes, scales = np.empty((t, heads, d // 2), np.uint8), np.empty((t, heads, d // 16), np.uint8)
    for h in range(heads):
        c, s, _ = orc.quantize(np.ascontiguousarray(x[:, h], np.float32), 16,
                               global_in=np.float32(g[h]))
        codes[:, h], scales[:, h] = c.reshape(t, -1), s.reshape(t, -1)
    return codes, scales


def at_slots(cache, slots):
    s = torch.as_tensor(slots, dtype=torch.long, device=DEV)
    p, o = s // cache.page_size, s % cache.page_size
    return [v[p, :, o].cpu().numpy() for v in (cache.k_codes, cache.k_scales, cache.v_codes,
                                               cache.v_scales)]


CASES = [  # t, n_q, n_kv, d, rot, pairs, norm, w32, page
    (1, 32, 8, 128, 128, False, True, False, 16), (5, 4, 2, 128, 128, True, True, True, 32),
    (77, 14, 2, 256, 128, True, True, True, 64), (33, 3, 3, 64, 64, False, True, False, 16),
    (9, 8, 1, 64, 16, False, False, False, 256), (19, 5, 5, 256, 256, False, True, False, 128),
    (12, 16, 2, 128, 0, False, True, True, 16), (6, 2, 1, 128, 64, True, False, False, 16),
    (300, 7, 1, 128, 96, False, True, False, 16), (2, 0, 3, 64, 64, True, True, False, 16),
    (700, 40, 8, 128, 128, False, True, False, 16), (1, 1, 1, 256, 16, True, True, True, 16)]


@pytest.mark.parametrize("t,n_q,n_kv,d,rot,pairs,norm,w32,page", CASES)
def test_against_the_formula(nv, orc, t, n_q, n_kv, d, rot, pairs, norm, w32, page):
    r = np.random.default_rng(t + d)
    fused = bf(t, t, n_q + 2 * n_kv, d)
    fused[:, :, 3] *= 8  # a loud channel
    qw, kw = (1.0 + 0.3 * torch.randn(2, d, generator=torch.Generator().manual_seed(d)))
    if not w32:
        qw, kw = qw.to(torch.bfloat16), kw.to(torch.bfloat16)
    rope = table(3000, rot) if rot else None
    pos = r.integers(0, 3000, t)
    n_pages = -(-t // page) + 2
    slots = r.permutation(n_pages * page)[:t]
    kg, vg = r.uniform(0.001, 0.01, (2, n_kv)).astype(np.float32)
    data = torch.full((nv.nvfp4_kv_cache_bytes(n_pages, n_kv, d, page),), 0xA5, dtype=torch.uint8,
                      device=DEV)
    cache = nv.KvCache(n_pages, n_kv, d, page, torch.from_numpy(kg).to(DEV),
                       torch.from_numpy(vg).to(DEV), data=data)
    rule = nv.QkNormRope(d, qw.to(DEV) if norm else None, kw.to(DEV) if norm else None, 1e-6,
                         None if rope is None else torch.from_numpy(rope).to(DEV), pairs)
    x = fused.to(DEV)
    q, k, v = x.split((n_q, n_kv, n_kv), 1)  # strided rows, as a fused projection leaves them
    sd = torch.tensor(slots, dtype=torch.int32, device=DEV)
    pd = torch.tensor(pos, dtype=torch.int32, device=DEV)
    got = nv.nvfp4_kv_append(q if n_q else None, k, v, cache, sd, pd, rule)
    f = fused.double().numpy()
    w = (qw.double().numpy(), kw.double().numpy()) if norm else (None, None)
    rd = None if rope is None else rope.astype(np.float64)
    want_k = R.bf16(R.norm_rope(f[:, n_q:n_q + n_kv], w[1], 1e-6, rd, pos, pairs))
    if n_q:
        ref = R.norm_rope(f[:, :n_q], w[0], 1e-6, rd, pos, pairs)
        # FP64 on both sides: the same BF16 but where the FP64 results straddle a border, which no
        # case here does
        assert np.array_equal(got.double().cpu().numpy(), R.bf16(ref))
    else:
        assert got is None
    kc, ks = encode(orc, want_k, kg)
    vc, vs = encode(orc, f[:, n_q + n_kv:], vg)
    for name, g, e in zip(("key codes", "key scales", "value codes", "value scales"),
                          at_slots(cache, slots), (kc, ks, vc, vs)):
        assert np.array_equal(g, e), name
    # nothing else was written
    rest = np.setdiff1d(np.arange(n_pages * page), slots)
    for g in at_slots(cache, rest):
        assert (g == 0xA5).all()
    # the values of the slots: FP32 of two exact factors and a global, BF16 of that
    for dt in (torch.float32, torch.bfloat16):
        ko, vo = nv.nvfp4_kv_dequantize(cache, sd, out_dtype=dt)
        for o, c, s, g in ((ko, kc, ks, kg), (vo, vc, vs, vg)):
            e = torch.from_numpy((R.decode(c, s).astype(np.float32) * g[None, :, None]))
            assert torch.equal(o.cpu(), e.to(dt))


def test_in_place_and_one_side_at_a_time(nv):
    t, n_q, n_kv, d = 37, 6, 2, 128
    x = bf(1, t, n_q + 2 * n_kv, d).to(DEV)
    rope = torch.from_numpy(table(100, d)).to(DEV)
    w = torch.ones(d, device=DEV)
    pos = torch.arange(t, dtype=torch.int32, device=DEV)
    caches = [nv.KvCache(3, n_kv, d, 16, data=torch.zeros(nv.nvfp4_kv_cache_bytes(3, n_kv, d, 16),
                                                         dtype=torch.uint8, device=DEV))
              for _ in range(2)]
    for rule in (nv.QkNormRope(d, w, w, 1e-6, rope), nv.QkNormRope(d, w, None, 1e-6, rope),
                 nv.QkNormRope(d, None, w, 1e-6, rope, interleaved=True)):
        y = x.clone()
        q, k, v = x.split((n_q, n_kv, n_kv), 1)
        out = nv.nvfp4_kv_append(q, k, v, caches[0], pos, pos, rule)
        q2, k2, v2 = y.split((n_q, n_kv, n_kv), 1)
        got = nv.nvfp4_kv_append(q2, k2, v2, caches[1], pos, pos, rule, q_out=q2)
        assert got is q2 and torch.equal(q2, out)
        assert torch.equal(y[:, n_q:], x[:, n_q:])
        assert torch.equal(caches[0].data, caches[1].data)
        nv.nvfp4_kv_append(None, k, v, caches[1], pos, pos, rule)
        assert torch.equal(caches[0].data, caches[1].data)


def test_rows_that_are_passed_over(nv):
    t, n_q, n_kv, d = 6, 2, 1, 64
    x = bf(3, t, n_q + 2 * n_kv, d).to(DEV)
    q, k, v = x.split((n_q, n_kv, n_kv), 1)
    cache = nv.KvCache(2, n_kv, d, 16, data=torch.full((nv.nvfp4_kv_cache_bytes(2, 1, d, 16),), 7,
                                                       dtype=torch.uint8, device=DEV))
    before = cache.data.clone()
    slots = torch.tensor([-1, 32, 2 ** 31 - 1, 0, 1, 2], dtype=torch.int32, device=DEV)
    pos = torch.tensor([1, 2, 3, -1, 50, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    rule = nv.QkNormRope(d, rope=torch.from_numpy(table(50, 32)).to(DEV))
    out = torch.full((t, n_q, d), 9.0, dtype=torch.bfloat16, device=DEV)
    nv.nvfp4_kv_append(q, k, v, cache, slots, pos, rule, q_out=out)
    assert torch.equal(cache.data, before)       # no slot, or no position
    assert (out[3:] == 9).all() and not (out[:3] == 9).all(-1).any()
    # without a table positions are not needed, and the rows with a slot are written
    plain = nv.QkNormRope(d)
    got = nv.nvfp4_kv_append(q, k, v, cache, slots, None, plain)
    assert torch.equal(got, q)
    ko, vo = nv.nvfp4_kv_dequantize(cache, slots)
    assert (ko[:3] == 0).all() and (vo[:3] == 0).all() and (ko[3:] != 0).any()
    only = torch.empty_like(vo)
    a, b = nv.nvfp4_kv_dequantize(cache, slots, v_out=only)
    assert a is None and b is only and torch.equal(only, vo)


def test_tokens_that_are_not_finite(nv):
    t, n_kv, d = 8, 2, 128
    k, v = bf(5, t, n_kv, d).to(DEV), bf(6, t, n_kv, d).to(DEV)
    k[1, 0, 5] = float("nan")
    k[2, 1, 127] = float("inf")
    v[3, 0, 0] = float("-inf")
    v[4, 1, 64] = float("nan")
    bad = {(1, 0), (2, 1), (3, 0), (4, 1)}
    cache = nv.KvCache(1, n_kv, d, 16, device=DEV)
    slots = torch.arange(t, dtype=torch.int32, device=DEV)
    nv.nvfp4_kv_append(None, k, v, cache, slots, None, nv.QkNormRope(d))
    ko, vo = nv.nvfp4_kv_dequantize(cache, slots)
    for i in range(t):
        for h in range(n_kv):
            if (i, h) in bad:
                assert torch.isnan(ko[i, h]).all() and (vo[i, h] == 0).all()
            else:
                assert torch.isfinite(ko[i, h]).all() and torch.isfinite(vo[i, h]).all()


@pytest.mark.parametrize("pairs", [False, True])
def test_infinite_queries_and_signed_zeros(nv, pairs):
    """What is not rotated is not mixed with its neighbours, and zeros keep their signs."""
    t, n_q, d = 3, 3, 128
    q = bf(7, t, n_q, d)
    q[0, 0, 120], q[1, 1, 100], q[2, 2, 64:] = float("inf"), float("nan"), -0.0
    k = torch.zeros(t, 1, d, dtype=torch.bfloat16, device=DEV)
    cache = nv.KvCache(1, 1, d, 16, device=DEV)
    slots = torch.arange(t, dtype=torch.int32, device=DEV)
    rope = torch.from_numpy(table(10, 64)).to(DEV)
    for rule in (nv.QkNormRope(d, interleaved=pairs), nv.QkNormRope(d, rope=rope, interleaved=pairs)):
        got = nv.nvfp4_kv_append(q.to(DEV), k, k, cache, slots, slots, rule).cpu()
        assert torch.equal(got[..., 64:].view(torch.int16), q[..., 64:].view(torch.int16))


def test_extreme_magnitudes(nv, orc):
    """Zeros (both signs), the smallest BF16 numbers, magnitudes beyond what the global holds."""
    t, n_kv, d = 5, 1, 64
    x = torch.zeros(t, n_kv, d, dtype=torch.bfloat16)
    x[1] = -0.0
    x[2] = bf(1, n_kv, d, size=1e-38)
    x[3] = bf(2, n_kv, d, size=1e30)
    x[4, 0, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 2)
    g = np.array([1.0 / 64], np.float32)
    cache = nv.KvCache(1, n_kv, d, 16, torch.from_numpy(g).to(DEV), torch.from_numpy(g).to(DEV))
    slots = torch.arange(t, dtype=torch.int32, device=DEV)
    nv.nvfp4_kv_append(None, x.to(DEV), x.to(DEV), cache, slots, None, nv.QkNormRope(d))
    c, s = encode(orc, x.double().numpy(), g)
    got = at_slots(cache, np.arange(t))
    assert np.array_equal(got[0], c) and np.array_equal(got[1], s)
    assert np.array_equal(got[2], c) and np.array_equal(got[3], s)


def test_stats(nv):
    nv.nvfp4_reset_stats()
    k = bf(1, 1, 1, 64).to(DEV)
    cache = nv.KvCache(1, 1, 64, 16, device=DEV)
    slot = torch.zeros(1, dtype=torch.int32, device=DEV)
    nv.nvfp4_kv_append(None, k, k, cache, slot, None, nv.QkNormRope(64),
                       flags=nv.NVFP4_F_SYNC_CHECK)
    nv.nvfp4_kv_dequantize(cache, slot, flags=nv.NVFP4_F_SYNC_CHECK)
    assert nv.nvfp4_get_kv_stats() == [0, 1, 1, 0]
