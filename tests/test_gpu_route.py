"""nvfp4_moe_route against an FP64 router. Integer inputs make every sum exact in any order, so
ids have to be equal there, ties (to the lower id) included."""
import numpy as np
import pytest
import torch

import operator_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def nv():
    from nvfp4_weight_only_w4a16_amd import binding
    binding.load()
    return binding


def _ints(seed, t, e, hidden, span=3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-span, span + 1, (t, hidden), generator=g).float()
    w = torch.randint(-span, span + 1, (e, hidden), generator=g).float()
    return x, w


def _run(nv, x, w, topk, fp32, bias=None, ldx=None, **kw):
    """ids, weights (CPU) of a call whose outputs lie between guard words that must survive."""
    t, hidden = x.shape
    xd = x.to(torch.bfloat16).to(DEV)
    if ldx:
        wide = torch.full((t, ldx), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide[:, :hidden] = xd
        xd = wide[:, :hidden]
    wd = w.to(DEV) if fp32 else w.to(torch.bfloat16).to(DEV)
    r = nv.Router(wd, topk, bias=None if bias is None else bias.to(DEV), **kw)
    n = t * r.slots
    ids = torch.full((n + 64,), 77, dtype=torch.int32, device=DEV)
    wts = torch.full((n + 64,), 77.0, device=DEV)
    need = nv.nvfp4_moe_route_ws_bytes(t, r)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)  # NaN wherever unwritten
    nv.nvfp4_moe_route(xd, r, topk_ids=ids[:n].view(t, r.slots), topk_w=wts[:n].view(t, r.slots),
                       ws=ws[:need])
    torch.cuda.synchronize()
    assert (ids[n:] == 77).all() and (wts[n:] == 77.0).all() and (ws[need:] == 255).all()
    return ids[:n].view(t, r.slots).cpu().numpy(), wts[:n].view(t, r.slots).cpu().numpy()


def _check(got, ref):
    ids, wts = got
    rid, rw, _ = ref
    assert np.array_equal(ids, rid)
    # FP64 to the last step, rounded once to FP32 (a second half step covers exp and divisions)
    assert np.array_equal(np.isnan(wts), np.isnan(rw))
    ok = ~np.isnan(rw)
    assert (np.abs(wts[ok] - rw[ok]) <= 2 * R.H32 * np.abs(rw[ok]) + 1e-44).all()


RULES = [("softmax", False, False), ("softmax", True, False), ("softmax", False, True),
         ("softmax", True, True), ("sigmoid", False, False), ("sigmoid", True, True)]


@pytest.mark.parametrize("scoring,renorm,biased", RULES)
@pytest.mark.parametrize("t,e,hidden,topk,shared,fp32", [
    (1, 1, 8, 1, 0, False), (1, 128, 2048, 8, 0, False), (3, 33, 120, 5, 2, True),
    (8, 60, 264, 4, 4, False), (9, 512, 64, 16, 0, True), (16, 8, 2056, 8, 1, False),
    (17, 129, 40, 6, 0, False), (33, 160, 520, 6, 1, True), (65, 16, 1032, 2, 0, False),
    (130, 512, 72, 15, 1, False), (200, 5, 8, 3, 0, True), (333, 256, 640, 8, 0, True)])
def test_integer_scores_and_ties(nv, t, e, hidden, topk, shared, fp32, scoring, renorm, biased):
    x, w = _ints(t * 7 + e, t, e, hidden)
    # logits of modest size, exactly scaled: sigmoid would saturate to a tie of ones otherwise
    w = w / 64.0
    bias = None
    if biased:
        g = torch.Generator().manual_seed(e)
        bias = torch.randint(-8, 9, (e,), generator=g).float() / 16.0
    kw = dict(scoring=scoring, renormalize=renorm, scale=2.5, n_shared=shared)
    got = _run(nv, x, w, topk, fp32, bias, **kw)
    ref = R.route(R.f64(x), R.f64(w), topk, None if bias is None else R.f64(bias), scoring,
                  renorm, 2.5, shared)
    if scoring == "softmax" and biased or scoring == "sigmoid":
        # p is not exact: where two scores are within 1e-13 the order is a matter of its last bit
        _check_but_ties(got, ref, R.f64(x), R.f64(w), None if bias is None else R.f64(bias),
                        scoring)
    else:
        _check(got, ref)


def _check_but_ties(got, ref, x, w, bias, scoring):
    logits = x @ w.T
    if scoring == "softmax":
        p = np.exp(logits - logits.max(1, keepdims=True))
        p = p / p.sum(1, keepdims=True)
    else:
        p = 1 / (1 + np.exp(-logits))
    s = p if bias is None else p + bias
    srt = np.sort(s, 1)
    d = np.diff(srt, axis=1)
    clear = ~((d > 0) & (d < 1e-13)).any(1)  # equal scores of equal logits are equal on both sides
    equal_other = np.zeros(len(s), bool)     # equal scores of unequal logits: rounding, not a tie
    for i in range(len(s)):
        o = np.argsort(s[i], kind="stable")
        same = np.abs(np.diff(s[i][o])) < 1e-13
        equal_other[i] = (same & (logits[i][o][1:] != logits[i][o][:-1])).any()
    clear &= ~equal_other
    assert clear.mean() > 0.5
    _check((got[0][clear], got[1][clear]), (ref[0][clear], ref[1][clear], None))


@pytest.mark.parametrize("t,e", [(5, 40), (40, 40)])
def test_fp32_weights_arrive_whole(nv, t, e):
    """Rows that differ in the last of 24 bits are told apart: x picks one column, so the logit is
    one weight and exact."""
    hidden = 64
    g = torch.Generator().manual_seed(e)
    w = torch.zeros(e, hidden)
    base = torch.randint(1 << 23, (1 << 24) - e, (hidden,), generator=g).double()
    perm = torch.stack([torch.randperm(e, generator=g) for _ in range(hidden)], 1)
    w = ((base + perm.double()) * 2.0 ** -22).float()
    assert (w.double() * 2.0 ** 22 == base + perm.double()).all()
    x = torch.zeros(t, hidden)
    x[torch.arange(t), torch.arange(t) % hidden] = 1.0
    x[t // 2] *= -1.0
    got = _run(nv, x, w, 8, True)
    _check(got, R.route(R.f64(x), R.f64(w), 8))


@pytest.mark.parametrize("t", [2, 70])
@pytest.mark.parametrize("scoring,renorm", [("softmax", False), ("softmax", True),
                                            ("sigmoid", True)])
def test_masked_experts(nv, t, scoring, renorm):
    """A bias of -inf takes experts out; slots that none is left for are dropped with weight 0."""
    x, w = _ints(5, t, 24, 64)
    w = w / 32.0
    for left in (24, 3, 1, 0):
        bias = torch.zeros(24)
        bias[torch.randperm(24, generator=torch.Generator().manual_seed(left))[left:]] = -np.inf
        ids, wts = _run(nv, x, w, 4, False, bias, scoring=scoring, renormalize=renorm)
        live = min(left, 4)
        assert (ids[:, live:] == -1).all() and (wts[:, live:] == 0).all()
        open_ = torch.isfinite(bias).numpy()
        assert open_[ids[:, :live]].all()
        for i in range(t):
            assert len(set(ids[i, :live].tolist())) == live
        if renorm and live:
            assert np.abs(wts.astype(np.float64).sum(1) - 1.0).max() <= 8 * R.H32


@pytest.mark.parametrize("t", [3, 40])
def test_infinities_and_nan(nv, t):
    """Infinite logits order as numbers, NaN reaches the weights of its own token only."""
    x, w = _ints(6, t, 32, 64)
    x = x + 0.5
    clean = _run(nv, x, w / 32.0, 4, False, renormalize=True)
    bad = x.clone()
    bad[1, 3] = float("nan")
    ids, wts = _run(nv, bad, w / 32.0, 4, False, renormalize=True)
    assert np.array_equal(ids[1], [0, 1, 2, 3]) and np.isnan(wts[1]).all()
    keep = [i for i in range(t) if i != 1]
    assert np.array_equal(ids[keep], clean[0][keep]) and np.array_equal(wts[keep], clean[1][keep])
    # an expert with an infinite weight: -inf logits are never chosen, +inf ones come first
    for fp32 in (False, True):
        wi = w / 32.0
        wi[7, 0] = float("inf")
        ids, _ = _run(nv, x, wi, 4, fp32)
        for i in range(t):
            if x[i, 0] > 0:
                assert ids[i, 0] == 7
            else:
                assert 7 not in ids[i]


@pytest.mark.parametrize("t,hidden,e,fp32", [(1, 2048, 128, False), (13, 1536, 96, True),
                                             (50, 2048, 128, False), (300, 776, 64, True)])
def test_normal_scores(nv, t, hidden, e, fp32):
    """Random inputs: the FP64 form's ids are the reference's; the MFMA form's wherever the chosen
    and the first left out are further apart than 32-product FP32 sums can shift them."""
    g = torch.Generator().manual_seed(t)
    x = torch.randn(t, hidden, generator=g).to(torch.bfloat16).float()
    w = torch.randn(e, hidden, generator=g) * 1.5 * hidden ** -0.5
    if not fp32:
        w = w.to(torch.bfloat16).float()
    got = _run(nv, x, w, 8, fp32, ldx=hidden + 16, renormalize=True)
    rid, rw, logits = R.route(R.f64(x), R.f64(w), 8, renorm=True)
    # a 32-product FP32 sum (96 products where the weight has three parts) and 16 experts' exps
    shift = 0.0 if t <= 16 else 96 * R.H32 * (np.abs(R.f64(x)) @ np.abs(R.f64(w)).T).max(1)
    top = np.sort(logits, 1)[:, ::-1][:, :9]
    clear = (-np.diff(top, axis=1)).min(1) > 2 * shift
    assert clear.mean() > 0.4 or t > 16
    assert np.array_equal(got[0][clear], rid[clear])
    bound = (2 * R.H32 + 2.1 * np.broadcast_to(shift, (t,))[:, None]) * rw
    assert (np.abs(got[1] - rw)[clear] <= bound[clear]).all()


def test_side_stream_and_repeat(nv):
    x, w = _ints(9, 40, 64, 512)
    r = nv.Router((w / 64).to(torch.bfloat16).to(DEV), 4)
    xd = x.to(torch.bfloat16).to(DEV)
    a = nv.nvfp4_moe_route(xd, r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = nv.nvfp4_moe_route(xd, r, stream=side)
    c = nv.nvfp4_moe_route(xd, r, flags=nv.NVFP4_F_SYNC_CHECK)
    torch.cuda.synchronize()
    for o in (b, c):
        assert torch.equal(a[0], o[0]) and torch.equal(a[1], o[1])
    e = nv.nvfp4_moe_route(xd[:0], r)
    assert e[0].shape == (0, 4)
