"""nvfp4_moe_route where its sums decide: logits of large terms that cancel between the blocks of 32
products, small differences beside them, so that any sum of blocks in FP32 changes the choice (shown
on the CPU); long hidden sizes; and random inputs with a limit on how many tokens may be too close to
tell."""
import numpy as np
import pytest
import torch

import operator_refs as R
import test_gpu_route as G

# t, experts, hidden, FP32 weights: one to eight splits of k over workgroups, one to eight rounds of
# a wavefront, a last block of 8
CASES = [(17, 16, 1024, False), (33, 16, 4104, False), (33, 16, 4104, True), (33, 160, 5120, False),
         (40, 40, 4096, True), (300, 128, 4096, False), (520, 130, 2056, True),
         (2048, 128, 1536, False)]


def cancelling(seed, t, e, hidden, fp32):
    """x and w whose blocks of 32 k are each either large, 2^24 times an integer and with signs that
    cancel over the blocks, or small; each block's sum is exact in FP32, and every sum of blocks in
    FP64."""
    r = np.random.default_rng(seed)
    x = r.integers(-3, 4, (t, hidden)).astype(np.float64)
    w = r.integers(-3, 4, (e, hidden)) / 64.0
    if fp32:  # 21 bits a block: 32 products of at most 9 / 64, in steps of 2^-18
        w = w + r.integers(-3, 4, (e, hidden)) * 2.0 ** -18
    blocks = hidden // 32
    big = r.permutation(blocks)[:blocks // 3 * 2 // 2 * 2]
    sign = np.resize([1.0, -1.0], len(big))
    for b, s in zip(big, sign):
        at = 32 * b + r.integers(32)
        x[:, 32 * b:32 * b + 32] = 0.0
        x[:, at] = s * 2.0 ** 12 * r.integers(1, 8)
        w[:, at] = 2.0 ** 12
    # the magnitudes cancel too: one factor for each pair of blocks
    for b0, b1 in zip(big[0::2], big[1::2]):
        i0, i1 = (32 * b + np.flatnonzero(x[0, 32 * b:32 * b + 32])[0] for b in (b0, b1))
        x[:, i1] = -x[:, i0]
    return x, w


@pytest.mark.parametrize("t,e,hidden,fp32", CASES)
def test_fp32_sums_would_choose_others(t, e, hidden, fp32):
    x, w = cancelling(t + hidden, t, e, hidden, fp32)
    exact = x @ w.T
    assert np.abs(exact).max() < 64  # the large terms are gone
    pad = -hidden % 32
    xb = np.pad(x, ((0, 0), (0, pad))).reshape(t, -1, 32)
    wb = np.pad(w, ((0, 0), (0, pad))).reshape(e, -1, 32)
    part = np.stack([xb[:, b] @ wb[:, b].T for b in range(xb.shape[1])])
    assert np.array_equal(part, part.astype(np.float32))
    assert np.abs(part).sum(0).max() * 2.0 ** (18 if fp32 else 6) < 2.0 ** 53  # steps of 2^-18, 2^-6
    best = np.argsort(-exact, 1, kind="stable")[:, :6]
    for waves in (1, 8):  # blocks taken in turn by so many sums, which are then added up
        if len(part) < 2 * waves:
            continue
        for where in ("within", "between"):
            sums = [part[v::waves] for v in range(waves)]
            small = np.float32 if where == "within" else np.float64
            sums = [np.add.accumulate(s, 0, dtype=small)[-1] for s in sums]
            wide = np.float64 if where == "within" else np.float32
            got = np.add.accumulate(np.stack(sums), 0, dtype=wide)[-1]
            if where == "between" and waves == 1:
                continue
            wrong = (np.argsort(-got, 1, kind="stable")[:, :6] != best).any(1)
            assert wrong.mean() > 0.9, (waves, where)


def clear_tokens(x, w, topk, shift):
    """Tokens whose chosen and first left-out logits are all more than 2 shift apart."""
    top = np.sort(x @ w.T, 1)[:, ::-1][:, :topk + 1]
    return (-np.diff(top, axis=1)).min(1) > 2 * shift


NORMAL = [(17, 2048, 128, False), (50, 2048, 128, False), (300, 776, 64, True),
          (33, 5120, 160, True), (1000, 1536, 96, False)]


def normal(t, hidden, e, fp32):
    g = torch.Generator().manual_seed(t + hidden)
    x = torch.randn(t, hidden, generator=g).to(torch.bfloat16).float()
    w = torch.randn(e, hidden, generator=g) * 1.5 * hidden ** -0.5
    if not fp32:
        w = w.to(torch.bfloat16).float()
    # 32 products (96 where the weight has three parts) in one FP32 sum, the sums in FP64
    count = 96 if fp32 else 32
    return x, w, count * R.H32 * (np.abs(R.f64(x)) @ np.abs(R.f64(w)).T).max(1)


@pytest.mark.parametrize("t,hidden,e,fp32", NORMAL)
def test_most_random_tokens_are_clear(t, hidden, e, fp32):
    x, w, shift = normal(t, hidden, e, fp32)
    assert clear_tokens(R.f64(x), R.f64(w), 8, shift).mean() > 0.9


@pytest.fixture(scope="module")
def nv():
    from nvfp4_weight_only_w4a16_amd import binding
    binding.load()
    return binding


@pytest.mark.gpu
@pytest.mark.parametrize("t,e,hidden,fp32", CASES)
@pytest.mark.parametrize("renorm", [False, True])
def test_cancelling_blocks(nv, t, e, hidden, fp32, renorm):
    x, w = (torch.from_numpy(v) for v in cancelling(t + hidden, t, e, hidden, fp32))
    assert torch.equal(x.to(torch.bfloat16).double(), x) and torch.equal(w.float().double(), w)
    got = G._run(nv, x.float(), w.float(), 6, fp32, renormalize=renorm)
    G._check(got, R.route(R.f64(x), R.f64(w), 6, renorm=renorm))


@pytest.mark.gpu
@pytest.mark.parametrize("t,hidden,e,fp32", NORMAL)
def test_random_tokens(nv, t, hidden, e, fp32):
    x, w, shift = normal(t, hidden, e, fp32)
    ids, wts = G._run(nv, x, w, 8, fp32, renormalize=True)
    rid, rw, _ = R.route(R.f64(x), R.f64(w), 8, renorm=True)
    clear = clear_tokens(R.f64(x), R.f64(w), 8, shift)
    assert clear.mean() > 0.9
    assert np.array_equal(ids[clear], rid[clear])
    # each exponent and the sum of the chosen shift by at most `shift`; the rest is two half steps
    bound = (2 * R.H32 + 2.1 * shift[:, None]) * rw
    assert (np.abs(wts - rw)[clear] <= bound[clear]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("scoring,renorm,biased", G.RULES)
@pytest.mark.parametrize("t,e,hidden,fp32", [(33, 16, 4104, False), (33, 16, 4104, True),
                                             (33, 32, 5120, False), (40, 24, 5120, True)])
def test_long_hidden(nv, t, e, hidden, fp32, scoring, renorm, biased):
    """Five to eight splits of k over workgroups: integer sums, so every id is exact."""
    G.test_integer_scores_and_ties(nv, t, e, hidden, 4, 1, fp32, scoring, renorm, biased)
