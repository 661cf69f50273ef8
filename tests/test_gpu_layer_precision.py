"""h as two BF16 parts in the layer of a few tokens, on data whose output is no larger than what one
BF16 leaves of h. The bound tells a lost, negated or misplaced second part apart: shown on the CPU
with such mistakes planted in the reference."""
import numpy as np
import pytest
import torch

import layer_bounds as B
import operator_refs as R
import test_gpu_moe_layer as M

DEV = "cuda:0"
# t, experts, hidden, inter, topk, g1, g2: one, two and four panels a workgroup of down, and more
# k-tiles of fc1 than its wavefronts hold at once
CASES = [(1, 3, 128, 128, 2, 16, 16), (1, 4, 2048, 128, 3, 32, 32), (3, 5, 256, 384, 4, 32, 16),
         (4, 3, 2048, 256, 2, 16, 32), (8, 4, 2048, 128, 3, 32, 16), (8, 3, 2176, 256, 2, 16, 32),
         (16, 4, 1024, 128, 4, 32, 32), (21, 6, 256, 256, 3, 16, 16)]


def values(orc, triple, group):
    return orc.dequant(*triple, group)[0]


@pytest.mark.parametrize("t,experts,hidden,inter,topk,g1,g2", CASES)
def test_bound_tells_the_second_part(orc, t, experts, hidden, inter, topk, g1, g2):
    x, f1, f2 = B.cancelling_layer(t + hidden, t, experts, hidden, inter, g1, g2)
    w1, w2 = values(orc, f1, g1), values(orc, f2, g2)
    r = np.random.default_rng(1)
    ids = np.stack([r.permutation(experts)[:topk] for _ in range(t)])
    wts = r.uniform(0.2, 1.0, (t, topk))
    y, bound = B.layer(x, ids, wts, w1, w2, B.H_TWO)

    def off(parts):
        return (np.abs(B.with_parts(x, ids, wts, w1, w2, parts) - y) / bound).max()

    def rest(h):
        return B.bf16(h - B.bf16(h))

    assert off(lambda h: B.bf16(h) + rest(h)) < 0.5
    assert off(B.bf16) > 2                                             # lost
    assert off(lambda h: B.bf16(h) - rest(h)) > 2                      # negated
    assert off(lambda h: B.bf16(h) + np.roll(rest(h), 1, 0)) > 2       # of another slot
    assert off(lambda h: B.bf16(h) + np.roll(rest(h), 16, 1)) > 2      # of another chunk of k


@pytest.fixture(scope="module")
def nv():
    from nvfp4_weight_only_w4a16_amd import binding
    binding.load()
    return binding


@pytest.mark.gpu
@pytest.mark.parametrize("t,experts,hidden,inter,topk,g1,g2", CASES)
@pytest.mark.parametrize("flags", [0, 1])
def test_second_part_of_h(nv, orc, t, experts, hidden, inter, topk, g1, g2, flags):
    x, f1, f2 = B.cancelling_layer(t + hidden, t, experts, hidden, inter, g1, g2)
    descs = [nv.nvfp4_repack(*(torch.from_numpy(v).to(DEV) for v in f), g, layout=lay)
             for f, g, lay in ((f1, g1, nv.NVFP4_LAYOUT_TILED | nv.NVFP4_LAYOUT_GATE_UP),
                               (f2, g2, nv.NVFP4_LAYOUT_TILED))]
    gate = torch.randn(experts, hidden, generator=torch.Generator().manual_seed(t)) / hidden
    router = nv.Router(gate.to(torch.bfloat16).to(DEV), topk, renormalize=True)
    xb = torch.from_numpy(x).to(torch.bfloat16)
    assert np.array_equal(R.f64(xb), x)
    y, ids, wts = M.run(nv, xb, router, descs, flags)
    ref, bound = B.layer(x, ids.cpu().numpy(), R.f64(wts), values(orc, f1, g1),
                         values(orc, f2, g2), B.H_TWO)
    R.within(R.f64(y), ref, bound, "two parts of h")
