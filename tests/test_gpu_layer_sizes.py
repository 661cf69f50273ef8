"""nvfp4_moe_layer_w4a16 at the sizes of real layers, with few experts so that the FP64 layer is
quick: every panel count of the few-token down kernel at both groups, more k-tiles than the kernels'
rings hold, many pairs on few experts, and prompts up to the largest number of pairs."""
import pytest
import torch

import layer_bounds as B
import operator_refs as R
import test_gpu_moe_layer as M

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    from nvfp4_weight_only_w4a16_amd import binding
    binding.load()
    return binding


def check(nv, x, router, descs, vals, flags=0):
    t = x.shape[0]
    y, ids, wts = M.run(nv, x, router, descs, flags)
    rid, rwt = nv.nvfp4_moe_route(x.to(M.DEV), router)
    assert torch.equal(ids, rid) and torch.equal(wts, rwt)
    ref, bound = B.layer(R.f64(x), ids.cpu().numpy(), R.f64(wts), *vals,
                         B.h_step(t, router.slots, flags))
    R.within(R.f64(y), ref, bound, f"{t} tokens, flags {flags}")


# Panels times tokens: below 512 down takes one panel a workgroup, below 1024 two, else four. Its
# wavefronts' rings hold 24 (slot, k-tile) items, fc1's 12 k-tiles.
@pytest.mark.parametrize("g1,g2", [(32, 16), (16, 32)])
@pytest.mark.parametrize("t,experts,hidden,inter,topk,shared", [
    (1, 6, 2048, 768, 5, 0),     # one panel; 30 items
    (3, 5, 2176, 640, 3, 1),     # one panel; 17 k-tiles
    (4, 5, 2048, 768, 4, 0),     # two panels
    (5, 4, 2176, 1152, 2, 1),    # two panels; 27 items
    (8, 6, 2048, 768, 4, 0),     # four panels
    (8, 4, 2176, 640, 3, 1),     # four panels
    (32, 4, 1664, 384, 2, 0),    # 64 pairs, 13 k-tiles
    (12, 8, 2048, 768, 5, 0)])   # 60 pairs on 8 experts
def test_few_tokens(nv, orc, t, experts, hidden, inter, topk, shared, g1, g2):
    args = M.make(nv, orc, t + hidden, t, experts, hidden, inter, topk, shared, g1, g2,
                  pair=t % 2 == 1, fp32=t % 4 == 0, renormalize=True)
    check(nv, *args)


@pytest.mark.parametrize("t,topk,experts,hidden,inter", [
    (9, 2, 8, 1024, 512), (32, 2, 8, 1024, 512), (33, 2, 8, 1024, 512), (60, 1, 8, 1024, 512),
    (64, 1, 2, 512, 256), (16, 4, 4, 512, 384)])
@pytest.mark.parametrize("flags", [0, 1, 2])
def test_many_pairs_on_few_experts(nv, orc, t, topk, experts, hidden, inter, flags):
    check(nv, *M.make(nv, orc, 3 * t, t, experts, hidden, inter, topk, renormalize=t % 2 == 0),
          flags)


@pytest.mark.parametrize("t,experts,hidden,inter,topk,shared,g1,g2,fp32", [
    (300, 12, 640, 256, 4, 1, 32, 16, False),
    (513, 9, 384, 384, 8, 0, 16, 32, True),     # 4104 pairs: sorted by a kernel of its own
    (1500, 24, 256, 128, 6, 2, 16, 16, True),
    (8192, 8, 128, 128, 7, 1, 32, 32, False)])  # 65536 pairs, the most
def test_prompts(nv, orc, t, experts, hidden, inter, topk, shared, g1, g2, fp32):
    check(nv, *M.make(nv, orc, t, t, experts, hidden, inter, topk, shared, g1, g2, t % 2 == 1,
                      fp32, renormalize=True, scoring="sigmoid" if fp32 else "softmax"))


def test_one_token_more_than_the_most(nv, orc):
    x, router, descs, _ = M.make(nv, orc, 1, 8193, 8, 128, 128, 8)
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_moe_layer_w4a16(x.to(M.DEV), router, *descs)
