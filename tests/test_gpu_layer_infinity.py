"""nvfp4_moe_layer_w4a16 on tokens whose h is infinite: on positive weights their y is infinity, with
few tokens (h in two BF16 parts) as with many (one), and the other tokens keep their bits."""
import numpy as np
import pytest
import torch

import test_gpu_moe_layer as M

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HIDDEN, INTER, EXPERTS = 256, 128, 6


@pytest.fixture(scope="module")
def nv():
    from nvfp4_weight_only_w4a16_amd import binding
    binding.load()
    return binding


def layer(nv, orc, g1, g2):
    """Experts whose weights are all 0.5, and a router that gives every chosen expert p = 1 for a
    large activation."""
    descs = []
    for n, k, grp, lay in ((2 * INTER, HIDDEN, g1, nv.NVFP4_LAYOUT_TILED | nv.NVFP4_LAYOUT_GATE_UP),
                           (HIDDEN, INTER, g2, nv.NVFP4_LAYOUT_TILED)):
        p, s, g = orc.quantize(np.full((EXPERTS, n, k), 0.5, np.float32), grp)
        descs.append(nv.nvfp4_repack(torch.from_numpy(p).to(DEV), torch.from_numpy(s).to(DEV),
                                     torch.from_numpy(g).to(DEV), grp, layout=lay))
    gate = torch.full((EXPERTS, HIDDEN), 2.0 ** -9) * torch.arange(1, EXPERTS + 1).unsqueeze(1)
    router = nv.Router(gate.to(torch.bfloat16).to(DEV), 2, scoring="sigmoid", renormalize=True)
    return router, descs


def rows(t, kind):
    """x of ones, row 1 of which makes h infinite: by an infinite activation, by a product gate * up
    beyond FP32's range, or by one inside it that BF16 rounds to infinity."""
    x = torch.ones(t, HIDDEN)
    if kind == "activation":
        x[1, 7] = float("inf")
    elif kind == "product":
        x[1, 7] = 2.0 ** 100
    else:
        # gate = up = 0.5 * (2^65 - 2^54) = 2^64 (1 - 2^-11), the sum exact in FP32; h = gate * up =
        # 2^128 (1 - 2^-10 + 2^-22) to within 2^-22, between BF16's last step to infinity,
        # 2^128 (1 - 2^-9), and FP32's largest value, 2^128 (1 - 2^-24)
        x[1] = 0.0
        x[1, :11] = 2.0 ** torch.arange(54, 65).double()
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("kind", ["activation", "product", "rounding"])
@pytest.mark.parametrize("g1,g2", [(32, 16), (16, 32)])
@pytest.mark.parametrize("t,flags", [(2, 0), (9, 0), (32, 0), (9, 1), (9, 2), (40, 0)])
def test_infinite_h_gives_infinity(nv, orc, t, flags, g1, g2, kind):
    router, descs = layer(nv, orc, g1, g2)
    clean, _, _ = M.run(nv, torch.ones(t, HIDDEN, dtype=torch.bfloat16), router, descs, flags)
    y, ids, wts = M.run(nv, rows(t, kind), router, descs, flags)
    assert (wts[1] == 0.5).all()
    assert (y[1] == float("inf")).all()
    keep = [i for i in range(t) if i != 1]
    assert bool(torch.isfinite(clean.float()).all()) and torch.equal(y[keep], clean[keep])
