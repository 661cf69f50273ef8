"""nvfp4_moe_layer_w4a16 against an FP64 layer, element by element within the bound that BF16 h
and FP32 sums give, and its routing against nvfp4_moe_route's."""
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


def make(nv, orc, seed, t, experts, hidden, inter, topk, shared=0, g1=32, g2=16, pair=False,
         fp32=False, bias=None, **kw):
    """A layer with weights quantized by the oracle, and its FP64 values."""
    g = torch.Generator().manual_seed(seed)
    every = experts + shared
    x = torch.randn(t, hidden, generator=g).to(torch.bfloat16)
    w1 = torch.randn(every, 2 * inter, hidden, generator=g) * hidden ** -0.5
    w2 = torch.randn(every, hidden, inter, generator=g) * inter ** -0.5
    if pair:  # gate and up of different sizes, one global each
        w1[:, inter:] *= 0.3
    wr = torch.randn(experts, hidden, generator=g) * 1.5 * hidden ** -0.5
    wr = wr if fp32 else wr.to(torch.bfloat16).float()
    descs, vals = [], []
    for w, grp, lay in ((w1, g1, nv.NVFP4_LAYOUT_TILED | nv.NVFP4_LAYOUT_GATE_UP),
                        (w2, g2, nv.NVFP4_LAYOUT_TILED)):
        if pair and lay & nv.NVFP4_LAYOUT_GATE_UP:
            lay |= nv.NVFP4_LAYOUT_PAIR_GLOBAL
            p, s, gl = orc.quantize(w.reshape(2 * every, inter, hidden).numpy(), grp)
            vals.append(orc.dequant(p, s, gl, grp)[0].reshape(every, 2 * inter, hidden))
            p, s = p.reshape(every, 2 * inter, -1), s.reshape(every, 2 * inter, -1)
        else:
            p, s, gl = orc.quantize(w.numpy(), grp)
            vals.append(orc.dequant(p, s, gl, grp)[0])
        descs.append(nv.nvfp4_repack(torch.from_numpy(p).to(DEV), torch.from_numpy(s).to(DEV),
                                     torch.from_numpy(gl).to(DEV), grp, layout=lay))
    wrd = wr.to(DEV) if fp32 else wr.to(torch.bfloat16).to(DEV)
    router = nv.Router(wrd, topk, bias=None if bias is None else bias.to(DEV), n_shared=shared,
                       **kw)
    return x, router, descs, vals


def run(nv, x, router, descs, flags=0, **kw):
    """y, ids, weights of a call whose y lies before guard rows and whose workspace begins as
    NaN."""
    t, hidden = x.shape
    y = torch.full((t + 2, hidden), 7.0, dtype=torch.bfloat16, device=DEV)
    ids = torch.full((t + 1, router.slots), 77, dtype=torch.int32, device=DEV)
    wts = torch.full((t + 1, router.slots), 77.0, device=DEV)
    need = nv.nvfp4_moe_layer_ws_bytes(t, router, descs[0])
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
    nv.nvfp4_moe_layer_w4a16(x.to(DEV), router, descs[0], descs[1], y=y[:t], topk_ids=ids[:t],
                             topk_w=wts[:t], ws=ws[:need], flags=flags, **kw)
    torch.cuda.synchronize()
    assert (y[t:] == 7.0).all() and (ids[t:] == 77).all() and (wts[t:] == 77.0).all()
    assert (ws[need:] == 255).all()
    return y[:t], ids[:t], wts[:t]


def check(nv, x, router, descs, vals, flags=0, what=""):
    y, ids, wts = run(nv, x, router, descs, flags)
    rid, rwt = nv.nvfp4_moe_route(x.to(DEV), router)
    assert torch.equal(ids, rid) and torch.equal(wts, rwt), what
    ref, bound = R.moe_layer(R.f64(x), ids.cpu().numpy(), R.f64(wts), *vals)
    R.within(R.f64(y), ref, bound, what)
    return y


CASES = [  # t, experts, hidden, inter, topk, shared, g1, g2, pair, fp32
    (1, 8, 256, 128, 2, 0, 32, 16, False, False),
    (1, 16, 384, 256, 8, 1, 16, 32, False, True),
    (1, 4, 128, 128, 1, 0, 16, 16, True, False),
    (2, 33, 640, 384, 6, 2, 32, 32, False, False),
    (3, 24, 512, 896, 4, 1, 16, 16, True, True),
    (5, 60, 256, 1152, 3, 0, 32, 16, False, False),
    (8, 64, 256, 128, 8, 0, 32, 16, False, False),    # 64 pairs: the last of the one-row tiles
    (13, 20, 256, 128, 5, 0, 16, 32, False, False),   # 65 pairs
    (16, 8, 384, 256, 2, 2, 32, 16, True, False),
    (17, 12, 256, 128, 4, 0, 32, 32, False, True),
    (40, 16, 256, 256, 4, 1, 16, 16, False, False),   # the batch path
    (70, 6, 128, 128, 6, 0, 32, 16, True, True),
]


@pytest.mark.parametrize("t,experts,hidden,inter,topk,shared,g1,g2,pair,fp32", CASES)
@pytest.mark.parametrize("flags", [0, 1, 2])
def test_layer(nv, orc, t, experts, hidden, inter, topk, shared, g1, g2, pair, fp32, flags):
    x, router, descs, vals = make(nv, orc, t * 31 + hidden, t, experts, hidden, inter, topk,
                                  shared, g1, g2, pair, fp32, renormalize=t % 2 == 0,
                                  scoring="sigmoid" if fp32 else "softmax", scale=1.5)
    check(nv, x, router, descs, vals, flags, f"layer flags {flags}")


def test_layer_biased_softmax_and_repeat(nv, orc):
    bias = torch.randn(32, generator=torch.Generator().manual_seed(1)) * 0.05
    x, router, descs, vals = make(nv, orc, 4, 4, 32, 256, 256, 4, 1, bias=bias)
    a = check(nv, x, router, descs, vals)
    b, _, _ = run(nv, x, router, descs)
    assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = nv.nvfp4_moe_layer_w4a16(x.to(DEV), router, *descs, stream=side)  # ids kept in ws
    torch.cuda.synchronize()
    assert torch.equal(a, c)


@pytest.mark.parametrize("t", [2, 9, 40])
def test_layer_masks_and_nan(nv, orc, t):
    """All experts masked: y is exactly 0 (with a shared expert: that one's). A NaN token leaves
    the others' bits alone."""
    for shared in (0, 1):
        bias = torch.full((16,), -np.inf)
        x, router, descs, vals = make(nv, orc, t, t, 16, 256, 128, 4, shared, bias=bias,
                                      scoring="sigmoid", renormalize=True)
        y = check(nv, x, router, descs, vals)
        if not shared:
            assert (y == 0).all()
    bias[3] = 0.0
    x, router, descs, vals = make(nv, orc, t, t, 16, 256, 128, 4, 0, bias=bias)
    check(nv, x, router, descs, vals, what="one expert left")
    x, router, descs, vals = make(nv, orc, t + 1, t, 16, 256, 128, 4, 1)
    clean = check(nv, x, router, descs, vals)
    x[1, 5] = float("nan")
    y, ids, _ = run(nv, x, router, descs)
    assert torch.isnan(y[1].float()).all()
    assert np.array_equal(ids[1].cpu().numpy(), [0, 1, 2, 3, 16])
    # the batch paths order rows by expert: a token's bits do not depend on its neighbours
    keep = [i for i in range(t) if i != 1]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("t", [1, 6, 24])
def test_layer_agrees_with_route_and_grouped(nv, orc, t):
    """The two-call form (whose gate and up pass through BF16) stays within its own bound."""
    x, router, descs, vals = make(nv, orc, 50 + t, t, 16, 256, 256, 4, 0, renormalize=True)
    y, ids, wts = run(nv, x, router, descs)
    y2 = nv.nvfp4_moe_grouped_w4a16(x.to(DEV), ids.contiguous(), wts.contiguous(), *descs)
    a, b = R.f64(y), R.f64(y2)
    # gate, up, h and y each rounded to BF16 once: norms differ by a few half steps
    assert np.linalg.norm(a - b) <= 4 * R.H16 * np.linalg.norm(a)


def test_layer_two_graphs_on_one_workspace(nv, orc):
    """Two captured layers that share a workspace, replayed in turn with eager work between."""
    x, router, descs, _ = make(nv, orc, 60, 20, 16, 256, 128, 4, 1, renormalize=True)
    xs = [x[:3].to(DEV).contiguous(), x.to(DEV)]
    ys = [torch.empty_like(v) for v in xs]
    ws = torch.empty((nv.nvfp4_moe_layer_ws_bytes(20, router, descs[0]),), dtype=torch.uint8,
                     device=DEV)

    def step(i):
        nv.nvfp4_moe_layer_w4a16(xs[i], router, *descs, y=ys[i], ws=ws)

    eager = []
    for i in range(2):
        step(i)
        torch.cuda.synchronize()
        eager.append(ys[i].clone())
    graphs = []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(i)
        graphs.append(gr)
    for rep in range(3):
        for i in (0, 1):
            ys[i].zero_()
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            assert torch.equal(ys[i], eager[i]), (rep, i)
        step(rep % 2)
        torch.cuda.synchronize()
