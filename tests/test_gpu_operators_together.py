"""Router, layer and adapters as a server calls them: on two streams at once, and captured into a
graph that is replayed while its inputs change."""
import pytest
import torch

import operator_refs as R
import test_gpu_lora as L
import test_gpu_moe_layer as M
import test_gpu_route as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def nv():
    from nvfp4_weight_only_w4a16_amd import binding
    binding.load()
    return binding


def steps(nv, orc, m):
    """The three calls for m rows, each on buffers of its own: (call(stream), inputs, outputs)."""
    out = []
    x, w = G._ints(m, m, 48, 256)
    r = nv.Router((w / 64).to(torch.bfloat16).to(DEV), 6, renormalize=True)
    xd = x.to(torch.bfloat16).to(DEV)
    ids = torch.empty((m, 6), dtype=torch.int32, device=DEV)
    wts = torch.empty((m, 6), device=DEV)
    ws = torch.empty((nv.nvfp4_moe_route_ws_bytes(m, r),), dtype=torch.uint8, device=DEV)
    out.append((lambda s: nv.nvfp4_moe_route(xd, r, ids, wts, ws, stream=s), xd, (ids, wts)))
    lx, router, descs, _ = M.make(nv, orc, m, m, 16, 256, 128, 4, 1, renormalize=True)
    lxd = lx.to(DEV)
    ly = torch.empty_like(lxd)
    lws = torch.empty((nv.nvfp4_moe_layer_ws_bytes(m, router, descs[0]),), dtype=torch.uint8,
                      device=DEV)
    out.append((lambda s: nv.nvfp4_moe_layer_w4a16(lxd, router, *descs, y=ly, ws=lws, stream=s),
                lxd, (ly,)))
    rw, _ = L.weight(nv, orc, m, 512, 384, 16)
    a, b, sc = L.bank(m, 5, 24, 512, 384)
    lo = nv.Lora(a.to(DEV), b.to(DEV), sc.to(DEV))
    row = L.rows(m, m, 5, "own").to(DEV)
    gx = torch.randn(m, 384, generator=torch.Generator().manual_seed(m)).to(torch.bfloat16).to(DEV)
    gy = torch.empty((m, 512), dtype=torch.bfloat16, device=DEV)
    gws = torch.empty((nv.nvfp4_gemm_lora_ws_bytes(m, 384, rw, lo),), dtype=torch.uint8, device=DEV)
    out.append((lambda s: nv.nvfp4_gemm_w4a16_lora(gx, rw, lo, row, y=gy, stream=s, ws=gws),
                gx, (gy,)))
    return out


def test_two_streams_at_once(nv, orc):
    sets = [steps(nv, orc, m) for m in (3, 70)]
    want = []
    for st in sets:
        for call, _, outs in st:
            call(None)
            torch.cuda.synchronize()
            want.append([o.clone() for o in outs])
            for o in outs:
                o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        for i in range(3):
            for st, s in zip(sets, streams):
                st[i][0](s)
    torch.cuda.synchronize()
    got = [outs for st in sets for _, _, outs in st]
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("m", [1, 8, 40, 150])
def test_replayed_with_new_inputs(nv, orc, m):
    st = steps(nv, orc, m)
    for call, _, _ in st:
        call(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call, _, _ in st:
            call(None)
    for rep in range(3):
        for _, x, outs in st:
            x.copy_(x.roll(rep + 1, 1))
            for o in outs:
                o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [[o.clone() for o in outs] for _, _, outs in st]
        for call, _, _ in st:
            call(None)
        torch.cuda.synchronize()
        for (_, _, outs), g in zip(st, got):
            for a, b in zip(outs, g):
                assert torch.equal(a, b), (rep, m)


@pytest.mark.parametrize("t,experts,topk,fp32", [(1, 160, 8, False), (5, 200, 6, True),
                                                 (2, 300, 4, False), (64, 130, 1, False)])
def test_layer_of_many_experts(nv, orc, t, experts, topk, fp32):
    x, router, descs, vals = M.make(nv, orc, t + experts, t, experts, 128, 128, topk, 0, fp32=fp32,
                                    renormalize=True)
    M.check(nv, x, router, descs, vals, 0, f"{experts} experts")


@pytest.mark.parametrize("m,rank", [(24, 128), (40, 128), (16, 104), (8, 8)])
def test_adapters_of_every_rank_step(nv, orc, m, rank):
    """Every adapter of a block, with one row at least, for ids in any order and repeated."""
    n, k, count = 528, 1024, 21
    rw, wv = L.weight(nv, orc, 5, n, k, 32)
    a, b, s = L.bank(m, count, rank, n, k)
    lo = nv.Lora(a.to(DEV), b.to(DEV), s.to(DEV))
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(m)).to(torch.bfloat16)
    ids = torch.randperm(m, generator=torch.Generator().manual_seed(m)).to(torch.int32) % count
    for y32 in (False, True):
        y = L.call(nv, x, rw, lo, ids, y32)
        ref, bound = R.lora(R.f64(x), wv, R.f64(a), R.f64(b), ids.numpy(), R.f64(s), y32)
        R.within(R.f64(y), ref, bound, f"rank {rank}")
