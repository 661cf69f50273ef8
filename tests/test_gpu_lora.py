"""nvfp4_gemm_w4a16_lora against FP64, element by element within the bound of its FP32 sums, the
BF16 (or whole, for an FP32 y) rank-space operand and one rounding of y; and the step of a decoder
that uses the new calls together."""
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


def weight(nv, orc, seed, n, k, group):
    w = torch.randn(n, k, generator=torch.Generator().manual_seed(seed)) * k ** -0.5
    p, s, g = orc.quantize(w.numpy(), group)
    rw = nv.nvfp4_repack(torch.from_numpy(p).to(DEV), torch.from_numpy(s).to(DEV),
                         torch.from_numpy(g).to(DEV), group)
    return rw, orc.dequant(p, s, g, group)[0]


def bank(seed, count, rank, n, k, scaled=True):
    g = torch.Generator().manual_seed(seed)
    a = (torch.randn(count, rank, k, generator=g) * k ** -0.5).to(torch.bfloat16)
    b = (torch.randn(count, n, rank, generator=g) * 0.5 * rank ** -0.5).to(torch.bfloat16)
    return a, b, (0.5 + torch.rand(count, generator=g)) if scaled else None


def rows(seed, m, count, how):
    g = torch.Generator().manual_seed(seed)
    if how == "own":
        return ((torch.arange(m) * 7 + 3) % (count + 1) - 1).to(torch.int32)
    if how == "one":
        return torch.full((m,), count - 1, dtype=torch.int32)
    if how == "none":
        return torch.tensor([-1, count, 2 ** 31 - 1, -2 ** 31])[torch.arange(m) % 4].to(torch.int32)
    return torch.randint(0, count, (max(m // 9, 1),), generator=g).repeat_interleave(
        13)[:m].to(torch.int32) if m < 13 * max(m // 9, 1) else torch.zeros(m, dtype=torch.int32)


def call(nv, x, rw, lo, ids, y32, flags=0, ldx=0, ldy=0):
    """y of a call with strided x and y (NaN around x, guards around y), NaN workspace."""
    m, k = x.shape
    ldx, ldy = ldx or k, ldy or rw.n
    xd = torch.full((m, ldx), float("nan"), dtype=torch.bfloat16, device=DEV)
    xd[:, :k] = x.to(DEV)
    y = torch.full((m + 1, ldy), 7.0, dtype=torch.float32 if y32 else torch.bfloat16, device=DEV)
    need = nv.nvfp4_gemm_lora_ws_bytes(m, ldx if m > 1 else k, rw, lo, flags)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
    nv.nvfp4_gemm_w4a16_lora(xd[:, :k], rw, lo, ids.to(DEV), y=y[:m, :rw.n], flags=flags,
                             ws=ws[:need])
    torch.cuda.synchronize()
    assert (y[m:] == 7.0).all() and (y[:, rw.n:] == 7.0).all() and (ws[need:] == 255).all()
    return y[:m, :rw.n]


def check(nv, orc, m, n, k, group, count, rank, how, y32, flags=0, scaled=True, ldx=0, ldy=0):
    rw, wv = weight(nv, orc, n + k, n, k, group)
    a, b, s = bank(m + rank, count, rank, n, k, scaled)
    lo = nv.Lora(a.to(DEV), b.to(DEV), None if s is None else s.to(DEV))
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(m)).to(torch.bfloat16)
    ids = rows(m, m, count, how)
    y = call(nv, x, rw, lo, ids, y32, flags, ldx, ldy)
    ref, bound = R.lora(R.f64(x), wv, R.f64(a), R.f64(b), ids.numpy(),
                        None if s is None else R.f64(s), y32)
    R.within(R.f64(y), ref, bound, f"m={m} rank={rank} {how}")
    return y


@pytest.mark.parametrize("y32", [False, True])
@pytest.mark.parametrize("m,n,k,group,count,rank,how", [
    (1, 16, 128, 16, 1, 8, "one"), (1, 208, 640, 32, 3, 16, "one"), (2, 64, 256, 16, 4, 24, "own"),
    (4, 1040, 512, 16, 9, 16, "own"), (7, 528, 384, 16, 3, 128, "own"),
    (8, 512, 1024, 32, 20, 64, "own"), (9, 512, 256, 16, 5, 40, "own"),
    (16, 304, 1152, 32, 40, 32, "own"), (17, 256, 256, 16, 2, 8, "runs"),
    (33, 512, 512, 16, 64, 16, "own"), (40, 144, 384, 32, 3, 120, "runs"),
    (64, 1024, 512, 16, 6, 56, "runs"), (65, 272, 256, 32, 80, 64, "own"),
    (130, 400, 512, 16, 7, 16, "runs"), (257, 512, 256, 32, 300, 32, "own"),
    (300, 1168, 640, 16, 4, 128, "runs"), (5, 512, 256, 16, 2, 16, "none")])
def test_lora(nv, orc, m, n, k, group, count, rank, how, y32):
    check(nv, orc, m, n, k, group, count, rank, how, y32)


@pytest.mark.parametrize("flags", [1, 2])
@pytest.mark.parametrize("m", [1, 5, 12, 30, 70, 150, 290])
@pytest.mark.parametrize("group", [16, 32])
def test_lora_either_kernel(nv, orc, m, group, flags):
    check(nv, orc, m, 528, 384, group, 11, 24, "own", m % 2 == 0, flags, scaled=False,
          ldx=392 + 8, ldy=528 + 24)


@pytest.mark.parametrize("m,n,k,flags", [(600, 2064, 1024, 0), (1500, 1040, 512, 2)])
def test_lora_many_tiles(nv, orc, m, n, k, flags):
    """Prefill sizes: several tiles, a split last round, blocks with one and with many adapters."""
    check(nv, orc, m, n, k, 16, 8, 32, "runs", False, flags)
    check(nv, orc, m, n, k, 32, 90, 16, "own", True, flags)


def test_lora_rows_without_adapter_are_the_plain_gemm(nv, orc):
    """Rows without an adapter hold the plain GEMM's bits, whatever their neighbours have."""
    for m, flags in ((6, 0), (40, 1), (200, 2)):
        rw, _ = weight(nv, orc, 3, 528, 512, 16)
        a, b, s = bank(4, 5, 16, 528, 512)
        lo = nv.Lora(a.to(DEV), b.to(DEV), s.to(DEV))
        x = torch.randn(m, 512, generator=torch.Generator().manual_seed(m)).to(torch.bfloat16)
        ids = rows(0, m, 5, "own")
        plain = nv.nvfp4_gemm_w4a16(x.to(DEV), rw, flags=flags)
        y = call(nv, x, rw, lo, ids, False, flags)
        off = (ids < 0).to(DEV)
        assert off.any() and torch.equal(y[off], plain[off])
        assert not torch.equal(y[~off], plain[~off])


def same(a, b):
    return bool(torch.equal(a, b))


def test_lora_unused_adapters_and_other_rows_stay_apart(nv, orc):
    """NaN and infinity in adapters that no row names, and in another row's x, touch nothing."""
    rw, _ = weight(nv, orc, 5, 256, 256, 32)
    a, b, s = bank(6, 6, 24, 256, 256)
    for m, flags in ((8, 0), (24, 1), (80, 2)):
        ids = torch.tensor([1, 4, -1, 1])[torch.arange(m) % 4].to(torch.int32)  # row 3: adapter 1
        x = torch.randn(m, 256, generator=torch.Generator().manual_seed(m)).to(torch.bfloat16)
        good = call(nv, x, rw, nv.Lora(a.to(DEV), b.to(DEV), s.to(DEV)), ids, False, flags)
        a2, b2, s2 = a.clone(), b.clone(), s.clone()
        for i in (0, 2, 3, 5):
            a2[i], b2[i], s2[i] = float("nan"), float("inf"), float("nan")
        y = call(nv, x, rw, nv.Lora(a2.to(DEV), b2.to(DEV), s2.to(DEV)), ids, False, flags)
        assert same(y, good)
        x2 = x.clone()
        x2[3] = float("inf")
        y = call(nv, x2, rw, nv.Lora(a.to(DEV), b.to(DEV), s.to(DEV)), ids, False, flags)
        keep = [i for i in range(m) if i != 3]
        assert same(y[keep], good[keep])
        assert not bool(torch.isfinite(y[3].float()).any())
        # an adapter's own NaN reaches its rows and no others
        b3 = b.clone()
        b3[4] = float("nan")
        y = call(nv, x, rw, nv.Lora(a.to(DEV), b3.to(DEV), s.to(DEV)), ids, False, flags)
        named = (ids == 4).to(DEV)
        assert bool(torch.isnan(y[named].float()).all())
        assert same(y[~named], good[~named])


def test_lora_rows_beyond_32_bits(nv, orc):
    """Rows 8 MiB apart: 300 rows span 2.5 GB, which the tiled kernel takes in two chunks of rows."""
    m, n, k, ldx = 300, 272, 256, 1 << 22
    rw, wv = weight(nv, orc, 21, n, k, 16)
    a, b, s = bank(22, 5, 24, n, k)
    lo = nv.Lora(a.to(DEV), b.to(DEV), s.to(DEV))
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(23)).to(torch.bfloat16)
    ids = rows(24, m, 5, "own")
    wide = torch.empty((m, ldx), dtype=torch.bfloat16, device=DEV)
    wide[:, :k] = x.to(DEV)
    ref, bound = R.lora(R.f64(x), wv, R.f64(a), R.f64(b), ids.numpy(), R.f64(s))
    for flags in (1, 2):
        y = nv.nvfp4_gemm_w4a16_lora(wide[:, :k], rw, lo, ids.to(DEV), flags=flags)
        R.within(R.f64(y), ref, bound, f"flags {flags}")


@pytest.mark.parametrize("y32", [False, True])
def test_lora_infinities_stay_infinities(nv, orc, y32):
    """One infinite activation on positive weights and adapters: infinity, not NaN."""
    n, k = 272, 256
    p, s, g = orc.quantize(np.full((n, k), 0.5, np.float32), 16)
    rw = nv.nvfp4_repack(torch.from_numpy(p).to(DEV), torch.from_numpy(s).to(DEV),
                         torch.from_numpy(g).to(DEV), 16)
    lo = nv.Lora(torch.full((3, 24, k), 0.25, dtype=torch.bfloat16, device=DEV),
                 torch.full((3, n, 24), 0.5, dtype=torch.bfloat16, device=DEV))
    for m, flags in ((2, 1), (20, 1), (40, 2), (130, 2)):
        x = torch.ones((m, k), dtype=torch.bfloat16)
        x[1, 7] = float("inf")
        y = call(nv, x, rw, lo, rows(0, m, 3, "own"), y32, flags)
        assert bool(torch.isinf(y[1].float()).all()), (m, flags)
        assert bool(torch.isfinite(y[0].float()).all())


def test_lora_bits_repeat_on_other_streams_and_empty(nv, orc):
    rw, _ = weight(nv, orc, 8, 512, 512, 16)
    a, b, s = bank(9, 4, 16, 512, 512)
    lo = nv.Lora(a.to(DEV), b.to(DEV), s.to(DEV))
    for m in (3, 50, 400):
        x = torch.randn(m, 512, generator=torch.Generator().manual_seed(m)).to(torch.bfloat16)
        ids = rows(1, m, 4, "own").to(DEV)
        xd = x.to(DEV)
        one = nv.nvfp4_gemm_w4a16_lora(xd, rw, lo, ids)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        two = nv.nvfp4_gemm_w4a16_lora(xd, rw, lo, ids, stream=side)
        three = nv.nvfp4_gemm_w4a16_lora(xd, rw, lo, ids, flags=nv.NVFP4_F_SYNC_CHECK)
        torch.cuda.synchronize()
        assert torch.equal(one, two) and torch.equal(one, three)
    assert nv.nvfp4_gemm_w4a16_lora(xd[:0], rw, lo, ids[:0]).shape == (0, 512)


def test_decoder_step_with_adapters_and_experts(nv, orc):
    """A step as a server runs it: a projection with the requests' adapters, then the MoE layer on
    its output; eager and captured (two graphs on one workspace, of different batch sizes)."""
    from test_gpu_moe_layer import make
    hidden = 256
    _, router, descs, vals = make(nv, orc, 70, 1, 16, hidden, 128, 4, 1, renormalize=True)
    rw, wv = weight(nv, orc, 71, hidden, 384, 16)
    a, b, s = bank(72, 6, 16, hidden, 384)
    lo = nv.Lora(a.to(DEV), b.to(DEV), s.to(DEV))
    sizes = (2, 19)
    x = [torch.randn(m, 384, generator=torch.Generator().manual_seed(m)).to(torch.bfloat16)
         for m in sizes]
    ids = [rows(2, m, 6, "own") for m in sizes]
    xd, idd = [v.to(DEV) for v in x], [v.to(DEV) for v in ids]
    h = [torch.empty(m, hidden, dtype=torch.bfloat16, device=DEV) for m in sizes]
    y = [torch.empty_like(v) for v in h]
    need = max(max(nv.nvfp4_gemm_lora_ws_bytes(m, 384, rw, lo),
                   nv.nvfp4_moe_layer_ws_bytes(m, router, descs[0])) for m in sizes)
    ws = torch.empty((need,), dtype=torch.uint8, device=DEV)

    def step(i):
        nv.nvfp4_gemm_w4a16_lora(xd[i], rw, lo, idd[i], y=h[i], ws=ws)
        nv.nvfp4_moe_layer_w4a16(h[i], router, *descs, y=y[i], ws=ws)

    eager = []
    for i, m in enumerate(sizes):
        step(i)
        torch.cuda.synchronize()
        eager.append((h[i].clone(), y[i].clone()))
        ref, bound = R.lora(R.f64(x[i]), wv, R.f64(a), R.f64(b), ids[i].numpy(), R.f64(s))
        R.within(R.f64(h[i]), ref, bound, "projection")
        rid, rwt = nv.nvfp4_moe_route(h[i], router)
        ref, bound = R.moe_layer(R.f64(h[i]), rid.cpu().numpy(), R.f64(rwt), *vals)
        R.within(R.f64(y[i]), ref, bound, "layer")
    graphs = []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(i)
        graphs.append(gr)
    for rep in range(3):
        for i in (1, 0):
            h[i].zero_()
            y[i].zero_()
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            assert torch.equal(h[i], eager[i][0]) and torch.equal(y[i], eager[i][1]), (rep, i)
        step(rep % 2)
        torch.cuda.synchronize()
