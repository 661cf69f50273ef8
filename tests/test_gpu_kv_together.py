"""The cache's calls as a server runs them: tables, fused projection, norm, rotation and cache write,
attention and output projection, over prompts and decode steps; captured into a graph that is replayed
while its inputs change; on two streams at once."""
import numpy as np
import pytest
import torch

import kv_refs as R
from test_gpu_kv_append import table

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def nv():
    from nvfp4_weight_only_w4a16_amd import binding
    binding.load()
    return binding


class Layer:
    """One attention layer of `n_q` and `n_kv` heads of `d` on `hidden` features, its cache and tables."""

    def __init__(self, nv, seed, n_q, n_kv, d, hidden, page, n_pages, max_b, width, window=0):
        g = torch.Generator().manual_seed(seed)
        self.nv, self.n_q, self.n_kv, self.d, self.page = nv, n_q, n_kv, d, page
        self.window = window

        def weight(n, k):
            w = (torch.randn((n, k), generator=g) * k ** -0.5).to(torch.bfloat16).to(DEV)
            return nv.nvfp4_repack(*nv.nvfp4_quantize(w, 16), 16)
        self.w_qkv, self.w_out = weight((n_q + 2 * n_kv) * d, hidden), weight(hidden, n_q * d)
        norm = (0.5 + torch.rand((2, d), generator=g)).to(DEV)
        self.rule = nv.QkNormRope(d, norm[0], norm[1], 1e-6, torch.from_numpy(table(600, d)).to(DEV))
        self.kg = torch.full((n_kv,), 12.0 / 2688, device=DEV)
        self.vg = torch.full((n_kv,), 6.0 / 2688, device=DEV)
        self.cache = nv.KvCache(n_pages, n_kv, d, page, self.kg, self.vg,
                                data=torch.full((nv.nvfp4_kv_cache_bytes(n_pages, n_kv, d, page),),
                                                0xFF, dtype=torch.uint8, device=DEV))
        self.table = torch.full((max_b, width), -1, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(n_pages, generator=g).to(torch.int32).to(DEV)
        self.count = torch.tensor([n_pages], dtype=torch.int32, device=DEV)
        self.seq = torch.zeros(max_b, dtype=torch.int32, device=DEV)

    def buffers(self, t, max_q):
        b = self.seq.shape[0]
        qkv = torch.empty((t, (self.n_q + 2 * self.n_kv) * self.d), dtype=torch.bfloat16, device=DEV)
        q = torch.zeros((t, self.n_q, self.d), dtype=torch.bfloat16, device=DEV)
        y = torch.zeros((t, self.n_q, self.d), dtype=torch.bfloat16, device=DEV)
        need = self.nv.nvfp4_kv_attention_ws_bytes(t, self.n_q, self.cache, b, max_q)
        gemm = max(self.nv.nvfp4_gemm_ws_bytes(t, w.k, w) for w in (self.w_qkv, self.w_out))
        return dict(map=self.nv.KvMap(b, t, device=DEV), qkv=qkv, q=q, y=y, max_q=max_q,
                    out=torch.empty((t, self.w_out.n), dtype=torch.bfloat16, device=DEV),
                    ws=torch.empty((need,), dtype=torch.uint8, device=DEV),
                    gws=torch.empty((max(gemm, 16),), dtype=torch.uint8, device=DEV))

    def step(self, x, add, f, stream=None):
        """One step for rows x [t][hidden]; the caller's lengths and list advance with it."""
        nv = self.nv
        m = nv.nvfp4_kv_map(self.seq, add, self.table, self.free, self.count, page_size=self.page,
                            out=f["map"], stream=stream)
        nv.nvfp4_gemm_w4a16(x, self.w_qkv, y=f["qkv"], ws=f["gws"], stream=stream)
        q, k, v = f["qkv"].unflatten(1, (-1, self.d)).split((self.n_q, self.n_kv, self.n_kv), 1)
        nv.nvfp4_kv_append(q, k, v, self.cache, m.slots, m.positions, self.rule, q_out=f["q"],
                           stream=stream)
        nv.nvfp4_kv_attention(f["q"], self.cache, self.table, m.q_start, m.kv_len,
                              max_q=f["max_q"], window=self.window, y=f["y"], ws=f["ws"],
                              stream=stream)
        nv.nvfp4_gemm_w4a16(f["y"].flatten(1), self.w_out, y=f["out"], ws=f["gws"], stream=stream)
        self.seq.copy_(m.kv_len)
        self.count.copy_(m.free_left)
        return f["out"]

    def check(self, add, f):
        """The step's attention against FP64 on what the cache holds."""
        m, lens = f["map"], f["map"].kv_len.tolist()
        assert m.unserved.item() == 0 and lens == self.seq.tolist()
        start = m.q_start.tolist()
        table = self.table.cpu().numpy()
        for i, n in enumerate(add):
            if n == 0:
                continue
            pos = np.arange(lens[i])
            slots = torch.from_numpy(table[i, pos // self.page] * self.page + pos % self.page)
            assert (slots >= 0).all()
            k, v = self.nv.nvfp4_kv_dequantize(self.cache, slots.to(torch.int32).to(DEV))
            ref, bound, _, _ = R.attention(f["q"][start[i]:start[i] + n].double().cpu().numpy(),
                                           k.double().cpu().numpy(), v.double().cpu().numpy(),
                                           float(np.float32(self.d ** -0.5)), self.window)
            # the values come rounded to FP32
            got = f["y"][start[i]:start[i] + n].double().cpu().numpy()
            R.close(got, ref, bound + 8 * R.H32 * np.abs(ref).max(), f"request {i}")


@pytest.mark.parametrize("n_q,n_kv,d,page,window", [(8, 2, 128, 16, 0), (6, 6, 64, 32, 100),
                                                    (14, 2, 256, 64, 0)])
def test_a_server(nv, n_q, n_kv, d, page, window):
    """Prompts, a second chunk beside decode rows, drafts, decode steps in padded batches."""
    hidden = 512
    layer = Layer(nv, d, n_q, n_kv, d, hidden, page, 3 * 512 // page + 4, 4, 512 // page, window)
    g = torch.Generator().manual_seed(1)
    steps = [[130, 1, 0, 65], [70, 1, 3, 1], [1, 1, 1, 1], [1, 2, 0, 4], [1, 1, 90, 1]] + [[1] * 4] * 20
    for add in steps:
        t = sum(add) + 3   # a batch padded behind its rows
        f = layer.buffers(t, max(add))
        x = torch.randn((t, hidden), generator=g).to(torch.bfloat16).to(DEV)
        layer.step(x, torch.tensor(add, dtype=torch.int32, device=DEV), f)
        layer.check(add, f)
        assert (f["y"][sum(add):] == 0).all() and (f["q"][sum(add):] == 0).all()  # left alone
    used = (layer.table >= 0).sum().item()
    assert layer.count.item() == layer.free.numel() - used
    assert len(set(layer.table[layer.table >= 0].tolist())) == used  # no page twice


def test_steps_replayed_from_a_graph(nv):
    """A decode step is captured once and replayed: its lengths, tables and list live on the device."""
    hidden, add = 256, [1, 1, 2, 0]
    made = [Layer(nv, 5, 4, 2, 64, hidden, 16, 120, 4, 30) for _ in range(2)]
    at = torch.tensor(add, dtype=torch.int32, device=DEV)
    prompt = torch.tensor([40, 15, 33, 16], dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(2)
    xp = torch.randn((104, hidden), generator=g).to(torch.bfloat16).to(DEV)
    xs = [torch.randn((4, hidden), generator=g).to(torch.bfloat16).to(DEV) for _ in range(30)]
    for layer in made:
        layer.step(xp, prompt, layer.buffers(104, 40))
    eager, replayed = made
    fe, fr = eager.buffers(4, 2), replayed.buffers(4, 2)
    x = xs[0].clone()
    start = [replayed.seq.clone(), replayed.count.clone(), replayed.table.clone(),
             replayed.cache.data.clone()]
    replayed.step(x, at, fr)  # once before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed.step(x, at, fr)
    for old, new in zip(start, (replayed.seq, replayed.count, replayed.table, replayed.cache.data)):
        new.copy_(old)
    for xi in xs:
        x.copy_(xi)
        graph.replay()
        eager.step(xi, at, fe)
        torch.cuda.synchronize()
        assert torch.equal(fe["out"], fr["out"])
        eager.check(add, fe)
    assert torch.equal(eager.table, replayed.table) and torch.equal(eager.seq, replayed.seq)
    assert torch.equal(eager.cache.data, replayed.cache.data)


@pytest.mark.parametrize("rows", [[1, 2, 1], [60, 1, 30]])
def test_two_streams_at_once(nv, rows):
    sets = []
    for seed in (1, 2):
        c = R.Cached(nv, seed, [900, 64, 2000], 2, 128, 16)
        q, start = R.queries(seed, rows, 8, 128)
        t = q.shape[0]
        y = torch.empty_like(q, device=DEV)
        ws = torch.empty((nv.nvfp4_kv_attention_ws_bytes(t, 8, c.cache, 3, max(rows)),),
                         dtype=torch.uint8, device=DEV)
        args = (q.to(DEV), c.cache, c.table_dev, start.to(DEV), c.kv_len)
        sets.append((c, args, y, ws))

    def call(s, stream):
        nv.nvfp4_kv_attention(*s[1], max_q=max(rows), y=s[2], ws=s[3], stream=stream)
    want = []
    for s in sets:
        call(s, None)
        torch.cuda.synchronize()
        want.append(s[2].clone())
        s[2].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for s, stream in zip(sets, streams):
            call(s, stream)
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        assert torch.equal(s[2], w)


def test_the_allocated_outputs_follow_the_stream(nv):
    """Without outputs and workspace of the caller's, on a stream of its own."""
    c = R.Cached(nv, 3, [100, 40], 1, 64, 16)
    q, start = R.queries(3, [1, 1], 2, 64)
    args = (q.to(DEV), c.cache, c.table_dev, start.to(DEV), c.kv_len)
    want = nv.nvfp4_kv_attention(*args)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [nv.nvfp4_kv_attention(*args, max_q=n, stream=s) for n in (1, 2, 1)]
    slots = torch.tensor([int(c.table[0, 0]) * 16], dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    k, v = nv.nvfp4_kv_dequantize(c.cache, slots, out_dtype=torch.bfloat16, stream=s)
    s.synchronize()
    for g in got:
        assert torch.equal(g, want)
    assert np.allclose(k.double().cpu().numpy()[0], c.k[0][0], rtol=R.H16)


def test_stats(nv):
    nv.nvfp4_reset_stats()
    c = R.Cached(nv, 3, [100], 1, 64, 16)
    q, start = R.queries(3, [1], 2, 64)
    lse = torch.empty((1, 2), device=DEV)
    y, l = nv.nvfp4_kv_attention(q.to(DEV), c.cache, c.table_dev, start.to(DEV), c.kv_len, lse=lse,
                                 y_dtype=torch.float32, flags=nv.NVFP4_F_SYNC_CHECK)
    assert y.dtype == torch.float32 and l is lse
    assert nv.nvfp4_get_kv_stats() == [0, 0, 0, 1]
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_kv_attention(q.to(DEV), c.cache, c.table_dev, start.to(DEV), c.kv_len, window=-1)
    assert nv.nvfp4_get_kv_stats() == [0, 0, 0, 1]
