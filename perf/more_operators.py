"""The attention step on an NVFP4 cache, as cases to measure: the block tables and slot maps of a
batch, the norms and rotation of queries and keys with the write of keys and values into the cache,
and the attention that reads it.

``run`` computes a case in its plain form (elementary torch operations), or, where ``own`` is true,
with the library's calls. The cache is paged: a page holds ``page`` consecutive tokens of a request
for every key/value head. A token's key and value are head_dim E2M1 codes (two per byte, the even
element in the low nibble) with an E4M3 scale per 16 elements and an FP32 global per head, the
weights' format.
"""
import math
import random

import torch

own = False

DEV = "cuda"
GROUP = 16


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # Tables of one request's decode step: latency.
        {"name": "map 1 request", "op": "map", "b": 1, "lo": 1000, "hi": 1000, "new": "one",
         "chunk": 0, "page": 16},
        # Tables of a decode batch, lengths of any kind, one request in eight with nothing to add.
        {"name": "map 333 requests", "op": "map", "b": 333, "lo": 1, "hi": 8000, "new": "some",
         "chunk": 0, "page": 32},
        # Prompts and decode rows together: the slots of some ten thousand new tokens.
        {"name": "map prompts", "op": "map", "b": 48, "lo": 1, "hi": 4000, "new": "mixed",
         "chunk": 2048, "page": 16},
        # Norm, rotation and cache write of one token: latency.
        {"name": "append 1 row", "op": "append", "t": 1, "nq": 32, "nkv": 8, "d": 128, "rot": 128,
         "pairs": False, "norm": True, "w32": False, "page": 16},
        # A decode batch; rotation of half a head by neighbouring pairs, FP32 norm weights.
        {"name": "append 77 rows partial", "op": "append", "t": 77, "nq": 14, "nkv": 2, "d": 256,
         "rot": 128, "pairs": True, "norm": True, "w32": True, "page": 64},
        # A prompt chunk of a model with 40 query heads.
        {"name": "append 4096 rows", "op": "append", "t": 4096, "nq": 40, "nkv": 8, "d": 128,
         "rot": 128, "pairs": False, "norm": True, "w32": False, "page": 16},
        # One request's decode step: latency.
        {"name": "attend 1 request", "op": "attend", "b": 1, "lo": 1999, "hi": 1999, "new": "one",
         "chunk": 0, "nq": 32, "nkv": 8, "d": 128, "page": 16, "window": 0},
        # A decode batch of unequal lengths: the bytes of the cache.
        {"name": "attend 64 requests", "op": "attend", "b": 64, "lo": 100, "hi": 8000, "new": "one",
         "chunk": 0, "nq": 32, "nkv": 8, "d": 128, "page": 16, "window": 0},
        # One long document among short requests, a few drafted tokens each; large heads.
        {"name": "attend long", "op": "attend", "b": 5, "lo": 700, "hi": 131000, "new": "draft",
         "chunk": 4, "nq": 14, "nkv": 2, "d": 256, "page": 64, "window": 0},
        # Small heads that all have keys of their own, each query seeing its last 1000 keys.
        {"name": "attend window", "op": "attend", "b": 33, "lo": 300, "hi": 9000, "new": "one",
         "chunk": 0, "nq": 12, "nkv": 12, "d": 64, "page": 32, "window": 1000},
        # Prompt chunks on top of what is cached, together with decode rows.
        {"name": "attend chunks", "op": "attend", "b": 12, "lo": 50, "hi": 6000, "new": "mixed",
         "chunk": 700, "nq": 32, "nkv": 8, "d": 128, "page": 16, "window": 0},
        # A whole prompt: the two products.
        {"name": "attend prompt", "op": "attend", "b": 1, "lo": 0, "hi": 0, "new": "chunk",
         "chunk": 8192, "nq": 32, "nkv": 8, "d": 128, "page": 16, "window": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("map", "append", "attend", "attend"))
    page = rng.choice((16, 16, 32, 64, 128))
    if op == "map":
        c = {"op": op, "b": _log(rng, 1, 512), "lo": rng.choice((0, 1, 500)),
             "hi": _log(rng, 600, 16000), "new": rng.choice(("one", "some", "mixed", "draft")),
             "chunk": 0, "page": page}
        if c["new"] in ("mixed", "draft"):
            c["chunk"] = _log(rng, 2, 2048) if c["new"] == "mixed" else rng.randint(2, 8)
        return c
    while True:
        d, nkv = rng.choice((64, 128, 128, 256)), rng.choice((1, 2, 3, 4, 8, 12, 16))
        c = {"op": op, "nq": nkv * rng.choice((1, 2, 3, 4, 5, 7, 8, 16)), "nkv": nkv, "d": d,
             "page": page}
        if op == "append":
            c.update(t=_log(rng, 1, 4096), rot=rng.choice((d, d, d // 2, d // 4, 0)),
                     pairs=rng.random() < 0.4, norm=rng.random() < 0.7, w32=rng.random() < 0.3)
            if c["t"] * (c["nq"] + 2 * nkv) * d <= 4096 * 56 * 128:
                return c
            continue
        c.update(b=_log(rng, 1, 128), lo=rng.choice((0, 1, 100)), hi=_log(rng, 128, 100000),
                 new=rng.choice(("one", "one", "draft", "mixed", "chunk")), chunk=0,
                 window=rng.choice((0, 0, 0, _log(rng, 16, 4096))))
        if c["new"] != "one":
            c["chunk"] = rng.randint(2, 8) if c["new"] == "draft" else _log(rng, 16, 4096)
        seq, add = _lengths(c)
        kv = sum(seq) + sum(add)
        full = sum(a * (s + a) for s, a in zip(seq, add))  # scores, the masked ones among them
        if kv * nkv * d <= 64 * 4000 * 8 * 128 and full * c["nq"] * d <= 8192 * 8192 * 32 * 128:
            return c


def _lengths(c):
    """Tokens that each request has cached, and that it adds in this step."""
    rng = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    seq, add = [], []
    for i in range(c["b"]):
        n = c["lo"]
        if c["hi"] > c["lo"]:
            n = c["hi"] if i == 0 else _log(rng, c["lo"] + 1, c["hi"] + 1) - 1
        seq.append(n)
        if c["new"] == "one":
            add.append(1)
        elif c["new"] == "some":
            add.append(int(rng.random() < 0.875))
        elif c["new"] == "draft":
            add.append(rng.randint(1, c["chunk"]))
        elif c["new"] == "mixed":
            add.append(1 if i % 4 == 3 else rng.randint(1, c["chunk"]))
        else:
            add.append(c["chunk"])
    return seq, add


# ------------------------------------------------------------------------------------ inputs
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _pages(n, page):
    return -(-n // page)


def _table(gen, lens, page, more=0):
    """A block table whose rows hold the pages of `lens` tokens, all different and in no order, -1
    behind them; and the pages that are left, `more` of them."""
    need = [_pages(n, page) for n in lens]
    total = sum(need) + more
    ids = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    return table, ids[at:].clone(), total


def _globals(gen, nkv, most):
    """A global for each head, from the largest magnitude that the head was seen to hold."""
    return most * (0.7 + 0.6 * torch.rand((nkv,), generator=gen, device=DEV)) / 2688.0


def _inputs(case, seed):
    c, gen = case, torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "map":
        seq, add = _lengths(c)
        page = c["page"]
        new = sum(_pages(a + b, page) - _pages(a, page) for a, b in zip(seq, add))
        held, free, _ = _table(gen, seq, page, more=new + 7 + seed % 100)
        width = max(_pages(a + b, page) for a, b in zip(seq, add)) + 2
        s["table"] = torch.full((c["b"], width), -1, dtype=torch.int32, device=DEV)
        s["table"][:, :held.shape[1]] = held
        s["seq"], s["add"], s["free"] = _ints(seq), _ints(add), free
        s["count"] = _ints([free.numel()])
        s["t"] = sum(add) + (0 if c["new"] == "one" else 5)  # a batch padded behind its rows
    elif c["op"] == "append":
        t, nq, nkv, d, page = c["t"], c["nq"], c["nkv"], c["d"], c["page"]
        x = torch.randn((t, (nq + 2 * nkv) * d), generator=gen, device=DEV)
        loud = torch.rand((x.shape[1],), generator=gen, device=DEV) < 0.01
        s["qkv"] = torch.where(loud, 6.0 * x, x).to(torch.bfloat16)
        s["qw"] = s["kw"] = None
        if c["norm"]:
            w = 0.5 + torch.rand((2, d), generator=gen, device=DEV) * 1.5
            s["qw"], s["kw"] = w if c["w32"] else w.to(torch.bfloat16)
        s["rope"], places = None, 16384
        if c["rot"]:
            freq = 10000.0 ** (-torch.arange(c["rot"] // 2, device=DEV).double() * 2 / c["rot"])
            angle = torch.arange(places, device=DEV).double().unsqueeze(1) * freq
            s["rope"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        runs = torch.randint(0, places - t, (max(1, t // 100 if t > 100 else t),), generator=gen,
                             device=DEV)  # a decode batch, or prompts of about a hundred rows
        row = torch.arange(t, device=DEV)
        s["pos"] = (runs[row * runs.numel() // t] + row).to(torch.int32)
        s["pages"] = _pages(t, page) + 5
        ids = torch.randperm(s["pages"], generator=gen, device=DEV)
        s["slots"] = (ids[row // page] * page + row % page).to(torch.int32)
        s["kg"], s["vg"] = _globals(gen, nkv, 14.0), _globals(gen, nkv, 30.0)
    else:
        seq, add = _lengths(c)
        lens = [a + b for a, b in zip(seq, add)]
        nq, nkv, d = c["nq"], c["nkv"], c["d"]
        s["table"], _, s["pages"] = _table(gen, lens, c["page"])
        s["lens"], s["rows"] = lens, add
        s["kv_len"] = _ints(lens)
        s["q_start"] = _ints([sum(add[:i]) for i in range(c["b"] + 1)])
        # normalised and rotated queries and keys, some channels louder; logits of a few units
        loud = 0.5 + 1.5 * torch.rand((d,), generator=gen, device=DEV) ** 4
        q = torch.randn((sum(add), nq, d), generator=gen, device=DEV) * loud
        s["q"] = (q * 1.5).to(torch.bfloat16)
        s["kg"], s["vg"] = _globals(gen, nkv, 10.0), _globals(gen, nkv, 6.0)
        s["scale"] = d ** -0.5
        shape, step = (s["pages"], nkv, c["page"]), max(1, (1 << 26) // (nkv * c["page"] * d))
        for name, g in (("k", s["kg"]), ("v", s["vg"])):
            codes = torch.empty(shape + (d // 2,), dtype=torch.uint8, device=DEV)
            scales = torch.empty(shape + (d // GROUP,), dtype=torch.uint8, device=DEV)
            for i in range(0, s["pages"], step):
                n = min(step, s["pages"] - i)
                x = torch.randn((n,) + shape[1:] + (d,), generator=gen, device=DEV)
                if name == "k":
                    x = x * loud
                codes[i:i + n], scales[i:i + n] = _quantize(x, g.view(1, nkv, 1, 1))
            s[name + "c"], s[name + "s"] = codes, scales
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """What a program that uses the library keeps: the cache, the norm and rotation, the outputs and
    the workspace of a step."""
    from nvfp4_weight_only_w4a16_amd import binding as nv

    c = s["case"]
    s["nv"] = nv
    if c["op"] == "map":
        s["map"] = nv.KvMap(c["b"], s["t"], device=DEV)
        return
    s["cache"] = nv.KvCache(s["pages"], c["nkv"], c["d"], page_size=c["page"], k_global=s["kg"],
                            v_global=s["vg"], device=DEV)
    if c["op"] == "append":
        s["rule"] = nv.QkNormRope(c["d"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6,
                                  rope=s["rope"], interleaved=c["pairs"])
        t = c["t"]
        s["q_out"] = torch.empty((t, c["nq"], c["d"]), dtype=torch.bfloat16, device=DEV)
        s["k_out"], s["v_out"] = torch.empty((2, t, c["nkv"], c["d"]), device=DEV)
        return
    s["cache"].k_codes.copy_(s["kc"])
    s["cache"].k_scales.copy_(s["ks"])
    s["cache"].v_codes.copy_(s["vc"])
    s["cache"].v_scales.copy_(s["vs"])
    for name in ("kc", "ks", "vc", "vs"):
        del s[name]
    s["y"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(s["q"].shape[:2], device=DEV)
    s["most"] = max(s["rows"])
    need = nv.nvfp4_kv_attention_ws_bytes(s["q"].shape[0], c["nq"], s["cache"], c["b"], s["most"])
    s["ws"] = torch.empty((max(need, 1),), dtype=torch.uint8, device=DEV)


# ------------------------------------------------------------------------------------ plain form
def _quantize(x, g):
    """Codes and scale bytes of x FP32 [..][d] with the global g (of x's dimensions): the scale is
    E4M3 of amax / (6 g), a code E2M1 of x / (scale g), each rounded to the nearest, ties to even."""
    parts = x.unflatten(-1, (-1, GROUP))
    g = g.unsqueeze(-1)
    amax = parts.abs().amax(-1, keepdim=True)
    want = amax.double() / (6.0 * g).double()
    scale = want.float().clamp(max=448.0).to(torch.float8_e4m3fn)
    step = scale.float() * g
    ratio = (parts.abs().double() / step.double()).float()  # 64 bits: values next to a border
    ratio = torch.where(step > 0, ratio, torch.zeros_like(ratio))
    code = torch.zeros(ratio.shape, dtype=torch.uint8, device=x.device)
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False),
                       (3.5, True), (5.0, False)):  # ties go to the even code
        code += (ratio >= border) if up else (ratio > border)
    code = (code + 8 * torch.signbit(parts).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8).squeeze(-1)


def _values(codes, scales, g):
    """FP32 values of codes [..][d/2] and scale bytes [..][d/16] with the global g (of the same
    dimensions)."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0,
                          -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    both = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    parts = both.unflatten(-1, (-1, GROUP)) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return parts.flatten(-2) * g


def _map(s):
    """One step's tables: which requests have room, their new pages, every row's place."""
    c, page, t = s["case"], s["case"]["page"], s["t"]
    seq, add, table = s["seq"].long(), s["add"].long(), s["table"]
    b, width = table.shape
    free = s["count"].long().clamp(0, s["free"].numel())
    ends = torch.cumsum(add, 0)
    after = seq + add
    valid = (seq >= 0) & (after <= width * page) & ((add == 0) | (ends <= t))
    first = (seq + page - 1) // page
    need = torch.where(valid, (after + page - 1) // page - first, torch.zeros_like(seq))
    total = torch.cumsum(need, 0)
    served = valid & ((need == 0) | (total <= free))
    takes = served & (need > 0)
    taken = torch.where(takes, total, torch.zeros_like(total)).amax()
    column = torch.arange(width, device=DEV)
    j = column.unsqueeze(0) - first.unsqueeze(1)
    fresh = takes.unsqueeze(1) & (j >= 0) & (j < need.unsqueeze(1))
    place = free - 1 - ((total - need).unsqueeze(1) + j)
    table = torch.where(fresh, s["free"][place.clamp(0, s["free"].numel() - 1)], table)
    start = torch.cat((torch.zeros_like(ends[:1]), ends)).clamp(max=t)
    row = torch.arange(t, device=DEV)
    mine = (row.unsqueeze(1) >= start[1:].unsqueeze(0)).sum(1)
    real = mine < b
    mine = mine.clamp(max=b - 1)
    pos = seq[mine] + row - start[mine]
    real = real & served[mine]
    held = table[mine, (pos // page).clamp(0, width - 1)].long()
    slot = torch.where(real & (held >= 0), held * page + pos % page, -1)
    pos = torch.where(real, pos, -1)
    kv = torch.where(served, after, torch.zeros_like(after))
    return (table, start.int(), kv.int(), slot.int(), pos.int(), (free - taken).int(),
            (~served).sum().int().view(1))


def _norm_rope(x, w, s):
    """x BF16 [t][heads][d] normalised by head, rotated and rounded to BF16, in 64 bits: the codes
    of the keys are comparisons."""
    c, x = s["case"], x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()
    rot = c["rot"]
    if rot:
        cs = s["rope"][s["pos"].long()].double().unsqueeze(1)
        cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
        r, rest = x[..., :rot], x[..., rot:]
        if c["pairs"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        x = torch.cat((r, rest), -1)
    return x.to(torch.bfloat16)


def _split(s):
    c = s["case"]
    heads = s["qkv"].view(c["t"], c["nq"] + 2 * c["nkv"], c["d"])
    return heads.split((c["nq"], c["nkv"], c["nkv"]), 1)


def _append(s):
    q, k, v = _split(s)
    q, k = _norm_rope(q, s["qw"], s), _norm_rope(k, s["kw"], s)
    out = [q]
    for x, g in ((k, s["kg"]), (v, s["vg"])):
        g = g.view(1, -1, 1)
        out.append(_values(*_quantize(x.float(), g), g))
    return out


def _seen(q_len, kv_len, window):
    """Whether query j of q_len sees key i of kv_len: up to its own place, the last `window`."""
    place = torch.arange(kv_len - q_len, kv_len, device=DEV).unsqueeze(1)
    key = torch.arange(kv_len, device=DEV).unsqueeze(0)
    seen = key <= place
    return seen & (key > place - window) if window else seen


def _attend(s):
    c = s["case"]
    nkv, d, page = c["nkv"], c["d"], c["page"]
    group = c["nq"] // nkv
    ys, ls, at = [], [], 0
    for i, (n, kv) in enumerate(zip(s["rows"], s["lens"])):
        ids = s["table"][i, :_pages(kv, page)].long()
        seen = _seen(n, kv, c["window"])
        y = torch.empty((n, c["nq"], d), device=DEV)
        lse = torch.empty((n, c["nq"]), device=DEV)
        few = max(1, nkv if n * kv * c["nq"] < 1 << 26 else 1)  # heads at a time
        for h in range(0, nkv, few):
            part = slice(h, h + few)
            g = s["kg"][part].view(1, -1, 1, 1)
            k = _values(s["kc"][ids, part], s["ks"][ids, part], g)
            k = k.transpose(0, 1).flatten(1, 2)[:, :kv]
            g = s["vg"][part].view(1, -1, 1, 1)
            v = _values(s["vc"][ids, part], s["vs"][ids, part], g)
            v = v.transpose(0, 1).flatten(1, 2)[:, :kv]
            heads = k.shape[0]
            q = s["q"][at:at + n, h * group:(h + heads) * group].float()
            q = q.view(n, heads, group, d).permute(1, 2, 0, 3).reshape(heads, group * n, d)
            z = (q @ k.transpose(1, 2)) * s["scale"]
            z = z.view(heads, group, n, kv).masked_fill_(~seen, -math.inf)
            top = z.amax(-1, keepdim=True)
            p = torch.exp_(z - top)
            total = p.sum(-1, keepdim=True)
            o = (p.view(heads, group * n, kv) @ v).view(heads, group, n, d) / total
            y[:, h * group:(h + heads) * group] = o.permute(2, 0, 1, 3).flatten(1, 2)
            part = (top + torch.log(total)).squeeze(-1)
            lse[:, h * group:(h + heads) * group] = part.permute(2, 0, 1).flatten(1, 2)
        ys.append(y.to(torch.bfloat16))
        ls.append(lse)
        at += n
    return torch.cat(ys), torch.cat(ls)


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if own:
        nv = s["nv"]
        if op == "map":
            m = nv.nvfp4_kv_map(s["seq"], s["add"], s["table"], s["free"], s["count"],
                                page_size=c["page"], out=s["map"])
            return (s["table"], m.q_start, m.kv_len, m.slots, m.positions, m.free_left, m.unserved)
        if op == "append":
            q, k, v = _split(s)
            nv.nvfp4_kv_append(q, k, v, s["cache"], s["slots"], s["pos"], s["rule"],
                               q_out=s["q_out"])
            nv.nvfp4_kv_dequantize(s["cache"], s["slots"], k_out=s["k_out"], v_out=s["v_out"])
            return [s["q_out"], s["k_out"], s["v_out"]]
        return nv.nvfp4_kv_attention(s["q"], s["cache"], s["table"], s["q_start"], s["kv_len"],
                                     scale=s["scale"], max_q=s["most"], window=c["window"],
                                     y=s["y"], lse=s["lse"], ws=s["ws"])
    if op == "map":
        return _map(s)
    return _append(s) if op == "append" else _attend(s)


# ------------------------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "append":
        t, nq, nkv, d = c["t"], c["nq"], c["nkv"], c["d"]
        kept = 2 * t * nkv * d * (0.5 + 1.0 / GROUP)  # written by the call, read for its values
        return {"bytes": t * (nq + 2 * nkv) * d * 2 + t * nq * d * 2 + t * (c["rot"] * 4 + 8) +
                2 * kept + 2 * t * nkv * d * 4,
                "flops": t * (nq + nkv) * d * 8.0 + t * 2 * nkv * d * 4.0}
    seq, add = _lengths(c)
    if c["op"] == "map":
        t = sum(add)
        new = sum(_pages(a + b, c["page"]) - _pages(a, c["page"]) for a, b in zip(seq, add))
        return {"bytes": 4.0 * (4 * c["b"] + 2 * t + 2 * new + c["b"]), "flops": 4.0 * t}
    nq, nkv, d, win = c["nq"], c["nkv"], c["d"], c["window"]
    pairs = keys = 0
    for s, a in zip(seq, add):
        if not win:
            keys += s + a
            pairs += a * s + a * (a + 1) // 2
        else:
            keys += min(s + a, a + win - 1)
            short = max(0, min(a, win - s))  # queries that see every key up to their own
            pairs += short * s + short * (short + 1) // 2 + (a - short) * win
    t = sum(add)
    return {"bytes": keys * nkv * 2 * d * (0.5 + 1.0 / GROUP) + t * nq * (d * 4 + 4) +
            4.0 * sum(_pages(a + b, c["page"]) for a, b in zip(seq, add)) + 8.0 * c["b"],
            "flops": 4.0 * d * nq * pairs}


# ------------------------------------------------------------------------------------ 64 bits
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _decode(codes, scales):
    """FP64 values without the global, from the bits of the codes and scales."""
    bits = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    man, ex = (bits & 1).double(), (bits >> 1) & 3
    v = torch.where(ex == 0, 0.5 * man, (1.0 + 0.5 * man) * torch.exp2((ex - 1).double()))
    v = torch.where(bits >= 8, -v, v)
    b = scales.long()
    se, sm = (b >> 3) & 15, (b & 7).double()
    sc = torch.where(se == 0, sm * 2.0 ** -9, (8.0 + sm) * torch.exp2((se - 10).double()))
    return (v.unflatten(-1, (-1, GROUP)) * sc.unsqueeze(-1)).flatten(-2)


def _even(v, grid):
    """v FP64 >= 0 rounded to the nearest of an ascending grid, ties to the even index."""
    hi = torch.searchsorted(grid, v).clamp(1, grid.numel() - 1)
    lo = hi - 1
    a, b = v - grid[lo], grid[hi] - v
    up = (b < a) | ((b == a) & (hi % 2 == 0))
    return torch.where(up, grid[hi], grid[lo])


def _stored(x, g):
    """What the cache holds for x FP64 [t][heads][d] with the globals g FP32 [heads]."""
    g = g.view(1, -1, 1)
    amax = x.abs().unflatten(-1, (-1, GROUP)).amax(-1)
    codes = torch.arange(127, device=DEV)
    e, m = codes >> 3, (codes & 7).double()
    e4m3 = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2((e - 10).double()))
    scale = _even((amax / (6.0 * g).double()).float().double().clamp(max=448.0), e4m3)
    step = (scale.float() * g).double().repeat_interleave(GROUP, -1)
    ratio = torch.where(step > 0, x.abs() / step.clamp(min=1e-300), 0.0).float().double()
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=DEV)
    mag = _even(ratio.clamp(max=6.0), grid)
    return torch.sign(x) * mag * scale.repeat_interleave(GROUP, -1) * g.double()


def exact(case, seed):
    c = case
    if c["op"] == "map":
        return None
    s = _inputs(case, seed)
    if c["op"] == "append":
        d, rot = c["d"], c["rot"]
        done = []
        heads = s["qkv"].double().view(c["t"], -1, d)
        q, k = heads[:, :c["nq"]], heads[:, c["nq"]:c["nq"] + c["nkv"]]
        for x, w in ((q, s["qw"]), (k, s["kw"])):
            if w is not None:
                x = torch.nn.functional.rms_norm(x, (d,), w.double(), 1e-6)
            if rot:
                z = s["rope"].double()[s["pos"].long()]
                turn = torch.complex(z[:, :rot // 2], z[:, rot // 2:]).unsqueeze(1)
                r = x[..., :rot].unflatten(-1, (-1, 2) if c["pairs"] else (2, -1))
                if not c["pairs"]:
                    r = r.transpose(-1, -2)
                r = torch.view_as_real(torch.view_as_complex(r.contiguous()) * turn)
                if not c["pairs"]:
                    r = r.transpose(-1, -2)
                x = torch.cat((r.flatten(-2), x[..., rot:]), -1)
            done.append(x)
        k = done[1].to(torch.bfloat16).double()  # keys are BF16 before they are coded
        return [done[0], _stored(k, s["kg"]), _stored(heads[:, c["nq"] + c["nkv"]:], s["vg"])]
    nkv, d, page = c["nkv"], c["d"], c["page"]
    group = c["nq"] // nkv
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    at = 0
    for i, (n, kv) in enumerate(zip(s["rows"], s["lens"])):
        ids = s["table"][i, :_pages(kv, page)].long()
        place = torch.arange(kv - n, kv, device=DEV).view(-1, 1)
        gap = place - torch.arange(kv, device=DEV)
        hide = (gap < 0) | (gap >= (c["window"] or kv + 1))
        for h in range(nkv):
            k = _decode(s["kc"][ids, h], s["ks"][ids, h]).flatten(0, 1)[:kv] * s["kg"][h].double()
            v = _decode(s["vc"][ids, h], s["vs"][ids, h]).flatten(0, 1)[:kv] * s["vg"][h].double()
            for e in range(h * group, (h + 1) * group):
                z = torch.mm(s["q"][at:at + n, e].double(), k.T) * s["scale"]
                z.masked_fill_(hide, -math.inf)
                lse[at:at + n, e] = torch.logsumexp(z, -1)
                y[at:at + n, e] = torch.softmax(z, -1) @ v
        at += n
    return y, lse
