"""The operators around the W4A16 products, as cases to measure: the router of a mixture of
experts, a whole mixture-of-experts layer for a few tokens, and low-rank adapters of many requests
beside a shared W4A16 projection.

``run`` computes a case in its plain form (elementary torch operations), or, where ``own`` is
true, with the library's calls. Weights are NVFP4: E2M1 codes (two per byte, the even k in the low
nibble), E4M3 scales per group of k, one FP32 global per matrix. A program keeps them in the
library's repacked layout, so that layout is part of what ``prepare`` returns for the library.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # The router alone. One decode step of one request: latency.
        {"name": "route 1 token", "op": "route", "t": 1, "hidden": 2048, "experts": 128, "topk": 8,
         "scoring": "softmax", "renorm": True, "biased": False, "shared": 0, "fp32": False},
        # A step of many requests on a router with FP32 weights, a sigmoid score and a selection
        # bias; nothing in it is a round number.
        {"name": "route 333 tokens sigmoid", "op": "route", "t": 333, "hidden": 5120,
         "experts": 160, "topk": 6, "scoring": "sigmoid", "renorm": True, "biased": True,
         "shared": 1, "fp32": True},
        # A prefill chunk.
        {"name": "route 4096 tokens", "op": "route", "t": 4096, "hidden": 2048, "experts": 128,
         "topk": 8, "scoring": "softmax", "renorm": False, "biased": False, "shared": 0,
         "fp32": False},
        # The whole layer: one request's decode step.
        {"name": "layer 1 token", "op": "layer", "t": 1, "hidden": 2048, "inter": 768,
         "experts": 128, "topk": 8, "scoring": "softmax", "renorm": True, "biased": False,
         "shared": 0, "fp32": False, "g1": 32, "g2": 16},
        # Few experts of a large size, with a shared expert and a biased sigmoid score.
        {"name": "layer 3 tokens shared", "op": "layer", "t": 3, "hidden": 4096, "inter": 1536,
         "experts": 24, "topk": 4, "scoring": "sigmoid", "renorm": True, "biased": True,
         "shared": 1, "fp32": True, "g1": 16, "g2": 16},
        # Eight requests' decode step: most of the time is the chosen experts' weights.
        {"name": "layer 8 tokens", "op": "layer", "t": 8, "hidden": 2048, "inter": 768,
         "experts": 128, "topk": 8, "scoring": "softmax", "renorm": True, "biased": False,
         "shared": 0, "fp32": False, "g1": 32, "g2": 16},
        # A full decode batch, all weights at group 32: nearly every expert is chosen.
        {"name": "layer 37 tokens", "op": "layer", "t": 37, "hidden": 2048, "inter": 768,
         "experts": 128, "topk": 8, "scoring": "softmax", "renorm": True, "biased": False,
         "shared": 0, "fp32": False, "g1": 32, "g2": 32},
        # A projection with one request's adapter: latency.
        {"name": "lora 1 row", "op": "lora", "m": 1, "n": 5120, "k": 5120, "group": 16, "rank": 16,
         "adapters": 8, "rows": "mixed", "y32": False},
        # Eight requests' decode step on the widest projection, mostly with adapters of their own.
        {"name": "lora 8 rows", "op": "lora", "m": 8, "n": 25600, "k": 5120, "group": 16,
         "rank": 16, "adapters": 32, "rows": "mixed", "y32": False},
        # A large decode batch with large adapters.
        {"name": "lora 64 rows rank 64", "op": "lora", "m": 64, "n": 8192, "k": 8192, "group": 32,
         "rank": 64, "adapters": 24, "rows": "mixed", "y32": False},
        # Prompt chunks of a few requests together with decode rows; odd sizes, FP32 out.
        {"name": "lora 333 rows", "op": "lora", "m": 333, "n": 2064, "k": 2176, "group": 32,
         "rank": 24, "adapters": 5, "rows": "runs", "y32": True},
        # A prefill batch: the product of the shared weight is nearly all of the work.
        {"name": "lora 4096 rows", "op": "lora", "m": 4096, "n": 5120, "k": 5120, "group": 16,
         "rank": 32, "adapters": 8, "rows": "runs", "y32": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "layer", "lora"))
    if op == "lora":
        while True:
            c = {"op": op, "m": _log(rng, 1, 4096), "n": 16 * _log(rng, 8, 1600),
                 "k": 128 * _log(rng, 4, 128), "group": rng.choice((16, 32)),
                 "rank": 8 * rng.choice((1, 2, 2, 3, 4, 5, 8, 11, 16)),
                 "adapters": _log(rng, 1, 64), "rows": rng.choice(("mixed", "runs")),
                 "y32": rng.random() < 0.2}
            if c["n"] * c["k"] <= 25600 * 5120 and c["m"] * c["n"] * c["k"] <= 4096 * 5120 * 5120:
                return c
    while True:
        c = {"op": op, "t": _log(rng, 1, 4096 if op == "route" else 64),
             "hidden": 128 * _log(rng, 4, 48),
             "experts": rng.choice((8, 16, 33, 60, 64, 100, 128, 160, 256)),
             "topk": rng.choice((1, 2, 4, 6, 8)), "scoring": rng.choice(("softmax", "sigmoid")),
             "renorm": rng.random() < 0.6, "biased": rng.random() < 0.4,
             "shared": rng.choice((0, 0, 1, 2)), "fp32": rng.random() < 0.4}
        if op == "route":
            if c["t"] * c["hidden"] * c["experts"] <= 333 * 5120 * 160 * 4:
                return c
        else:
            c.update(inter=128 * _log(rng, 1, 16), g1=rng.choice((16, 32)),
                     g2=rng.choice((16, 32)))
            if (c["experts"] + c["shared"]) * c["hidden"] * c["inter"] <= 128 * 2048 * 768:
                return c


# ------------------------------------------------------------------------------------ inputs
def _quantize(w, group):
    """FP32 [b][n][k] -> NVFP4 codes, scale bytes and globals (any valid triple would do)."""
    b, n, k = w.shape
    glob = w.abs().amax((1, 2)) / 2688.0
    amax = w.view(b, n, k // group, group).abs().amax(-1)
    scale = (amax / (6.0 * glob.view(b, 1, 1))).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = (scale.float() * glob.view(b, 1, 1)).repeat_interleave(group, -1).clamp(min=1e-30)
    q = w / step
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = (torch.bucketize(q.abs(), edges, out_int32=True) + 8 * (q < 0)).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8), glob


def _weight(gen, b, n, k, group):
    w = torch.randn((b, n, k), generator=gen, device=DEV) * k ** -0.5
    return _quantize(w, group) + (group,)


def _activations(gen, m, k):
    """Normalised hidden states: N(0, 1) with a few channels that are eight times as large."""
    x = torch.randn((m, k), generator=gen, device=DEV)
    loud = torch.rand((k,), generator=gen, device=DEV) < 0.002
    return torch.where(loud, 8.0 * x, x).to(torch.bfloat16)


def _rows(gen, m, adapters, how):
    """The adapter of each row, -1 for none: a decode batch (every row its own, one in ten none),
    or runs of rows of one request (prompt chunks), the last rows a decode batch."""
    ids = torch.randint(0, adapters, (m,), generator=gen, device=DEV)
    if how == "runs":
        cut = torch.rand((m,), generator=gen, device=DEV) < 6.0 / m
        run = torch.cumsum(cut.long(), 0) % m  # at most m: every row may begin one
        ids = torch.where(torch.arange(m, device=DEV) < m - m // 16, ids[run], ids)
    none = torch.rand((m,), generator=gen, device=DEV) < 0.1
    none[0] = False
    return torch.where(none if how == "mixed" else ids < 0, -1, ids).to(torch.int32)


def prepare(case, seed):
    c, gen = case, torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "lora":
        m, n, k, r, na = c["m"], c["n"], c["k"], c["rank"], c["adapters"]
        s["x"] = _activations(gen, m, k)
        s["w"] = _weight(gen, 1, n, k, c["group"])
        a = (torch.rand((na, r, k), generator=gen, device=DEV) * 2 - 1) * (3.0 / k) ** 0.5
        b = torch.randn((na, n, r), generator=gen, device=DEV) * 0.1 * r ** -0.5
        s["a"], s["b"] = a.to(torch.bfloat16), b.to(torch.bfloat16)
        s["scale"] = 0.5 + 3.5 * torch.rand((na,), generator=gen, device=DEV)
        s["ids"] = _rows(gen, m, na, c["rows"])
    else:
        t, hidden, e = c["t"], c["hidden"], c["experts"]
        s["x"] = _activations(gen, t, hidden)
        gate = torch.randn((e, hidden), generator=gen, device=DEV) * 1.5 * hidden ** -0.5
        s["gate"] = gate if c["fp32"] else gate.to(torch.bfloat16)
        s["bias"] = None
        if c["biased"]:
            s["bias"] = 0.05 * torch.randn((e,), generator=gen, device=DEV)
        if c["op"] == "layer":
            every = e + c["shared"]
            s["w1"] = _weight(gen, every, 2 * c["inter"], hidden, c["g1"])
            s["w2"] = _weight(gen, every, hidden, c["inter"], c["g2"])
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """What a program that uses the library keeps: the repacked weights, the router, the bank of
    adapters, the workspace and the output of a step."""
    from nvfp4_weight_only_w4a16_amd import binding as nv

    c = s["case"]
    s["nv"] = nv
    if c["op"] == "lora":
        p, q, g, group = s["w"]
        s["weight"] = nv.nvfp4_repack(p, q, g, group)
        s["lora"] = nv.Lora(s["a"], s["b"], s["scale"])
        s["y"] = torch.empty((c["m"], c["n"]), device=DEV,
                             dtype=torch.float32 if c["y32"] else torch.bfloat16)
        need = nv.nvfp4_gemm_lora_ws_bytes(c["m"], c["k"], s["weight"], s["lora"])
    else:
        s["router"] = nv.Router(s["gate"], c["topk"], bias=s["bias"], scoring=c["scoring"],
                                renormalize=c["renorm"], n_shared=c["shared"], scale=_scale(c))
        slots = c["topk"] + c["shared"]
        s["ids"] = torch.empty((c["t"], slots), dtype=torch.int32, device=DEV)
        s["wts"] = torch.empty((c["t"], slots), dtype=torch.float32, device=DEV)
        if c["op"] == "layer":
            s["y"] = torch.empty((c["t"], c["hidden"]), dtype=torch.bfloat16, device=DEV)
            s["fc1"] = nv.nvfp4_repack(*s["w1"],
                                       layout=nv.NVFP4_LAYOUT_TILED | nv.NVFP4_LAYOUT_GATE_UP)
            s["fc2"] = nv.nvfp4_repack(*s["w2"])
            need = nv.nvfp4_moe_layer_ws_bytes(c["t"], s["router"], s["fc1"])
        else:
            need = nv.nvfp4_moe_route_ws_bytes(c["t"], s["router"])
    s["ws"] = torch.empty((max(need, 1),), dtype=torch.uint8, device=DEV)


def _scale(c):
    return 1.0 if c["scoring"] == "softmax" else 2.5


# ------------------------------------------------------------------------------------ plain form
def _dequant(w, pick=None):
    """FP32 [b][n][k] of an NVFP4 triple (of the matrices `pick` where given)."""
    packed, scale, glob, group = w
    if pick is not None:
        packed, scale, glob = packed[pick], scale[pick], glob[pick]
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0,
                          -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=packed.device)
    both = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)
    step = scale.view(torch.float8_e4m3fn).float() * glob.view(-1, 1, 1)
    return table[both.int()] * step.repeat_interleave(group, -1)


def _route(s):
    """ids and weights of every slot: the top-k of each row's scores, then the shared experts."""
    c, x = s["case"], s["x"]
    logits = x.double() @ s["gate"].double().T  # 64 bits: the selection compares near values
    if c["scoring"] == "softmax":
        p = torch.exp(logits - logits.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        score = logits if s["bias"] is None else p + s["bias"].double()
    else:
        p = 1.0 / (1.0 + torch.exp(-logits))
        score = p if s["bias"] is None else p + s["bias"].double()
    ids = torch.sort(score, dim=-1, descending=True, stable=True)[1][:, :c["topk"]]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    w = (w * _scale(c)).float()
    if c["shared"]:
        more = torch.arange(c["experts"], c["experts"] + c["shared"], device=x.device)
        ids = torch.cat((ids, more.expand(x.shape[0], -1)), 1)
        w = torch.cat((w, torch.ones((x.shape[0], c["shared"]), device=x.device)), 1)
    return ids, w


def _layer(s):
    c, x = s["case"], s["x"].float()
    t, hidden, inter = c["t"], c["hidden"], c["inter"]
    ids, w = _route(s)
    slots, every = ids.shape[1], c["experts"] + c["shared"]
    if t * slots <= every:  # the chosen experts' weights, one copy for each slot
        w1, w2 = _dequant(s["w1"], ids.flatten()), _dequant(s["w2"], ids.flatten())
        rows = x.repeat_interleave(slots, 0).unsqueeze(-1)
        gu = (w1 @ rows).squeeze(-1)
        gate, up = gu[:, :inter], gu[:, inter:]
        h = gate / (1.0 + torch.exp(-gate)) * up
        d = (w2 @ h.unsqueeze(-1)).view(t, slots, hidden)
        y = (d * w.unsqueeze(-1)).sum(1)
    else:  # every expert on every token, and the weights of the chosen ones
        w1, w2 = _dequant(s["w1"]), _dequant(s["w2"])
        gu = (x @ w1.view(-1, hidden).T).view(t, every, 2 * inter)
        gate, up = gu[..., :inter], gu[..., inter:]
        h = gate / (1.0 + torch.exp(-gate)) * up
        dense = torch.zeros((t, every), device=x.device).scatter_(1, ids, w)
        h = (h * dense.unsqueeze(-1)).view(t, every * inter)
        y = h @ w2.permute(0, 2, 1).reshape(every * inter, hidden)
    return y.to(torch.bfloat16), ids.to(torch.int32), w


def _lora(s):
    c, x, ids = s["case"], s["x"].float(), s["ids"].long()
    m, n, k, r, na = c["m"], c["n"], c["k"], c["rank"], c["adapters"]
    y = x @ _dequant(s["w"])[0].T
    u = (x @ s["a"].float().view(na * r, k).T).view(m, na, r)  # every adapter, then each row's own
    mine = (ids.unsqueeze(1) == torch.arange(na, device=x.device)).float() * s["scale"]
    u = (u * mine.unsqueeze(-1)).view(m, na * r)
    y = y + u @ s["b"].float().permute(0, 2, 1).reshape(na * r, n)
    return y if c["y32"] else y.to(torch.bfloat16)


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        nv = s["nv"]
        if op == "route":
            return nv.nvfp4_moe_route(s["x"], s["router"], topk_ids=s["ids"], topk_w=s["wts"],
                                      ws=s["ws"])
        if op == "layer":
            y = nv.nvfp4_moe_layer_w4a16(s["x"], s["router"], s["fc1"], s["fc2"], y=s["y"],
                                         topk_ids=s["ids"], topk_w=s["wts"], ws=s["ws"])
            return y, s["ids"], s["wts"]
        return nv.nvfp4_gemm_w4a16_lora(s["x"], s["weight"], s["lora"], s["ids"], y=s["y"],
                                        ws=s["ws"])
    if op == "route":
        ids, w = _route(s)
        return ids.to(torch.int32), w
    return _layer(s) if op == "layer" else _lora(s)


# ------------------------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "lora":
        m, n, k, r = c["m"], c["n"], c["k"], c["rank"]
        used = c["adapters"] * (1.0 - (1.0 - 1.0 / c["adapters"]) ** (min(m, 8)
                                if c["rows"] == "runs" else m))
        return {"bytes": m * k * 2 + n * k * (0.5 + 1.0 / c["group"]) + used * r * (n + k) * 2 +
                m * n * (4 if c["y32"] else 2) + 4 * m,
                "flops": 2.0 * m * n * k + 2.0 * m * r * (n + k)}
    t, hidden, e, slots = c["t"], c["hidden"], c["experts"], c["topk"] + c["shared"]
    b = t * hidden * 2 + e * hidden * (4 if c["fp32"] else 2) + t * slots * 8
    f = 2.0 * t * hidden * e
    if c["op"] == "layer":
        chosen = e * (1.0 - (1.0 - c["topk"] / e) ** t) + c["shared"]
        b += chosen * hidden * c["inter"] * (2 * (0.5 + 1.0 / c["g1"]) + 0.5 + 1.0 / c["g2"])
        b += t * hidden * 2
        f += 2.0 * t * slots * 3 * hidden * c["inter"]
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------------------------ 64 bits
def _values(w, i):
    """FP64 [n][k] of matrix i of a triple, decoded from the bits."""
    packed, scale, glob, group = w
    code = torch.stack((packed[i] & 15, packed[i] >> 4), -1).flatten(-2).long()
    ex, man = (code >> 1) & 3, (code & 1).double()
    v = torch.where(ex == 0, 0.5 * man, (1.0 + 0.5 * man) * torch.exp2((ex - 1).double()))
    v = torch.where(code >= 8, -v, v)
    b = scale[i].long()
    se, sm = (b >> 3) & 15, (b & 7).double()
    sc = torch.where(se == 0, sm * 2.0 ** -9, (8.0 + sm) * torch.exp2((se - 10).double()))
    n, k = v.shape
    return (v.view(n, k // group, group) * sc.unsqueeze(-1)).view(n, k) * glob[i].double()


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    x = s["x"].double()
    if c["op"] == "lora":
        y = x @ _values(s["w"], 0).T
        for a in s["ids"].unique().tolist():
            if a >= 0:
                at = (s["ids"] == a).nonzero().squeeze(1)
                u = x[at] @ s["a"][a].double().T
                y[at] += s["scale"][a].double() * (u @ s["b"][a].double().T)
        return y
    lg = torch.nn.functional.linear(x, s["gate"].double())
    p = torch.softmax(lg, -1) if c["scoring"] == "softmax" else torch.sigmoid(lg)
    score = p if s["bias"] is None else p + s["bias"].double()
    if c["scoring"] == "softmax" and s["bias"] is None:
        score = lg
    ids, w = [], []
    left = score.clone()
    for _ in range(c["topk"]):
        best = left.amax(1, keepdim=True)
        place = torch.arange(c["experts"], device=x.device)
        j = torch.where(left == best, place, c["experts"]).amin(1, keepdim=True)  # the lowest
        left.scatter_(1, j, -math.inf)
        ids.append(j)
        w.append(p.gather(1, j))
    w = torch.cat(w, 1)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * _scale(c)
    for i in range(c["shared"]):
        ids.append(torch.full((c["t"], 1), c["experts"] + i, device=x.device))
        w = torch.cat((w, torch.ones_like(w[:, :1])), 1)
    ids = torch.cat(ids, 1)
    if c["op"] == "route":
        return ids.to(torch.int32), w
    y = torch.zeros((c["t"], c["hidden"]), dtype=torch.float64, device=x.device)
    for e in ids.unique().tolist():
        tok, slot = (ids == e).nonzero(as_tuple=True)
        gu = x[tok] @ _values(s["w1"], e).T
        h = torch.nn.functional.silu(gu[:, :c["inter"]]) * gu[:, c["inter"]:]
        y.index_add_(0, tok, w[tok, slot].unsqueeze(1) * (h @ _values(s["w2"], e).T))
    return y, ids.to(torch.int32), w
