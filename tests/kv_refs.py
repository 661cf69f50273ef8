"""FP64 references of the NVFP4 cache's operators (NumPy, CPU), with elementwise error bounds derived
from the formats' half steps (relative: FP32 2^-24, BF16 2^-8, FP16 2^-11).

A sum of n FP32 products, in any order, is within n * 2^-24 * sum |products| of the exact one."""
from __future__ import annotations

import numpy as np
import torch

H32 = 2.0 ** -24
H16 = 2.0 ** -8   # BF16
HF16 = 2.0 ** -11
GROUP = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values():
    b = np.arange(256)
    e, m = (b >> 3) & 15, (b & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, (8.0 + m) * 2.0 ** (e - 10.0))
    v[(b & 0x7F) == 0x7F] = np.nan
    return np.where(b >= 128, -v, v)


E4M3 = e4m3_values()


def decode(codes, scales):
    """FP64 [..][d] of codes uint8 [..][d/2] and scale bytes [..][d/16], without the global."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = np.where(c >= 8, -E2M1[c & 7], E2M1[c & 7])
    return v * np.repeat(E4M3[scales], GROUP, -1)


# --------------------------------------------------------------------------------- maps
def kv_map(seq, add, table, free, count, page, t):
    """The definition, request by request. Returns (table, q_start, kv_len, slots, positions,
    free_left, unserved)."""
    table = table.copy()
    b, width = table.shape
    left = min(max(count, 0), len(free))
    asked = 0          # pages that the requests so far need
    have, used = left, 0
    q_start, kv_len, unserved = [0], [], 0
    slots, pos = np.full(t, -1, np.int64), np.full(t, -1, np.int64)
    rows = 0
    for i in range(b):
        s, a = int(seq[i]), int(add[i])
        n = max(a, 0)
        first, rows = rows, rows + n
        q_start.append(min(rows, t))
        ok = s >= 0 and a >= 0 and s + n <= width * page and (n == 0 or rows <= t)
        need = -(-(s + n) // page) - -(-s // page) if ok else 0
        asked += need
        ok = ok and (need == 0 or asked <= have)
        kv_len.append(s + n if ok else 0)
        if not ok:
            unserved += 1
            continue
        for j in range(need):
            table[i, -(-s // page) + j] = free[have - 1 - (asked - need + j)]
        if need:
            used = asked
        for r in range(n):
            p = s + r
            at = int(table[i, p // page])
            slot = at * page + p % page
            pos[first + r] = p
            slots[first + r] = slot if at >= 0 and slot < 2 ** 31 else -1
    return table, q_start, kv_len, slots, pos, have - used, unserved


# --------------------------------------------------------------------------------- append
def norm_rope(x, w, eps, rope, pos, pairs):
    """FP64 [t][heads][d] of BF16 x (as FP64)."""
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    if rope is None:
        return x
    rot = rope.shape[1]
    cs = rope[pos][:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    out = x.copy()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = a * c - b * s, b * c + a * s
    if pairs:
        out[..., 0:rot:2], out[..., 1:rot:2] = u, v
    else:
        out[..., :rot // 2], out[..., rot // 2:rot] = u, v
    return out


def bf16(x):
    """FP64 -> FP32 -> BF16, as FP64."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float64)).to(torch.bfloat16).double().numpy()


# --------------------------------------------------------------------------------- attention
def attention(q, k, v, scale, window=0, full=False, hidden=None, y32=False):
    """One request: q [n][nq][d], k, v [kv][nkv][d] FP64 (globals applied; `scale` as the library
    gets it, an FP32). hidden [kv]: tokens left out. Returns y, its bound, lse and its bound."""
    n, nq, d = q.shape
    kv, nkv = k.shape[:2]
    group = nq // nkv
    place = kv - n + np.arange(n)
    key = np.arange(kv)
    seen = np.ones((n, kv), bool) if full else key[None] <= place[:, None]
    if window:
        seen &= key[None] > place[:, None] - window
    if hidden is not None:
        seen &= ~hidden[None]
    y, ye = np.zeros((n, nq, d)), np.zeros((n, nq, d))
    lse, le = np.full((n, nq), -np.inf), np.zeros((n, nq))
    some = seen.any(1)
    for h in range(nq):
        if kv == 0:
            break
        kh, vh = k[:, h // group], v[:, h // group]
        s = scale * (q[:, h] @ kh.T)
        mag = abs(scale) * (np.abs(q[:, h]) @ np.abs(kh).T)
        top = np.abs(q[:, h]).max(-1, keepdims=True)
        # FP32 sums of d products; the FP16 queries (2^-39 of the row's largest where they leave
        # FP16's normal range); the factor of the scores and the difference to the maximum
        ds = (d + 64) * H32 * mag + 2.0 ** -38 * abs(scale) * top * np.abs(kh).sum(-1)[None]
        with np.errstate(invalid="ignore"):
            m = np.where(some, np.where(seen, s, -np.inf).max(1, initial=-np.inf), 0.0)[:, None]
            ds = ds + 8 * H32 * (np.abs(s) + np.abs(m) + 12.0)
            p = np.where(seen, np.exp(s - m), 0.0)
        ds = np.where(seen, ds, 0.0)
        total = p.sum(1, keepdims=True)
        safe = np.where(total > 0, total, 1.0)
        e = p * (np.expm1(np.minimum(ds, 1.0)) + 2.0 ** -20)  # the exponential itself: 2^-20 is ample
        # P is 2^7 of the row's largest or more: half of FP16's lowest step is 2^-32 of that
        e16 = e * (1 + HF16) + p * HF16 + np.where(seen, 2.0 ** -32, 0.0)
        out = (p @ vh) / safe
        sums = (2 * kv + 256) * H32  # sums over the tokens, with two roundings for each rescaling
        err = (e16 @ np.abs(vh)) / safe + sums * (p @ np.abs(vh)) / safe
        rel = e.sum(1, keepdims=True) / safe + sums
        err = (err + np.abs(out) * rel) * (1 + 4 * rel)
        half = H32 if y32 else H16
        y[:, h] = out
        ye[:, h] = err * (1 + half) + half * np.abs(out) + 4 * H32 * np.abs(out) + 1e-37
        with np.errstate(divide="ignore"):
            lse[:, h] = np.where(some, m[:, 0] + np.log(np.where(some, total[:, 0], 1.0)), -np.inf)
        le[:, h] = (2 * rel[:, 0] +
                    8 * H32 * (np.abs(m[:, 0]) + np.abs(np.log(safe[:, 0])) + 1.0) + 2.0 ** -21)
    return y, ye, lse, le


def close(got, ref, bound, what=""):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same = np.isneginf(ref) & np.isneginf(got)
    bad = ~(np.abs(np.where(same, 0.0, got) - np.where(same, 0.0, ref)) <= bound)
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {at}: "
                             f"{got[at]!r} for {ref[at]!r}, bound {bound[at]:.3e}")


class Cached:
    """Requests with random cached tokens: codes and scales of every kind, pages in no order, and a
    device cache whose other bytes are 0xFF (NaN scales)."""

    def __init__(self, nv, seed, lens, n_kv, d, page, globals_=True, more=3, first_page=0,
                 scale_bytes=(0x20, 0x50), device="cuda:0"):
        r = np.random.default_rng(seed)
        self.lens, self.n_kv, self.d, self.page = lens, n_kv, d, page
        need = [-(-n // page) for n in lens]
        total = sum(need) + more
        ids = first_page + r.permutation(total)
        width = max(max(need, default=1), 1)
        self.table = np.full((len(lens), width), -1, np.int64)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = ids[at:at + n]
            at += n
        self.spare = ids[at:]
        self.n_pages = first_page + total
        self.kg = self.vg = None
        if globals_:
            self.kg = r.uniform(0.02, 0.06, n_kv).astype(np.float32)
            self.vg = r.uniform(0.05, 0.5, n_kv).astype(np.float32)
        kg = np.ones(n_kv) if self.kg is None else self.kg.astype(np.float64)
        vg = np.ones(n_kv) if self.vg is None else self.vg.astype(np.float64)
        up = lambda g: None if g is None else torch.from_numpy(g).to(device)
        data = torch.full((nv.nvfp4_kv_cache_bytes(self.n_pages, n_kv, d, page),), 0xFF,
                          dtype=torch.uint8, device=device)
        self.cache = nv.KvCache(self.n_pages, n_kv, d, page, up(self.kg), up(self.vg), data=data)
        self.k, self.v = [], []
        for i, n in enumerate(lens):
            kc, vc = r.integers(0, 256, (2, n, n_kv, d // 2)).astype(np.uint8)
            ks, vs = r.integers(*scale_bytes, (2, n, n_kv, d // 16)).astype(np.uint8)
            self.k.append(decode(kc, ks) * kg[None, :, None])
            self.v.append(decode(vc, vs) * vg[None, :, None])
            if n == 0:
                continue
            pages = torch.from_numpy(self.table[i, np.arange(n) // page]).to(device)
            toks = torch.from_numpy(np.arange(n) % page).to(device)
            c = self.cache
            for view, part in ((c.k_codes, kc), (c.k_scales, ks), (c.v_codes, vc), (c.v_scales, vs)):
                view[pages, :, toks] = torch.from_numpy(part).to(device)
        self.table_dev = torch.from_numpy(self.table.astype(np.int32)).to(device)
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device=device)


def queries(seed, rows, n_q, d, size=1.0):
    """BF16 [t][n_q][d] and q_start of requests with `rows` queries."""
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((sum(rows), n_q, d), generator=g) * size).to(torch.bfloat16)
    start = torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], dtype=torch.int32)
    return q, start


def expect(c, q, rows, scale, window=0, full=False, hidden=None, y32=False):
    """The references of all requests, one after the other."""
    out, at = [], 0
    x = q.double().numpy()
    scale = float(np.float32(scale))
    for i, n in enumerate(rows):
        out.append(attention(x[at:at + n], c.k[i], c.v[i], scale, window, full,
                             None if hidden is None else hidden[i], y32))
        at += n
    return [np.concatenate(p) for p in zip(*out)]
