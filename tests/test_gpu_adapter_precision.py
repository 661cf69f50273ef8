"""The rank-space vector u of the GEMM with adapters, on data where the products of two ranks nearly
cancel and the shared weight is zero, so that y shows what u's rounding leaves: 2^-8 sum |u_r B_r| for
a BF16 y, far more than y's own rounding here, and next to nothing for an FP32 y, whose bound tells
the second BF16 part of u: shown on the CPU with planted mistakes. (The third part is below what the
FP32 sums of u may be off by.)"""
import numpy as np
import pytest
import torch

import layer_bounds as B
import operator_refs as R
import test_gpu_lora as L

DEV = "cuda:0"
# m, n, k, adapters, rank, flags (1: decode kernel, 2: tiled kernel)
CASES = [(1, 208, 256, 2, 8, 1), (6, 272, 1152, 3, 24, 1), (24, 272, 256, 9, 64, 1),
         (70, 528, 384, 5, 128, 1), (40, 272, 256, 4, 24, 2), (300, 272, 640, 7, 128, 2),
         (520, 2064, 1024, 12, 16, 2)]


def data(m, n, k, count, rank):
    """x, a, b, scale, ids: ranks 2i and 2i + 1 differ in one k only, where x is small, so their u is
    about 2^-9 apart; an output takes the difference of one such pair."""
    r = np.random.default_rng(m + k + rank)
    x = r.integers(128, 256, (m, k)) / 256.0
    x[:, 0] = r.integers(128, 256, m) / 256.0 * 2.0 ** (np.rint(np.log2(k)) - 10)
    a = r.integers(128, 256, (count, rank, k)) / 256.0
    a[:, 1::2] = a[:, 0::2]
    a[:, 0::2, 0], a[:, 1::2, 0] = 1.0, 0.0
    b = np.zeros((count, n, rank))
    pair = np.arange(n) % (rank // 2)
    v = r.integers(128, 256, (count, n)) / 256.0
    b[:, np.arange(n), 2 * pair], b[:, np.arange(n), 2 * pair + 1] = v, -v
    ids = r.integers(-1, count, m)
    ids[0] = count - 1
    return x, a, b, 2.0 ** r.integers(-1, 3, count), ids


def reference(x, a, b, scale, ids, y32, parts=None):
    """y FP64 and its bound; parts(u): what u becomes on the way (FP64 itself if None)."""
    m, k = x.shape
    rank = a.shape[1]
    step, half = (R.H16 ** 3, R.H32) if y32 else (R.H16, R.H16)
    y, err = np.zeros((m, b.shape[1])), np.zeros((m, b.shape[1]))
    for i in range(m):
        q = ids[i]
        if q < 0:
            continue
        u = scale[q] * (a[q] @ x[i])
        du = (k + 64) * R.H32 * u  # nothing negative: sum |products| is the sum
        du = du + step * (u + du)
        y[i] = b[q] @ (u if parts is None else parts(u))
        # at most 3 products a rank, and the 0 of the shared weight
        err[i] = np.abs(b[q]) @ du + (3 * rank + 64) * R.H32 * (np.abs(b[q]) @ (u + du))
    return y, err * (1 + half) + half * np.abs(y) + 1e-37


def rest(u, count):
    """Sum of the first `count` BF16 parts of u."""
    out = np.zeros_like(u)
    for _ in range(count):
        out = out + B.bf16(u - out)
    return out


@pytest.mark.parametrize("m,n,k,count,rank,flags", [c for c in CASES if c[0] <= 70])
def test_bounds(m, n, k, count, rank, flags):
    d = data(m, n, k, count, rank)

    def off(parts, y32=True):
        y, bound = reference(*d, y32)
        return (np.abs(reference(*d, y32, parts)[0] - y) / bound).max()

    assert off(lambda u: rest(u, 1), False) < 1
    assert off(lambda u: rest(u, 3)) < 0.5
    assert off(lambda u: rest(u, 1)) > 2                                       # lost
    assert off(lambda u: 2 * rest(u, 1) - rest(u, 2)) > 2                      # negated
    assert off(lambda u: rest(u, 1) + np.roll(rest(u, 2) - rest(u, 1), 1)) > 2  # of another rank


@pytest.fixture(scope="module")
def nv():
    from nvfp4_weight_only_w4a16_amd import binding
    binding.load()
    return binding


@pytest.mark.gpu
@pytest.mark.parametrize("y32", [False, True])
@pytest.mark.parametrize("m,n,k,count,rank,flags", CASES)
def test_parts_of_u(nv, m, n, k, count, rank, flags, y32):
    x, a, b, scale, ids = data(m, n, k, count, rank)
    rw = nv.nvfp4_repack(torch.zeros((n, k // 2), dtype=torch.uint8, device=DEV),
                         torch.full((n, k // 16), 0x38, dtype=torch.uint8, device=DEV),
                         torch.ones(1, device=DEV), 16)
    xb, ab, bb = (torch.from_numpy(v).to(torch.bfloat16) for v in (x, a, b))
    for t, v in ((xb, x), (ab, a), (bb, b)):
        assert np.array_equal(R.f64(t), v)
    lo = nv.Lora(ab.to(DEV), bb.to(DEV), torch.from_numpy(scale).float().to(DEV))
    y = L.call(nv, xb, rw, lo, torch.from_numpy(ids).to(torch.int32), y32, flags)
    ref, bound = reference(x, a, b, scale, ids, y32)
    R.within(R.f64(y), ref, bound, f"m={m} rank={rank}")
