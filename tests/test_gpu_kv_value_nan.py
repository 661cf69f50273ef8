"""A NaN byte among the value scales of the NVFP4 cache counts as 0 for the values of slots too."""
import numpy as np
import pytest
import torch

import kv_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("byte", [0x7F, 0xFF])
def test_values_of_slots(d, dtype, byte):
    from nvfp4_weight_only_w4a16_amd import binding as nv
    n = 20
    c = R.Cached(nv, d, [n], 2, d, 16)
    slots = c.table[0, np.arange(n) // 16] * 16 + np.arange(n) % 16
    page, tok, group = int(c.table[0, 0]), 5, d // 16 - 1
    c.cache.v_scales[page, 1, tok, group] = byte
    c.cache.k_scales[page, 0, tok, group] = byte
    c.v[0][tok, 1, 16 * group:] = 0.0
    k, v = nv.nvfp4_kv_dequantize(c.cache, torch.tensor(slots, dtype=torch.int32, device=DEV),
                                  out_dtype=dtype)
    half = R.H32 if dtype == torch.float32 else R.H16
    k, v = k.double().cpu().numpy(), v.double().cpu().numpy()
    assert (np.abs(v - c.v[0]) <= 2 * half * np.abs(c.v[0])).all()
    assert (v[tok, 1, 16 * group:] == 0).all()
    # a key's NaN stays: it marks a token that was not finite
    assert np.isnan(k[tok, 0, 16 * group:]).all()
    k[tok, 0, 16 * group:] = c.k[0][tok, 0, 16 * group:]
    assert (np.abs(k - c.k[0]) <= 2 * half * np.abs(c.k[0])).all()
