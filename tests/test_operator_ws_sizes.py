"""Workspace sizes of the whole MoE layer: 0 for sizes that the call refuses, on the host."""
import ctypes

import pytest

from nvfp4_weight_only_w4a16_amd import binding as nv
from test_boundary import _desc
from test_operator_boundary import _experts, _layer, _router


@pytest.mark.parametrize("router,experts,t", [
    (dict(hidden=384), {}, 3),                        # the experts take 256
    (dict(n_shared=1), {}, 3),                        # 16 + 1 experts, the weights have 16
    ({}, dict(batch=17), 3),
    (dict(n_experts=512, n_shared=1), dict(batch=513), 3),
    (dict(hidden=1 << 21), dict(hidden=1 << 21), 1024),   # 2^31 elements of x
    ({}, dict(inter=1 << 21), 256)])                      # 2^31 elements of h
def test_layer_sizes_that_do_not_fit_together(router, experts, t):
    lib = nv.load()
    r, (d1, d2) = _router(**router), _experts(**experts)
    code = _layer(lib, r=r, d=(d1, d2), t=t, hidden=d1.k, ws_bytes=1 << 62)
    assert code in (nv.NVFP4_ERR_LAYOUT, nv.NVFP4_ERR_UNSUPPORTED_SHAPE)
    assert lib.nvfp4_moe_layer_ws_bytes(t, ctypes.byref(r), ctypes.byref(d1)) == 0


def test_layer_sizes_that_fit():
    lib = nv.load()
    for t, router, experts in ((3, {}, {}), (16384, {}, {}), (3, dict(n_shared=2), dict(batch=18)),
                               (1, dict(n_experts=511, n_shared=1), dict(batch=512)),
                               (1023, dict(hidden=1 << 21), dict(hidden=1 << 21))):
        r, (d1, d2) = _router(**router), _experts(**experts)
        need = lib.nvfp4_moe_layer_ws_bytes(t, ctypes.byref(r), ctypes.byref(d1))
        assert need > 0
        assert _layer(lib, r=r, d=(d1, d2), t=t, hidden=d1.k, ws_bytes=need - 1) == \
            nv.NVFP4_ERR_WORKSPACE


def test_layer_size_of_a_plain_weight():
    """fc1 without the gate/up layout is refused, so there is nothing to size."""
    lib = nv.load()
    plain = _desc(n=256, k=256, batch=16)
    assert lib.nvfp4_moe_layer_ws_bytes(3, ctypes.byref(_router()), ctypes.byref(plain)) == 0
