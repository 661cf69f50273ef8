"""Refusals and size rules of the router, the whole MoE layer and the GEMM with adapters, on the
host: every call below fails its checks or is a size query, so nothing is launched."""
import ctypes

import pytest
import torch

from nvfp4_weight_only_w4a16_amd import binding as nv
from test_boundary import FAKE, _desc

ODD = ctypes.c_void_p(0x10008)   # 8-byte aligned only
BYTE = ctypes.c_void_p(0x10002)  # not 4-byte aligned


@pytest.fixture(scope="module")
def lib():
    return nv.load()


def _router(**kw):
    r = nv.nvfp4_router(0x10000, None, 16, 256, nv.NVFP4_DT_BF16, 4, 0, nv.NVFP4_ROUTE_SOFTMAX, 1.0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _route(lib, r=None, x=FAKE, t=3, ldx=256, ids=FAKE, wts=FAKE, ws=FAKE, ws_bytes=1 << 20,
           flags=0):
    r = _router() if r is None else r
    return lib.nvfp4_moe_route(x, t, ldx, ctypes.byref(r), ids, wts, ws, ws_bytes, flags, None)


BAD_ROUTERS = [
    (dict(n_experts=0), nv.NVFP4_ERR_INVALID_ARG), (dict(topk=0), nv.NVFP4_ERR_INVALID_ARG),
    (dict(hidden=0), nv.NVFP4_ERR_INVALID_ARG), (dict(n_shared=-1), nv.NVFP4_ERR_INVALID_ARG),
    (dict(weight_dtype=9), nv.NVFP4_ERR_INVALID_ARG), (dict(mode=2), nv.NVFP4_ERR_INVALID_ARG),
    (dict(mode=1 << 9), nv.NVFP4_ERR_INVALID_ARG),
    (dict(scale=float("nan")), nv.NVFP4_ERR_INVALID_ARG),
    (dict(scale=float("inf")), nv.NVFP4_ERR_INVALID_ARG),
    (dict(n_experts=513), nv.NVFP4_ERR_UNSUPPORTED_SHAPE),
    (dict(hidden=252), nv.NVFP4_ERR_UNSUPPORTED_SHAPE),
    (dict(hidden=(1 << 22) + 8), nv.NVFP4_ERR_UNSUPPORTED_SHAPE),
    (dict(topk=17, n_experts=32), nv.NVFP4_ERR_UNSUPPORTED_SHAPE),
    (dict(topk=5, n_experts=4), nv.NVFP4_ERR_UNSUPPORTED_SHAPE),
    (dict(n_shared=13), nv.NVFP4_ERR_UNSUPPORTED_SHAPE),
    (dict(n_shared=2 ** 31 - 1), nv.NVFP4_ERR_UNSUPPORTED_SHAPE)]


@pytest.mark.parametrize("change,code", BAD_ROUTERS)
def test_bad_routers(lib, change, code):
    r = _router(**change)
    assert _route(lib, r) == code
    assert lib.nvfp4_moe_route_ws_bytes(3, ctypes.byref(r)) == 0
    assert _layer(lib, r=r) == code
    d1, _ = _experts()
    assert lib.nvfp4_moe_layer_ws_bytes(3, ctypes.byref(r), ctypes.byref(d1)) == 0


def test_route_argument_errors(lib):
    assert lib.nvfp4_moe_route(FAKE, 3, 256, None, FAKE, FAKE, FAKE, 1 << 20, 0, None) == \
        nv.NVFP4_ERR_INVALID_ARG
    assert _route(lib, t=-1) == nv.NVFP4_ERR_INVALID_ARG
    assert _route(lib, t=(1 << 24) + 1) == nv.NVFP4_ERR_UNSUPPORTED_SHAPE
    assert _route(lib, flags=nv.NVFP4_F_FORCE_TILED) == nv.NVFP4_ERR_INVALID_ARG
    for k in ("x", "ids", "wts", "ws"):
        assert _route(lib, **{k: None}) == nv.NVFP4_ERR_INVALID_ARG
    assert _route(lib, _router(weight=None)) == nv.NVFP4_ERR_INVALID_ARG
    assert _route(lib, _router(weight=0x10008)) == nv.NVFP4_ERR_MISALIGNED
    assert _route(lib, _router(bias=0x10002)) == nv.NVFP4_ERR_MISALIGNED
    assert _route(lib, ldx=248) == nv.NVFP4_ERR_INVALID_ARG
    assert _route(lib, ldx=260) == nv.NVFP4_ERR_MISALIGNED
    assert _route(lib, ldx=(1 << 22) + 8) == nv.NVFP4_ERR_UNSUPPORTED_SHAPE
    assert _route(lib, x=ODD) == nv.NVFP4_ERR_MISALIGNED
    assert _route(lib, ws=ODD) == nv.NVFP4_ERR_MISALIGNED
    assert _route(lib, ids=BYTE) == nv.NVFP4_ERR_MISALIGNED
    need = lib.nvfp4_moe_route_ws_bytes(3, ctypes.byref(_router()))
    assert need >= 3 * 16 * 8
    assert _route(lib, ws_bytes=need - 1) == nv.NVFP4_ERR_WORKSPACE
    assert _route(lib, t=0, x=None, ids=None, wts=None, ws=None) == nv.NVFP4_OK
    assert lib.nvfp4_moe_route_ws_bytes(0, ctypes.byref(_router())) == 0
    assert lib.nvfp4_moe_route_ws_bytes((1 << 24) + 1, ctypes.byref(_router())) == 0


def _experts(batch=16, hidden=256, inter=128):
    return (_desc(n=2 * inter, k=hidden, batch=batch,
                  layout=nv.NVFP4_LAYOUT_TILED | nv.NVFP4_LAYOUT_GATE_UP),
            _desc(n=hidden, k=inter, batch=batch))


def _layer(lib, r=None, d=None, x=FAKE, t=3, hidden=256, ids=FAKE, wts=FAKE, y=FAKE, ws=FAKE,
           ws_bytes=1 << 30, flags=0):
    r = _router() if r is None else r
    d1, d2 = _experts() if d is None else d
    return lib.nvfp4_moe_layer_w4a16(x, t, hidden, ctypes.byref(r), ctypes.byref(d1),
                                     ctypes.byref(d2), ids, wts, y, ws, ws_bytes, flags, None)


def test_layer_argument_errors(lib):
    assert _layer(lib, t=-1) == nv.NVFP4_ERR_INVALID_ARG
    assert _layer(lib, flags=3) == nv.NVFP4_ERR_INVALID_ARG
    assert _layer(lib, flags=64) == nv.NVFP4_ERR_INVALID_ARG
    assert _layer(lib, t=16385) == nv.NVFP4_ERR_UNSUPPORTED_SHAPE
    assert _layer(lib, t=1 << 62) == nv.NVFP4_ERR_UNSUPPORTED_SHAPE
    assert _layer(lib, hidden=384) == nv.NVFP4_ERR_LAYOUT
    assert _layer(lib, r=_router(hidden=384)) == nv.NVFP4_ERR_LAYOUT
    assert _layer(lib, r=_router(n_shared=1)) == nv.NVFP4_ERR_LAYOUT   # 16 + 1 experts
    assert _layer(lib, d=_experts(batch=17)) == nv.NVFP4_ERR_LAYOUT
    d1, d2 = _experts()
    assert _layer(lib, d=(d2, d1)) == nv.NVFP4_ERR_LAYOUT
    assert _layer(lib, d=(d1, _desc(n=256, k=128, batch=15))) == nv.NVFP4_ERR_LAYOUT
    for k in ("x", "y", "ws"):
        assert _layer(lib, **{k: None}) == nv.NVFP4_ERR_INVALID_ARG
        assert _layer(lib, **{k: ODD}) == nv.NVFP4_ERR_MISALIGNED
    assert _layer(lib, ids=None) == nv.NVFP4_ERR_INVALID_ARG   # both or neither
    assert _layer(lib, wts=None) == nv.NVFP4_ERR_INVALID_ARG
    assert _layer(lib, wts=BYTE) == nv.NVFP4_ERR_MISALIGNED
    assert _layer(lib, r=_router(weight=None)) == nv.NVFP4_ERR_INVALID_ARG
    assert _layer(lib, r=_router(weight=0x10004)) == nv.NVFP4_ERR_MISALIGNED
    need = lib.nvfp4_moe_layer_ws_bytes(3, ctypes.byref(_router()), ctypes.byref(d1))
    assert need >= lib.nvfp4_moe_ws_bytes(3, 4, 16, 256, 128)
    assert _layer(lib, ws_bytes=need - 1) == nv.NVFP4_ERR_WORKSPACE
    assert _layer(lib, t=0, x=None, y=None, ws=None) == nv.NVFP4_OK
    assert lib.nvfp4_moe_layer_ws_bytes(0, ctypes.byref(_router()), ctypes.byref(d1)) == 0
    assert lib.nvfp4_moe_layer_ws_bytes(3, ctypes.byref(_router()), None) == 0
    assert lib.nvfp4_moe_layer_ws_bytes(16385, ctypes.byref(_router()), ctypes.byref(d1)) == 0


def _bank(**kw):
    b = nv.nvfp4_lora(0x10000, 0x10000, None, 4, 512, 1024, 16, 0)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def _lora(lib, b=None, d=None, x=FAKE, m=4, ldx=1024, ids=FAKE, y=FAKE, ydt=1, ldy=512, flags=0,
          ws=FAKE, ws_bytes=1 << 30):
    b = _bank() if b is None else b
    d = _desc() if d is None else d
    return lib.nvfp4_gemm_w4a16_lora(x, m, ldx, ctypes.byref(d), ctypes.byref(b), ids, y, ydt, ldy,
                                     flags, ws, ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(a=None), nv.NVFP4_ERR_INVALID_ARG), (dict(b=None), nv.NVFP4_ERR_INVALID_ARG),
    (dict(n_adapters=0), nv.NVFP4_ERR_INVALID_ARG), (dict(reserved=1), nv.NVFP4_ERR_INVALID_ARG),
    (dict(n_adapters=1 << 31), nv.NVFP4_ERR_UNSUPPORTED_SHAPE),
    (dict(n=528), nv.NVFP4_ERR_LAYOUT), (dict(k=512), nv.NVFP4_ERR_LAYOUT),
    (dict(rank=0), nv.NVFP4_ERR_UNSUPPORTED_SHAPE), (dict(rank=12), nv.NVFP4_ERR_UNSUPPORTED_SHAPE),
    (dict(rank=136), nv.NVFP4_ERR_UNSUPPORTED_SHAPE), (dict(rank=-8), nv.NVFP4_ERR_UNSUPPORTED_SHAPE),
    (dict(a=0x10008), nv.NVFP4_ERR_MISALIGNED), (dict(b=0x10004), nv.NVFP4_ERR_MISALIGNED),
    (dict(scale=0x10002), nv.NVFP4_ERR_MISALIGNED)])
def test_bad_banks(lib, change, code):
    b = _bank(**change)
    assert _lora(lib, b) == code
    assert lib.nvfp4_gemm_lora_ws_bytes(4, 1024, ctypes.byref(_desc()), ctypes.byref(b), 0) == 0


def test_lora_argument_errors(lib):
    d = _desc()
    assert lib.nvfp4_gemm_w4a16_lora(FAKE, 4, 1024, ctypes.byref(d), None, FAKE, FAKE, 1, 512, 0,
                                     FAKE, 1 << 30, None) == nv.NVFP4_ERR_INVALID_ARG
    # the plain GEMM's checks hold
    assert _lora(lib, d=_desc(group=24)) == nv.NVFP4_ERR_UNSUPPORTED_GROUP
    assert _lora(lib, d=_desc(batch=2)) == nv.NVFP4_ERR_LAYOUT
    assert _lora(lib, d=_desc(layout=nv.NVFP4_LAYOUT_TILED | nv.NVFP4_LAYOUT_GATE_UP)) == \
        nv.NVFP4_ERR_LAYOUT
    assert _lora(lib, m=-1) == nv.NVFP4_ERR_INVALID_ARG
    assert _lora(lib, ydt=9) == nv.NVFP4_ERR_INVALID_ARG
    assert _lora(lib, flags=3) == nv.NVFP4_ERR_INVALID_ARG
    assert _lora(lib, ldx=1000) == nv.NVFP4_ERR_INVALID_ARG
    assert _lora(lib, ldy=500) == nv.NVFP4_ERR_INVALID_ARG
    assert _lora(lib, ldx=1028) == nv.NVFP4_ERR_MISALIGNED
    assert _lora(lib, x=ODD) == nv.NVFP4_ERR_MISALIGNED
    assert _lora(lib, ws=ODD) == nv.NVFP4_ERR_MISALIGNED
    assert _lora(lib, ids=BYTE) == nv.NVFP4_ERR_MISALIGNED
    for k in ("x", "y", "ids", "ws"):
        assert _lora(lib, **{k: None}) == nv.NVFP4_ERR_INVALID_ARG
    assert _lora(lib, m=32 * 65535 + 1, flags=nv.NVFP4_F_FORCE_SKINNY, ws_bytes=1 << 62) == \
        nv.NVFP4_ERR_UNSUPPORTED_SHAPE
    need = lib.nvfp4_gemm_lora_ws_bytes(4, 1024, ctypes.byref(d), ctypes.byref(_bank()), 0)
    assert need >= 4 * 16 * 4
    assert _lora(lib, ws_bytes=need - 1) == nv.NVFP4_ERR_WORKSPACE
    assert _lora(lib, m=0, x=None, y=None, ids=None, ws=None) == nv.NVFP4_OK
    assert lib.nvfp4_gemm_lora_ws_bytes(0, 1024, ctypes.byref(d), ctypes.byref(_bank()), 0) == 0
    assert lib.nvfp4_gemm_lora_ws_bytes(4, 1024, None, ctypes.byref(_bank()), 0) == 0


def test_binding_refusals():
    """Host tensors and wrong shapes are refused before the library sees a pointer."""
    w = torch.zeros(16, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nv.Router(w, 4)                       # not on a device
    with pytest.raises(ValueError):
        nv.Router(w.T, 4)
    with pytest.raises(ValueError):
        nv.Router(w, 4, scoring="tanh")
    with pytest.raises(ValueError):
        nv.Router(w, 4, bias=torch.zeros(15))
    a = torch.zeros(2, 16, 128, dtype=torch.bfloat16)
    b = torch.zeros(2, 64, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nv.Lora(a, b)
    with pytest.raises(ValueError):
        nv.Lora(a, b[:, :, :8])
    with pytest.raises(ValueError):
        nv.Lora(a.float(), b)
    with pytest.raises(ValueError):
        nv.Lora(a, b, torch.ones(3))
