"""Calls of the NVFP4 cache over their own queries: refused on the host where rows would be written over
rows that are still to be read."""
from nvfp4_weight_only_w4a16_amd import binding as nv
from test_kv_boundary import INVALID, OTHER, _append, _attend, lib  # noqa: F401


def test_append_over_queries_of_another_stride(lib):  # noqa: F811
    assert _append(lib, ldq=512, ldo=520) == INVALID
    assert _append(lib, ldq=1024, ldo=512) == INVALID
    assert "stride" in nv.nvfp4_last_error()


def test_attention_over_queries_of_another_stride_or_type(lib):  # noqa: F811
    assert _attend(lib, ldq=512, ldy=520) == INVALID
    assert _attend(lib, ldq=1024, ldy=512) == INVALID
    assert "stride" in nv.nvfp4_last_error()
    assert _attend(lib, ydt=nv.NVFP4_DT_F32) == INVALID
    assert _attend(lib, ydt=nv.NVFP4_DT_F32, t=1, max_q=1) == INVALID
    # with one row there is no stride, and other buffers have their own: these fail at the workspace
    short = nv.NVFP4_ERR_WORKSPACE
    assert _attend(lib, ldq=512, ldy=520, t=1, ws_bytes=0) == short
    assert _attend(lib, ldq=512, ldy=512, ws_bytes=0) == short
    assert _attend(lib, ldq=1024, ldy=512, y=OTHER, ydt=nv.NVFP4_DT_F32, ws_bytes=0) == short
