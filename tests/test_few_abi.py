"""The few-token layer's refusals, on the host before any HIP call (no GPU needed)."""
import ctypes

import pytest
import torch

from moe_layer_03_amd import binding as B

P16, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1002)


def _shape(**kw):
    base = dict(T=8, H=256, E=8, K=2, I=256, e_begin=0, e_end=8)
    base.update(kw)
    return B.Shape(**base)


def _call(s, mx=False, x=P16, xd=B.MOE_BF16, wr=P16, wd=B.MOE_BF16, bias=None, packed=P16, out=P16, idx=None, w=None,
          ws=P16, ws_bytes=1 << 40):
    f = B.load().moe_layer_few_tokens_mxfp8 if mx else B.load().moe_layer_few_tokens
    return f(ctypes.byref(s.c()), x, xd, wr, wd, bias, packed, out, idx, w, ws, ws_bytes, None)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), B.MOE_ERR_INVALID_ARG),
    (dict(K=9), B.MOE_ERR_INVALID_ARG),
    (dict(e_begin=4, e_end=4), B.MOE_ERR_INVALID_ARG),
    (dict(H=100), B.MOE_ERR_UNSUPPORTED),
    (dict(E=128, K=65, e_end=128), B.MOE_ERR_UNSUPPORTED),
    (dict(T=B.MOE_FEW_TOKENS_MAX + 1), B.MOE_ERR_UNSUPPORTED),
    (dict(T=32, K=8, I=256 * 6000), B.MOE_ERR_UNSUPPORTED),      # 3 parts of T K I 16-bit values past 2 GiB
    (dict(T=32, H=256 * 50000), B.MOE_ERR_UNSUPPORTED),
])
def test_shapes(mx, kw, status):
    s = _shape(**kw)
    assert _call(s, mx) == status
    query = B.moe_layer_few_tokens_workspace_bytes_mxfp8 if mx else B.moe_layer_few_tokens_workspace_bytes
    assert query(s) == 0


def test_mxfp8_needs_multiples_of_256():
    s = _shape(H=320)
    assert B.moe_layer_few_tokens_workspace_bytes(s) > 0
    assert B.moe_layer_few_tokens_workspace_bytes_mxfp8(s) == 0
    assert _call(s, True) == B.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("mx", [False, True])
def test_pointers_types_and_workspace(mx):
    s = _shape()
    need = B.moe_layer_few_tokens_workspace_bytes(s)
    assert _call(s, mx, ws_bytes=need - 1) == B.MOE_ERR_WORKSPACE
    assert _call(s, mx, xd=B.MOE_F16, wd=B.MOE_F16) == B.MOE_ERR_UNSUPPORTED
    assert _call(s, mx, wd=B.MOE_F32) == B.MOE_ERR_UNSUPPORTED
    for name in ("x", "wr", "packed", "out", "ws"):
        assert _call(s, mx, **{name: None}) == B.MOE_ERR_INVALID_ARG, name
        assert _call(s, mx, **{name: ODD}) == B.MOE_ERR_INVALID_ARG, name
    for name in ("bias", "idx", "w"):
        assert _call(s, mx, **{name: ODD}) == B.MOE_ERR_INVALID_ARG, name


def test_no_tokens_is_a_no_op():
    assert _call(_shape(T=0), x=None, out=None, packed=None, wr=None) == B.MOE_OK


def test_workspace_grows_with_tokens():
    sizes = [B.moe_layer_few_tokens_workspace_bytes(_shape(T=t)) for t in (1, 4, 16, 32)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def test_binding_refuses_host_tensors():
    s = _shape()
    x = torch.zeros((s.T, s.H), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.moe_layer_few_tokens(s, x, torch.zeros((s.H, s.E), dtype=torch.bfloat16), torch.zeros(8, dtype=torch.uint8))
