"""8-bit rows and their products: the norm that writes them, the int8 quantiser and the int8 dense product.

The second part of the ctypes binding, in the manner of ``binding``: functions carry the C names, take torch tensors
on the GPU, pass their pointers and the current HIP stream and raise ``MoeError`` on a non-zero status; what the caller
does not pass is allocated on the call's stream.  A decoder block's feed-forward half with a shared expert in int8::

    h, y, codes, scales = moe_add_rmsnorm(attn, weight, h, q_dtype=MOE_I8, y_dtype=torch.bfloat16)
    out = binding.moe_layer(shape, y, w_router, experts)
    g = moe_dense_gemm_int8(gate_up, codes, scales, packed_gate_up, MOE_EPI_SWIGLU)
    moe_dense_gemm_int8(down, *moe_quantize_int8(g), packed_down, residual=out, c=out)
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import binding as _b
from .binding import MOE_EPI_NONE, MOE_F32, MOE_I8, MOE_MXFP8, DenseShape

__all__ = ["MOE_I8", "MOE_MXFP8", "moe_add_rmsnorm", "moe_quantize_int8", "moe_packed_dense_bytes_int8",
           "moe_pack_dense_int8", "moe_dense_gemm_int8"]


def moe_add_rmsnorm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                    eps: float = 1e-6, *, sum_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                    y_dtype: Optional[torch.dtype] = None, codes: Optional[torch.Tensor] = None,
                    scales: Optional[torch.Tensor] = None, q_dtype: Optional[int] = None, stream=None):
    """The norm of h = x + residual (rounded to the residual's type; x without one), rows of [rows, H].

    Returns (h, y, codes, scales).  y is computed where y or y_dtype is given, codes and scales where q_dtype is:
    MOE_I8 (int8 [rows, H], float32 [rows]) or MOE_MXFP8 (uint8 [rows, H], uint8 [rows, H/32]); with none of them y is
    computed in x's type.  sum_out receives h and may be residual or x."""
    rows, H = x.shape
    dev = x.device
    if y is not None and y_dtype is not None and y.dtype != y_dtype:
        raise TypeError(f"y is {y.dtype}, y_dtype {y_dtype}")
    if q_dtype is None and (codes is not None or scales is not None):
        raise ValueError("codes and scales need a q_dtype")
    if q_dtype not in (None, MOE_I8, MOE_MXFP8):
        raise ValueError("q_dtype is MOE_I8 or MOE_MXFP8")
    if residual is None:
        if sum_out is not None:
            raise ValueError("sum_out needs a residual")
    elif sum_out is None:
        sum_out = _b._empty((rows, H), residual.dtype, dev, stream)
    elif sum_out.dtype != residual.dtype:
        raise TypeError(f"sum_out is {sum_out.dtype}, the residual {residual.dtype}")
    if y is None and (y_dtype is not None or q_dtype is None):
        y = _b._empty((rows, H), y_dtype or x.dtype, dev, stream)
    pq = ps = None
    ldq = 0
    if q_dtype is not None:
        int8 = q_dtype == MOE_I8
        if codes is None:
            codes = _b._empty((rows, H), torch.int8 if int8 else torch.uint8, dev, stream)
        if scales is None:
            scales = _b._empty((rows,) if int8 else (rows, H // 32), torch.float32 if int8 else torch.uint8, dev, stream)
        if codes.dtype != (torch.int8 if int8 else torch.uint8):
            raise TypeError(f"codes must be {'int8' if int8 else 'uint8'}, got {codes.dtype}")
        pq, ldq = _b._rows(codes, rows, H, "codes")
        ps = _b._ptr(scales, torch.float32 if int8 else torch.uint8, rows if int8 else rows * (H // 32), "scales")
    px, ldx = _b._rows(x, rows, H, "x")
    pr, ldr = _b._rows(residual, rows, H, "residual")
    pt, lds = _b._rows(sum_out, rows, H, "sum_out")
    py, ldy = _b._rows(y, rows, H, "y")
    args = (rows, H, px, _b._dt(x), ldx, pr, _b._dt(residual) if residual is not None else MOE_F32, ldr, pt, lds,
            _b._ptr(weight, None, H, "weight"), _b._dt(weight) if weight is not None else MOE_F32, eps, py,
            _b._dt(y) if y is not None else MOE_F32, ldy, pq, q_dtype or 0, ldq, ps)
    _b._same_device(dev, residual=residual, sum_out=sum_out, weight=weight, y=y, codes=codes, scales=scales)
    st = _b.load().moe_add_rmsnorm(*args, _b._stream_on(dev, stream))
    if st:
        _b._check("moe_add_rmsnorm", st)
    return x if residual is None else sum_out, y, codes, scales


def moe_quantize_int8(x: torch.Tensor, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                      stream=None):
    """x [rows, K], any row stride, fp32, bf16 or fp16 -> (codes int8 [rows, K], scales float32 [rows])."""
    rows, K = x.shape
    dev = x.device
    if codes is None:
        codes = _b._empty((rows, K), torch.int8, dev, stream)
    if scales is None:
        scales = _b._empty((rows,), torch.float32, dev, stream)
    if codes.dtype != torch.int8:
        raise TypeError(f"codes must be int8, got {codes.dtype}")
    px, ldx = _b._rows(x, rows, K, "x")
    pq, ldq = _b._rows(codes, rows, K, "codes")
    args = (rows, K, px, _b._dt(x), ldx, pq, ldq, _b._ptr(scales, torch.float32, rows, "scales"))
    _b._same_device(dev, codes=codes, scales=scales)
    st = _b.load().moe_quantize_int8(*args, _b._stream_on(dev, stream))
    if st:
        _b._check("moe_quantize_int8", st)
    return codes, scales


@functools.lru_cache(maxsize=256)
def _dense_int8_of(d: DenseShape):
    """(C shape, packed bytes) of a shape."""
    c = d.c()
    return c, int(_b.load().moe_packed_dense_bytes_int8(c))


def moe_packed_dense_bytes_int8(d: DenseShape) -> int:
    return _dense_int8_of(d)[1]


def moe_pack_dense_int8(d: DenseShape, w: torch.Tensor, w_up: Optional[torch.Tensor] = None, *,
                        scales: Optional[torch.Tensor] = None, up_scales: Optional[torch.Tensor] = None,
                        packed: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Pack w [K, N] (gated: the gate weight, with w_up [K, N]): int8 codes with scales [N] (up_scales), or fp32, bf16
    or fp16 weights, quantised per column here; M does not matter."""
    need = moe_packed_dense_bytes_int8(d)
    if packed is None:
        packed = _b._empty(max(need, 16), torch.uint8, w.device, stream)
    if packed.dtype != torch.uint8 or packed.numel() < need:
        raise ValueError(f"packed must be a uint8 buffer of at least {need} bytes")
    n = d.N * d.K
    _b._same_device(w.device, w_up=w_up, scales=scales, up_scales=up_scales, packed=packed)
    args = (ctypes.byref(d.c()), _b._ptr(w, None, n, "w"), _b._ptr(w_up, w.dtype, n, "w_up"),
            MOE_I8 if w.dtype == torch.int8 else _b._dt(w), _b._ptr(scales, torch.float32, d.N, "scales"),
            _b._ptr(up_scales, torch.float32, d.N, "up_scales"), _b._ptr(packed, torch.uint8, None, "packed"))
    _b._check("moe_pack_dense_int8", _b.load().moe_pack_dense_int8(*args, _b._stream_on(w.device, stream)))
    return packed


def moe_dense_gemm_int8(d: DenseShape, a: torch.Tensor, a_scales: torch.Tensor, packed: torch.Tensor,
                        epilogue: int = MOE_EPI_NONE, *, bias: Optional[torch.Tensor] = None,
                        residual: Optional[torch.Tensor] = None, c: Optional[torch.Tensor] = None,
                        c_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """act((a @ W) * a_scales * scales + bias) + residual on moe_pack_dense_int8 weights (gated: MOE_EPI_SWIGLU,
    bias [2, N]).

    a [M, K] int8, residual and c [M, N] may have any row stride; c may be residual.  c_dtype is c's, or bfloat16."""
    shape, need = _dense_int8_of(d)
    if packed.numel() < need:
        raise ValueError(f"packed must hold {need} bytes, got {packed.numel()}")
    dev = a.device
    if a.dtype != torch.int8:
        raise TypeError(f"a must be int8, got {a.dtype}")
    if c is None:
        c = _b._empty((d.M, d.N), c_dtype or torch.bfloat16, dev, stream)
    elif c_dtype is not None and c.dtype != c_dtype:
        raise TypeError(f"c is {c.dtype}, c_dtype {c_dtype}")
    pa, lda = _b._rows(a, d.M, d.K, "a")
    pr, ldr = _b._rows(residual, d.M, d.N, "residual")
    pc, ldc = _b._rows(c, d.M, d.N, "c")
    args = (shape, pa, lda, _b._ptr(a_scales, torch.float32, d.M, "a_scales"),
            _b._ptr(packed, torch.uint8, None, "packed"), epilogue,
            _b._ptr(bias, torch.float32, d.N * (2 if d.gated else 1), "bias"), pr,
            _b._dt(residual) if residual is not None else MOE_F32, ldr, pc, _b._dt(c), ldc)
    _b._same_device(dev, a_scales=a_scales, packed=packed, bias=bias, residual=residual, c=c)
    st = _b.load().moe_dense_gemm_int8(*args, _b._stream_on(dev, stream))
    if st:
        _b._check("moe_dense_gemm_int8", st)
    return c
