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
from .binding import MOE_BF16, MOE_EPI_NONE, MOE_F16, MOE_F32, MOE_I8, MOE_MXFP8, DenseShape

__all__ = ["MOE_I8", "MOE_MXFP8", "moe_add_rmsnorm", "moe_quantize_int8", "moe_packed_dense_bytes_int8",
           "moe_pack_dense_int8", "moe_dense_gemm_int8"]


# Argument checks as binding's, with fewer calls into torch: a decode step's kernels are shorter than a careful call.

_DTYPES = {torch.bfloat16: MOE_BF16, torch.float16: MOE_F16, torch.float32: MOE_F32}
_CODES = {MOE_I8: torch.int8, MOE_MXFP8: torch.uint8}
# bound once; a torch without a GPU has neither, and no call there gets past the check of its first tensor
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _dt(t: torch.Tensor) -> int:
    code = _DTYPES.get(t.dtype)
    return _b._dt(t) if code is None else code         # which refuses it


def _rows(t: torch.Tensor, shape, index: int, name: str):
    """(pointer, row stride) of a tensor of `shape`, (rows, n), on GPU `index` whose rows are contiguous."""
    if t.shape == shape and t.get_device() == index:
        if t.is_contiguous():
            return t.data_ptr() or None, shape[1]
        ld, one = t.stride()
        if one == 1 and ld >= shape[1]:
            return t.data_ptr() or None, ld
    r = _b._rows(t, shape[0], shape[1], name)          # which says what is wrong
    _b._same_device(torch.device("cuda", index), **{name: t})
    return r


def _flat(t: torch.Tensor, dtype, n: int, index: int, name: str):
    """Pointer of n contiguous elements on GPU `index`."""
    if t.dtype == dtype and t.numel() == n and t.get_device() == index and t.is_contiguous():
        return t.data_ptr() or None
    r = _b._ptr(t, dtype, n, name)
    _b._same_device(torch.device("cuda", index), **{name: t})
    return r


def _index(t: torch.Tensor, name: str) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    return index


def _stream(index: int, stream):
    if stream is None and _current_device() == index:
        return _current_stream(index) or None
    return _b._stream_on(torch.device("cuda", index), stream)


def moe_add_rmsnorm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                    eps: float = 1e-6, *, sum_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                    y_dtype: Optional[torch.dtype] = None, codes: Optional[torch.Tensor] = None,
                    scales: Optional[torch.Tensor] = None, q_dtype: Optional[int] = None, stream=None):
    """The norm of h = x + residual (rounded to the residual's type; x without one), rows of [rows, H].

    Returns (h, y, codes, scales).  y is computed where y or y_dtype is given, codes and scales where q_dtype is:
    MOE_I8 (int8 [rows, H], float32 [rows]) or MOE_MXFP8 (uint8 [rows, H], uint8 [rows, H/32]); with none of them y is
    computed in x's type.  sum_out receives h and may be residual or x, y may be x or residual (not both the same).
    x, residual, sum_out, y and codes may have any row stride."""
    shape = x.shape
    rows, H = shape
    index = _index(x, "x")
    pr = pt = pw = py = pq = ps = None
    rd = wd = yd = MOE_F32
    ldr = lds = ldy = ldq = 0
    if residual is not None:
        if sum_out is None:
            sum_out = _b._empty((rows, H), residual.dtype, x.device, stream)
        elif sum_out.dtype != residual.dtype:
            raise TypeError(f"sum_out is {sum_out.dtype}, the residual {residual.dtype}")
        rd = _dt(residual)
        pr, ldr = _rows(residual, shape, index, "residual")
        pt, lds = _rows(sum_out, shape, index, "sum_out")
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    if weight is not None:
        wd = _dt(weight)
        pw = _flat(weight, weight.dtype, H, index, "weight")
    if y is not None:
        if y_dtype is not None and y.dtype != y_dtype:
            raise TypeError(f"y is {y.dtype}, y_dtype {y_dtype}")
    elif y_dtype is not None or q_dtype is None:
        y = _b._empty((rows, H), y_dtype or x.dtype, x.device, stream)
    if y is not None:
        yd = _dt(y)
        py, ldy = _rows(y, shape, index, "y")
    if q_dtype is not None:
        kind = _CODES.get(q_dtype)
        if kind is None:
            raise ValueError("q_dtype is MOE_I8 or MOE_MXFP8")
        int8 = q_dtype == MOE_I8
        if codes is None:
            codes = _b._empty((rows, H), kind, x.device, stream)
        elif codes.dtype != kind:
            raise TypeError(f"codes must be {kind}, got {codes.dtype}")
        if scales is None:
            scales = _b._empty((rows,) if int8 else (rows, H // 32), torch.float32 if int8 else torch.uint8, x.device,
                               stream)
        pq, ldq = _rows(codes, shape, index, "codes")
        ps = _flat(scales, torch.float32 if int8 else torch.uint8, rows if int8 else rows * (H // 32), index, "scales")
    elif codes is not None or scales is not None:
        raise ValueError("codes and scales need a q_dtype")
    px, ldx = _rows(x, shape, index, "x")
    st = _b.load().moe_add_rmsnorm(rows, H, px, _dt(x), ldx, pr, rd, ldr, pt, lds, pw, wd, eps, py, yd, ldy, pq,
                                   q_dtype or 0, ldq, ps, _stream(index, stream))
    if st:
        _b._check("moe_add_rmsnorm", st)
    return x if residual is None else sum_out, y, codes, scales


def moe_quantize_int8(x: torch.Tensor, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                      stream=None):
    """x [rows, K], any row stride, fp32, bf16 or fp16 -> (codes int8 [rows, K], scales float32 [rows])."""
    shape = x.shape
    rows, K = shape
    index = _index(x, "x")
    if codes is None:
        codes = _b._empty((rows, K), torch.int8, x.device, stream)
    elif codes.dtype != torch.int8:
        raise TypeError(f"codes must be int8, got {codes.dtype}")
    if scales is None:
        scales = _b._empty((rows,), torch.float32, x.device, stream)
    px, ldx = _rows(x, shape, index, "x")
    pq, ldq = _rows(codes, shape, index, "codes")
    st = _b.load().moe_quantize_int8(rows, K, px, _dt(x), ldx, pq, ldq, _flat(scales, torch.float32, rows, index, "scales"),
                                     _stream(index, stream))
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
    cshape, need = _dense_int8_of(d)
    M, N = d.M, d.N
    index = _index(a, "a")
    if a.dtype != torch.int8:
        raise TypeError(f"a must be int8, got {a.dtype}")
    size = packed.numel()
    if size < need:
        raise ValueError(f"packed must hold {need} bytes, got {size}")
    if c is None:
        c = _b._empty((M, N), c_dtype or torch.bfloat16, a.device, stream)
    elif c_dtype is not None and c.dtype != c_dtype:
        raise TypeError(f"c is {c.dtype}, c_dtype {c_dtype}")
    pb = pr = None
    rd, ldr = MOE_F32, 0
    if bias is not None:
        pb = _flat(bias, torch.float32, 2 * N if d.gated else N, index, "bias")
    if residual is not None:
        rd = _dt(residual)
        pr, ldr = _rows(residual, (M, N), index, "residual")
    pa, lda = _rows(a, (M, d.K), index, "a")
    pc, ldc = _rows(c, (M, N), index, "c")
    st = _b.load().moe_dense_gemm_int8(cshape, pa, lda, _flat(a_scales, torch.float32, M, index, "a_scales"),
                                       _flat(packed, torch.uint8, size, index, "packed"), epilogue, pb, pr, rd, ldr, pc,
                                       _dt(c), ldc, _stream(index, stream))
    if st:
        _b._check("moe_dense_gemm_int8", st)
    return c
