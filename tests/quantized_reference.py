"""The 8-bit rows' definition on the CPU: float32 steps as stated in the header, everything else in 64 bits."""
import numpy as np
import torch

from oracle import mxfp8

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SMALLEST = 2.0 ** -126


def to_type(v, t):
    """Nearest value of a type; fp16 saturates (NaN stays)."""
    return (v.clamp(-65504, 65504) if t == torch.float16 else v).to(t)


def placed(v, pad=0, offset=0, junk=float("nan")):
    """v [rows, n] on the GPU inside a buffer of junk: rows n + pad apart, `offset` elements in.  Returns (view, buffer)."""
    rows, n = v.shape
    buf = torch.full((offset + rows * (n + pad) + 8,), junk, dtype=v.dtype, device="cuda")
    at = buf[offset: offset + rows * (n + pad)].view(rows, n + pad)[:, :n]
    at.copy_(v)
    return at, buf


def around(buf, view, junk):
    """Whether everything of buf but view still holds junk."""
    rest = buf.clone()
    rest.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(junk)
    return bool((rest == junk).all())


def normed(x, residual, weight, eps):
    """(h, v float32, v in 64 bits) of CPU rows."""
    h = x if residual is None else to_type(x.float() + residual.float(), residual.dtype)
    d = h.double()
    s = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    v = h.float() * s.float()
    exact = d * s
    if weight is not None:
        v, exact = v * weight.float(), exact * weight.double()
    return h, v, exact


def int8_rows(v, dim=1):
    """(codes, scales) of float32 rows (dim 0: columns) by the rule, the quotients in 64 bits: 24-bit numbers whose quotient
    is not half an integer differ from one by 2^-33 relatively, which a double resolves."""
    most = v.abs().amax(dim, keepdim=True)
    scale = torch.clamp((most.double() / 127).float(), min=SMALLEST)
    codes = torch.round(v.double() / scale.double()).clamp(-127, 127)
    bad = ~torch.isfinite(v).all(dim, keepdim=True)
    codes = torch.where(bad, torch.zeros_like(codes), codes).to(torch.int8)
    return codes, torch.where(bad, torch.full_like(scale, float("nan")), scale).squeeze(dim)


def mx_rows(v):
    """(codes, scale bytes) of float32 rows: the MXFP8 oracle's, NaN where a block is not finite."""
    b = v.reshape(v.shape[0], -1, 32)
    bad = ~torch.isfinite(b).all(2)
    clean = torch.where(bad[..., None], torch.zeros_like(b), b).reshape(v.shape)
    codes, scales = mxfp8.quantize(clean.numpy().astype(np.float64))
    codes = torch.from_numpy(codes.astype(np.uint8)).reshape(b.shape)
    scales = torch.from_numpy(scales.astype(np.uint8)).reshape(bad.shape)
    codes = torch.where(bad[..., None], torch.full_like(codes, 0x7F), codes).reshape(v.shape)
    return codes, torch.where(bad, torch.full_like(scales, 255), scales)
