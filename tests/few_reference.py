"""The few-token layer and its inputs in 64 bits, from the definition (torch on the CPU or the GPU)."""
import math

import torch

from moe_layer_03_amd import binding as B


def make(s, dtype="bf16", mx=False, seed=0, bias=False, device="cuda", std=0.02):
    """Inputs of a layer share: float32 layers' weights are fp16 values, MXFP8 layers' weights MXFP8 values."""
    g = torch.Generator().manual_seed(seed)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    n = s.E_loc

    def weights(rows, cols):
        v = torch.randn((n, rows, cols), generator=g) * std
        if mx:
            b = v.view(n, rows // 32, 32, cols)
            scale = torch.exp2(torch.floor(torch.log2(b.abs().amax(2, keepdim=True))) - 8)
            return ((b / scale).clamp(-448, 448).to(torch.float8_e4m3fn).float() * scale).view(n, rows, cols)
        return v.bfloat16().float() if dtype == "bf16" else v.half().float()

    d = dict(x=torch.randn((s.T, s.H), generator=g).to(t), w_router=(torch.randn((s.H, s.E), generator=g) * 0.02).to(t),
             bias=torch.randn(s.E, generator=g) * 0.5 if bias else None,
             gate=weights(s.H, s.I), up=weights(s.H, s.I), down=weights(s.I, s.H))
    return {k: v if v is None else v.to(device) for k, v in d.items()}


def pack(s, d, dtype="bf16", mx=False):
    w = [d[k] if dtype == "f32" and not mx else d[k].bfloat16() for k in ("gate", "up", "down")]
    return (B.moe_pack_weights_mxfp8 if mx else B.moe_pack_weights)(s, *w)


def reference(s, d):
    """(out, topk_idx, topk_w, bound): bound is the largest error float32 accumulation can leave, per element.

    A float32 sum of n products in any order is off by at most n u sum|products| (u = 2^-24).  With G = |x||Wg| and
    U = |x||Wu| the gate and up sums are off by H u G and H u U; silu has slope at most 1.1 and, from expf and a
    division, 4 u of its own; the rows are kept to 2^-22; the down product adds I K u of its absolute sum."""
    x = d["x"].double()
    logits = x @ d["w_router"].double()
    if d["bias"] is not None:
        logits = logits + d["bias"].double()
    out = torch.zeros((s.T, s.H), dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(out)
    idx = torch.empty((s.T, s.K), dtype=torch.int64)
    w = torch.empty((s.T, s.K), dtype=torch.float64)
    u = 2.0 ** -24
    for t, row in enumerate(logits.tolist()):
        pick = sorted(range(s.E), key=lambda e: (-row[e], e))[: s.K]
        ex = [math.exp(row[e] - row[pick[0]]) for e in pick]
        for j, e in enumerate(pick):
            idx[t, j], w[t, j] = e, ex[j] / math.fsum(ex)
            if not s.e_begin <= e < s.e_end:
                continue
            wg, wu, wd = (d[k][e - s.e_begin].double() for k in ("gate", "up", "down"))
            a, b = x[t] @ wg, x[t] @ wu
            sg = a * torch.sigmoid(a)
            da, db = s.H * u * (x[t].abs() @ wg.abs()), s.H * u * (x[t].abs() @ wu.abs())
            h = w[t, j] * sg * b
            dh = w[t, j] * (1.1 * da * b.abs() + sg.abs() * db + 1.1 * da * db) + (12 * u + 2.0 ** -22) * h.abs() + 2.0 ** -35
            out[t] += h @ wd
            bound[t] += (dh @ wd.abs()) + (s.I * s.K * u) * (h.abs() @ wd.abs())
    return out, idx, w, bound


def check(s, d, got, idx, w, rms=3e-6):
    """out within the bound everywhere, and within rms of its RMS: random rounding of the longest float32 chain here
    (512 additions in a wave) leaves 0.6 u sqrt(512) = 8e-7 per product, of which there are three, doubled."""
    ref, ridx, rw, bound = reference(s, d)
    assert torch.equal(idx.cpu().long(), ridx)
    assert (w.cpu().double() - rw).abs().max().item() <= 1e-6 if rw.numel() else True
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    assert (err <= bound).all(), f"largest error {err.max().item():.3e} over its bound by {(err - bound).max().item():.3e}"
    size = ref.pow(2).mean().sqrt().item()
    assert err.pow(2).mean().sqrt().item() <= rms * size
    none = ~((ridx >= s.e_begin) & (ridx < s.e_end)).any(1)
    assert (got[none.to(got.device)] == 0).all()
