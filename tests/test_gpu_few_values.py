"""The few-token layer's digits: rows far below and above one, NaN of every payload."""
import math

import pytest
import torch

from few_reference import make, pack
from moe_layer_03_amd import binding as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def reference(s, d, parts):
    """(out, bound, spread) in 64 bits; bound is the largest error that float32 accumulation and the rows' parts can
    leave, spread a token's largest difference of logits between its first and a local expert.

    A float32 sum of n products in any order is off by at most n u sum|products|.  silu has slope at most 1.1; expf
    (2 u), its sum, the division and three products leave 8 u of a row's value; the weight of a logit d below the first
    (d + K + 6) u: d rounded to float32, expf, a sum of K (whose own d exp(-d) is at most 0.37 each) and a division.
    Two fp16 parts of a row scaled to a largest value in [2^14, 2^15) (x) or [2^-9, 2^15) (the down step's input) hold
    each value to 2^-22 of it plus 2^-36, that is 2^-50 or 2^-27 of the token's largest; three bf16 parts to 2^-24."""
    x = d["x"].double()
    f32 = d["x"].dtype == torch.float32
    logits = x @ d["w_router"].double()
    if d["bias"] is not None:
        logits = logits + d["bias"].double()
    xa = x.abs()
    dx = torch.zeros_like(x)
    if f32:
        dx = 2.0 ** -24 * xa if parts == 3 else 2.0 ** -22 * xa + 2.0 ** -50 * xa.amax(1, keepdim=True)
    out = torch.zeros((s.T, s.H), dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(out)
    spread = torch.zeros(s.T, dtype=torch.float64, device=x.device)
    for t, row in enumerate(logits.tolist()):
        pick = sorted(range(s.E), key=lambda e: (-row[e], e))[: s.K]
        ex = [math.exp(row[e] - row[pick[0]]) for e in pick]
        rows = []
        for j, e in enumerate(pick):
            if not s.e_begin <= e < s.e_end:
                continue
            wg, wu, wd = (d[k][e - s.e_begin].double() for k in ("gate", "up", "down"))
            a, b = x[t] @ wg, x[t] @ wu
            sg, w = a * torch.sigmoid(a), ex[j] / math.fsum(ex)
            da = s.H * U * (xa[t] @ wg.abs()) + dx[t] @ wg.abs()
            db = s.H * U * (xa[t] @ wu.abs()) + dx[t] @ wu.abs()
            h = w * sg * b
            dh = w * (1.1 * da * b.abs() + sg.abs() * db + 1.1 * da * db) + (
                (14 + s.K + row[pick[0]] - row[e]) * U + 2.0 ** -22) * h.abs()
            rows.append((h, dh, wd))
            spread[t] = max(spread[t].item(), row[pick[0]] - row[e])
        top = max((h.abs().max().item() for h, _, _ in rows), default=0.0)
        for h, dh, wd in rows:
            dh = dh + (2.0 ** -27 * top if parts == 2 else 0)
            out[t] += h @ wd
            bound[t] += dh @ wd.abs() + s.I * s.K * U * (h.abs() @ wd.abs())
    return out, bound, spread


def call(s, d, packed, mx=False, **kw):
    ws = torch.full((B.moe_layer_few_tokens_workspace_bytes(s),), 0xFF, dtype=torch.uint8, device="cuda")
    f = B.moe_layer_few_tokens_mxfp8 if mx else B.moe_layer_few_tokens
    got = f(s, d["x"], d["w_router"], packed, d["bias"], ws=ws, **kw)
    torch.cuda.synchronize()
    return got


def check(s, d, got, parts, rms=3e-6):
    """Within the bound everywhere, and every token within rms of its own RMS (and its weights' error), however small
    that is: random rounding of the longest float32 chain (512 additions) leaves 8e-7 in each of three products."""
    ref, bound, spread = reference(s, d, parts)
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    assert (err <= bound + 2.0 ** -148).all(), f"{(err / bound.clamp(min=1e-300)).max().item():.3g} of the bound"
    size = ref.pow(2).mean(1).sqrt()
    assert (err.pow(2).mean(1).sqrt() <= (rms + spread * U) * size + 2.0 ** -148).all()


SHAPES = [(1, 64, 4, 1, 64, 0, 4), (3, 256, 16, 4, 256, 2, 14), (8, 512, 64, 8, 256, 0, 64),
          (13, 256, 32, 4, 512, 0, 32), (20, 256, 8, 4, 256, 0, 8), (32, 512, 128, 8, 256, 16, 100)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("std", [1e-2, 1e-3, 1e-4, 1e-7, 1e-12, 30.0])
def test_rows_of_any_size(shape, dtype, std):
    """x of std 1e-12 makes rows of 1e-25 and smaller."""
    s = B.Shape(*shape)
    d = make(s, dtype, seed=70 + s.T)
    d["x"] = (d["x"].float() * std).to(d["x"].dtype)
    check(s, d, call(s, d, pack(s, d, dtype)), 2)


@pytest.mark.parametrize("T", [1, 7, 12, 32])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_every_size_together(T, dtype):
    """A call whose tokens lie 2^46 apart, a zero row among them, and experts whose weights shrink their rows."""
    s = B.Shape(T, 256, 24, 4, 256, 1, 23)
    d = make(s, dtype, seed=80 + T, bias=True)
    scale = torch.tensor([2.0 ** -(7 * t % 47) for t in range(T)], device="cuda")[:, None]
    if T > 3:
        scale[3] = 0.0
    d["x"] = (d["x"].float() * scale).to(d["x"].dtype)
    d["up"][5:9] = (d["up"][5:9] * 2.0 ** -6).to(torch.float16 if dtype == "f32" else torch.bfloat16).float()
    check(s, d, call(s, d, pack(s, d, dtype)), 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_large_value_in_a_small_row(dtype):
    """One large x in a row of small ones, and one expert's row far above the others of its token."""
    s = B.Shape(6, 512, 16, 4, 256, 0, 16)
    d = make(s, dtype, seed=90)
    x = d["x"].float() * 1e-5
    x[:, 17] = 100.0
    d["x"] = x.to(d["x"].dtype)
    check(s, d, call(s, d, pack(s, d, dtype)), 2)
    d = make(s, dtype, seed=91)
    d["bias"] = torch.linspace(0, 8, 16, device="cuda")      # routing weights from 1 to e^-8
    check(s, d, call(s, d, pack(s, d, dtype)), 2)


def test_fewest_levels():
    """So many rows that only the unscaled ones fit below 2 GiB."""
    s = B.Shape(32, 64, 64, 64, 134400, 0, 2)
    d = make(s, seed=92)
    check(s, d, call(s, d, pack(s, d)), 2)


def test_scaled_rows_up_to_2_gib():
    """Scaled rows whose offsets come near the end of the range."""
    s = B.Shape(32, 64, 64, 64, 44800, 0, 2)
    d = make(s, seed=93)
    d["x"] = (d["x"].float() * 1e-12).bfloat16()
    check(s, d, call(s, d, pack(s, d)), 2)


@pytest.mark.parametrize("std", [1e-3, 1e-7, 30.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_mxfp8_rows_of_any_size(std, dtype):
    s = B.Shape(9, 512, 24, 4, 256, 0, 20)
    d = make(s, dtype, mx=True, seed=95)
    d["x"] = (d["x"].float() * std).to(d["x"].dtype)
    check(s, d, call(s, d, pack(s, d, dtype, True), True), 3)


def test_mxfp8_largest_float32_row():
    """x at float32's largest number, beside weights that bring it back."""
    s = B.Shape(2, 256, 4, 1, 256, 0, 4)
    d = make(s, "f32", mx=True, seed=96)
    d["x"].zero_()
    d["x"][:, 7] = torch.tensor([3.4028234663852886e38, -3.4e38])
    d["w_router"].zero_()
    for k, e in (("gate", -110), ("up", -110), ("down", -8)):
        d[k].fill_(2.0 ** e)
    got = call(s, d, pack(s, d, "f32", True), True)
    check(s, d, got, 3)


@pytest.mark.parametrize("nan", [0x7FC00000, 0x7FFFFFFF, 0x7F800001, 0xFFFFFFFF, 0xFF800001])
@pytest.mark.parametrize("mx", [False, True])
def test_every_nan_stays_in_its_token(nan, mx):
    s = B.Shape(5, 256, 24, 4, 256, 0, 24)
    d = make(s, "f32", mx, seed=97)
    x = d["x"].cpu()
    x.view(torch.int32)[2, 5] = nan - (1 << 32) if nan >> 31 else nan
    d["x"] = x.cuda()
    got = call(s, d, pack(s, d, "f32", mx), mx)
    assert torch.isnan(got[2]).all()
    assert torch.isfinite(got[[0, 1, 3, 4]]).all()


@pytest.mark.parametrize("mx", [False, True])
def test_nan_over_the_shards(mx):
    """A token whose logits are NaN chooses K experts like any other: the ranks that hold one of them write NaN, the
    rest zeros, and the sum over the ranks is NaN."""
    full = B.Shape(5, 256, 24, 4, 256, 0, 24)
    d = make(full, mx=mx, seed=98)
    d["x"][2, 5] = math.nan
    idx = torch.empty((5, 4), dtype=torch.int32, device="cuda")
    total = torch.zeros((5, 256), device="cuda")
    for b, e in ((0, 2), (2, 9), (9, 24)):
        s = B.Shape(5, 256, 24, 4, 256, b, e)
        part = dict(d, **{k: d[k][b:e].contiguous() for k in ("gate", "up", "down")})
        got = call(s, part, pack(s, part, mx=mx), mx, topk_idx=idx)
        here = ((idx[2] >= b) & (idx[2] < e)).any().item()
        assert torch.isnan(got[2]).all() if here else (got[2] == 0).all()
        total += got
    assert torch.isnan(total[2]).all() and torch.isfinite(total[[0, 1, 3, 4]]).all()


@pytest.mark.parametrize("shape", [(4, 8, 8), (8, 8, 8), (6, 8, 4), (12, 8, 8), (12, 64, 4), (16, 8, 3), (16, 32, 8),
                                   (32, 8, 8), (32, 64, 4)])
@pytest.mark.parametrize("mx", [False, True])
def test_down_tiles(shape, mx):
    """T, E, K: one MFMA tile and two, rows that are the tokens throughout and rows by segments."""
    T, E, K = shape
    s = B.Shape(T, 256, E, K, 512, 0, E)
    d = make(s, mx=mx, seed=100 + T)
    check(s, d, call(s, d, pack(s, d, mx=mx), mx), 3 if mx else 2)


@pytest.mark.parametrize("T", [1, 8, 20])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_small_and_ordinary_rows_in_turn(T, dtype):
    """One workspace, eager and in a graph, whose calls change between rows that need scales and rows that do not."""
    s = B.Shape(T, 256, 32, 4, 256, 0, 30)
    d = make(s, dtype, seed=110 + T)
    packed = pack(s, d, dtype)
    x = d["x"].clone()
    mixed = torch.where(torch.arange(T, device="cuda")[:, None] % 2 == 0, 1.0, 1e-6)
    inputs = [(x.float() * f).to(x.dtype) for f in (1.0, 1e-5, mixed, 1.0, 1e-9)]
    refs = [call(s, dict(d, x=v), packed) for v in inputs]
    ws = torch.empty(B.moe_layer_few_tokens_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    out = torch.empty((T, s.H), device="cuda")
    args = (s, d["x"], d["w_router"], packed, d["bias"])
    B.moe_layer_few_tokens(*args, out=out, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.moe_layer_few_tokens(*args, out=out, ws=ws)
    for v, ref in zip(inputs + inputs, refs + refs):
        d["x"].copy_(v)
        out.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
        out.fill_(math.nan)
        B.moe_layer_few_tokens(*args, out=out, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
