"""Every variant of the int8 product's kernels and of the rows' kernels on the GPU, against the definition."""
import pytest
import torch

import quantized_sizes as sizes
from moe_layer_03_amd import binding as B
from moe_layer_03_amd import quantized as Q
from quantized_reference import TYPES, U, int8_rows, mx_rows, to_type
from test_gpu_dense_int8 import EPI, inputs, pack, reference

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def buffer(rows, n, dtype, ld, junk):
    """[rows, n], rows ld apart, in a buffer of junk that ends with the last row; and the buffer."""
    buf = torch.full(((rows - 1) * ld + n,), junk, dtype=dtype, device="cuda")
    return buf.as_strided((rows, n), (ld, 1)), buf


def untouched(buf, view, junk):
    view.fill_(junk)                                   # after the comparison
    return bool((buf == junk).all())


@pytest.mark.parametrize("M,N,K,gated,rows16", sizes.products())
@pytest.mark.parametrize("c,residual", [("f32", "bf16"), ("bf16", "f32")])
def test_products(M, N, K, gated, rows16, c, residual):
    act = "swiglu" if gated else "silu"
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    d = inputs(1, N, K, act, bias=True, seed=M + N + K)
    ld = (K + 15) // 16 * 16 if rows16 else K + (1 if K % 16 != 15 else 2)
    a, _ = buffer(M, K, torch.int8, ld, -128)          # nothing behind the last row: it ends the buffer
    a.copy_(torch.randint(-128, 128, (M, K), generator=g, device="cuda"))
    sa = torch.rand(M, generator=g, device="cuda") * 0.02
    r = torch.randn((M, N), generator=g, device="cuda").to(TYPES[residual])
    ldc = (N + 3) // 4 * 4 + 4
    out, buf = buffer(M, N, TYPES[c], ldc, 77.0)
    s = B.DenseShape(M, N, K, gated=gated)
    got = Q.moe_dense_gemm_int8(s, a, sa, pack(s, d), EPI[act], bias=d["bias"], residual=r, c=out)
    ref, bound = reference(a, sa, d["w"], d["sw"], d["bias"], r, act, c)
    assert ((got.double() - ref).abs() <= bound).all()
    assert untouched(buf, out, 77.0)


def rows_inputs(rows, H, x, residual, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda t, s: (torch.randn((rows, H), generator=g, device="cuda") * s).to(TYPES[t])   # noqa: E731
    return mk(x, 1.0), mk(residual, 2.0) if residual else None, 1 + 0.2 * torch.randn(H, generator=g, device="cuda")


def normed(x, r, w):
    """(h, v) by the definition: s from a mean in 64 bits, rounded once, then single float32 products."""
    h = x if r is None else to_type(x.float() + r.float(), r.dtype)
    s = (1 / torch.sqrt((h.double() ** 2).mean(1, keepdim=True) + EPS)).float()
    return h, h.float() * s * w


def check_int8(v, codes, scales):
    want, ws = int8_rows(v)
    assert torch.equal(scales, ws) and torch.equal(codes, want)


def id_of(v):
    return "-".join(str(e) for e in v)


@pytest.mark.parametrize("case", list(sizes.norms()), ids=id_of)
def test_norms(case):
    """Rows a few elements apart, at odd places where H is odd: what lies between them stays.  A double's sum in another
    order may move a row's s by a step of float32, in fewer than one row of a million: such a row is compared with the
    neighbouring s."""
    rows, H, xt, rt, yt, want_codes = case
    x, r, w = rows_inputs(rows, H, xt, rt, rows + H)
    pad = 3 if H % 2 else 8
    kw, bufs = {}, []

    def output(name, dtype, junk):
        kw[name], buf = buffer(rows, H, dtype, H + pad, junk)
        bufs.append((buf, kw[name], junk))
    if rt:
        output("sum_out", TYPES[rt], 7.0)
    if yt:
        output("y", TYPES[yt], 7.0)
    output("codes", torch.int8, 99)
    h, y, codes, scales = Q.moe_add_rmsnorm(x, w, r, EPS, q_dtype=Q.MOE_I8, **kw)
    wh, v = normed(x, r, w)
    if rt:
        assert torch.equal(h, wh)
    want, ws = int8_rows(v)
    off = (scales != ws) | (codes != want).any(1)
    if yt:
        off |= (y != to_type(v, TYPES[yt])).any(1)
    assert off.sum() <= 2, f"{int(off.sum())} rows differ"
    for i in off.nonzero()[:, 0].tolist():
        d = wh[i:i + 1].double()
        s = (1 / torch.sqrt((d * d).mean() + EPS)).float()
        near = [torch.nextafter(s, torch.full_like(s, e)) for e in (0.0, 1e30)]
        for t in near:
            u = wh[i:i + 1].float() * t * w
            c, cs = int8_rows(u)
            if torch.equal(c, codes[i:i + 1]) and torch.equal(cs, scales[i:i + 1]):
                assert yt is None or torch.equal(y[i:i + 1], to_type(u, TYPES[yt]))
                break
        else:
            raise AssertionError(f"row {i} has no such s")
    for buf, view, junk in bufs:
        assert untouched(buf, view, junk), "written outside the rows"


@pytest.mark.parametrize("rows,H", [(55000, 128), (5301, 1321), (1700, 4096), (571, 12291), (175, 40001), (215, 32800)])
@pytest.mark.parametrize("sum_at,y_at", [("x", "r"), ("r", "x"), (None, "r")])
def test_norms_in_place_past_the_caches(rows, H, sum_at, y_at):
    """The passes of a long row read h again from where the first has just written it, past the caches."""
    x, r, w = rows_inputs(rows, H, "f32", "f32", H)
    wh, v = normed(x, r, w)
    at = {"x": x, "r": r}
    h, y, codes, scales = Q.moe_add_rmsnorm(x, w, r, EPS, sum_out=at.get(sum_at), y=at[y_at], q_dtype=Q.MOE_I8)
    assert torch.equal(h, wh)
    assert torch.equal(y, v)
    check_int8(v, codes, scales)


@pytest.mark.parametrize("rows,H", [(55000, 128), (28000, 256), (14000, 512), (6800, 1024), (5300, 1312), (1700, 4096),
                                    (430, 16384), (215, 32800), (3500, 992), (2100, 1120)])
@pytest.mark.parametrize("x,residual", [("f32", "bf16"), ("bf16", None)])
def test_norms_with_mxfp8_codes(rows, H, x, residual):
    """y in float32 is v: the codes are the MXFP8 quantiser's of it, and, for some rows, the oracle's."""
    x, r, w = rows_inputs(rows, H, x, residual, H)
    _, y, codes, scales = Q.moe_add_rmsnorm(x, w, r, EPS, y_dtype=torch.float32, q_dtype=Q.MOE_MXFP8)
    exact = normed(x, r, w)[1]
    assert ((y.double() - exact.double()).abs() <= 2 * U * exact.double().abs()).all()   # a step of s at most
    some = list(range(0, rows, rows // 13))[-12:] + [rows - 1]
    want, ws = mx_rows(y[some].cpu())
    assert torch.equal(codes[some].cpu(), want) and torch.equal(scales[some].cpu(), ws)
    want, ws = B.moe_quantize_mxfp8(y)
    assert torch.equal(codes, want.view(torch.uint8).view(codes.shape)) and torch.equal(scales, ws.view(scales.shape))


@pytest.mark.parametrize("case", sizes.quantisers(), ids=id_of)
def test_quantisers(case):
    rows, K, t = case
    x, _, _ = rows_inputs(rows, K, t, None, rows)
    pad = 3 if K % 2 else 8
    codes, buf = buffer(rows, K, torch.int8, K + pad, 99)
    _, scales = Q.moe_quantize_int8(x, codes=codes)
    check_int8(x.float(), codes, scales)
    assert untouched(buf, codes, 99)


# ---- the largest calls ------------------------------------------------------------------------

@pytest.mark.parametrize("N,K,gated", [(8, 48, False), (6, 41, True), (196, 48, False), (100, 48, True)])
def test_most_rows_of_a_product(N, K, gated):
    M = 1 << 21
    g = torch.Generator(device="cuda").manual_seed(N)
    d = inputs(1, N, K, "swiglu" if gated else "none", seed=N)
    a = torch.randint(-128, 128, (M, (K + 15) // 16 * 16), generator=g, device="cuda", dtype=torch.int8)[:, :K]
    sa = torch.rand(M, generator=g, device="cuda")
    s = B.DenseShape(M, N, K, gated=gated)
    act = "swiglu" if gated else "none"
    got = Q.moe_dense_gemm_int8(s, a, sa, pack(s, d), EPI[act], c_dtype=torch.float32)
    ref, bound = reference(a, sa, d["w"], d["sw"], None, None, act, "f32")
    assert ((got.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("K", [48, 41])
@pytest.mark.parametrize("gated", [False, True])
def test_most_columns_of_a_product(M, K, gated):
    N = 1 << 18
    g = torch.Generator(device="cuda").manual_seed(M)
    w = [torch.randint(-128, 128, (K, N), generator=g, device="cuda", dtype=torch.int8) for _ in range(1 + gated)]
    sw = [torch.rand(N, generator=g, device="cuda") * 1e-3 for _ in w]
    a = torch.randint(-128, 128, (M, 48), generator=g, device="cuda", dtype=torch.int8)[:, :K]
    sa = torch.rand(M, generator=g, device="cuda")
    s = B.DenseShape(M, N, K, gated=gated)
    act = "swiglu" if gated else "none"
    packed = Q.moe_pack_dense_int8(s, *w, scales=sw[0], up_scales=sw[1] if gated else None)
    got = Q.moe_dense_gemm_int8(s, a, sa, packed, EPI[act], c_dtype=torch.float32)
    ref, bound = reference(a, sa, w, sw, None, None, act, "f32")
    assert ((got.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("H", [8, 136, 520, 1032])
def test_most_rows_of_a_quantiser_and_a_norm(H):
    rows = 1 << 21
    x, _, w = rows_inputs(rows, H, "bf16", None, H)
    codes, scales = Q.moe_quantize_int8(x)
    some = torch.cat([torch.arange(0, rows, 4099), torch.arange(rows - 70, rows)]).cuda()
    check_int8(x[some].float(), codes[some], scales[some])
    del codes, scales
    _, y, codes, scales = Q.moe_add_rmsnorm(x, w, eps=EPS, y_dtype=torch.bfloat16, q_dtype=Q.MOE_I8)
    _, v = normed(x[some], None, w)
    check_int8(v, codes[some], scales[some])
    assert torch.equal(y[some], to_type(v, torch.bfloat16))
