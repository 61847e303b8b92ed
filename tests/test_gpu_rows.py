"""The norm with the residual's sum and 8-bit rows, and the int8 quantiser, on the GPU against their definition."""
import math

import pytest
import torch

from moe_layer_03_amd import binding as B
from moe_layer_03_amd import quantized as Q
from quantized_reference import SMALLEST, TYPES, U, around, int8_rows, mx_rows, normed, placed, to_type

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def inputs(rows, H, x="bf16", residual="bf16", weight="bf16", seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    mk = lambda t, s=1.0, *n: (torch.randn(n, generator=g) * s).to(TYPES[t])   # noqa: E731
    return (mk(x, std, rows, H), mk(residual, 2 * std, rows, H) if residual else None,
            (1 + 0.2 * torch.randn((H,), generator=g)).to(TYPES[weight]) if weight else None)


def check(got, x, residual, weight, eps, y, q):
    """got: (h, y, codes, scales) as CPU tensors."""
    h, v, exact = normed(x, residual, weight, eps)
    if residual is not None:
        assert torch.equal(got[0], h)
    if y is not None:
        t = TYPES[y]
        half = torch.finfo(t).eps / 2
        # s and two products round once each: 3 u; then half a step of y's type
        bound = (3.01 * U + half) * exact.abs() + (2.0 ** -25 if t == torch.float16 else 2.0 ** -133)
        ref = exact.clamp(-65504, 65504) if t == torch.float16 else exact
        assert ((got[1].double() - ref).abs() <= bound).all()
        assert torch.equal(got[1], to_type(v, t))        # bit for bit, every step but the mean being float32's own
    if q == "int8":
        codes, scales = int8_rows(v)
        assert torch.equal(got[3], scales) and torch.equal(got[2], codes)
        # and against 64 bits alone: half a step of the code, the value's 3 u and the scale's 4 u of up to 127 codes
        assert ((got[2].double() * got[3].double()[:, None] - exact).abs()
                <= (0.5 + 127 * 7 * U) * got[3].double()[:, None]).all()
    elif q == "mxfp8":
        codes, scales = mx_rows(v)
        assert torch.equal(got[3], scales) and torch.equal(got[2], codes)


def run(rows, H, x="bf16", residual="bf16", weight="bf16", y="bf16", q="int8", eps=EPS, seed=0, pad=0, offset=0, std=1.0,
        data=None, want_sum=True):
    cx, cr, cw = data or inputs(rows, H, x, residual, weight, seed, std)
    gx, _ = placed(cx, pad, offset)
    gr = placed(cr, pad, offset)[0] if cr is not None else None
    kw, bufs = {}, []

    def output(name, dtype, n, junk):
        kw[name], buf = placed(torch.full((rows, n), junk, dtype=dtype), pad, offset, junk)
        bufs.append((buf, kw[name], junk))
    if cr is not None:
        output("sum_out", cr.dtype, H, 7.0)
    if y:
        output("y", TYPES[y], H, 7.0)
    if q:
        output("codes", torch.int8 if q == "int8" else torch.uint8, H, 99)
        kw["q_dtype"] = Q.MOE_I8 if q == "int8" else Q.MOE_MXFP8
    got = Q.moe_add_rmsnorm(gx, cw.cuda() if cw is not None else None, gr, eps, **kw)
    torch.cuda.synchronize()
    for buf, view, junk in bufs:
        assert around(buf, view, junk), "written outside the rows"
    got = [t.cpu() if t is not None else None for t in got]
    check(got, cx, cr, cw, eps, y, q)
    return got


SIZES = [(1, 1), (2, 2), (3, 7), (1, 8), (5, 9), (4, 31), (2, 33), (7, 63), (1, 100), (9, 255), (3, 257), (130, 511), (2, 513),
         (1, 1000), (5, 1023), (300, 1025), (2, 2047), (3, 2311), (1, 4095), (4, 4097), (2, 8191), (1, 8200), (3, 12289),
         (2, 16385), (1, 32767), (2, 40001)]
ROUND = [(1, 32), (3, 64), (65, 96), (1, 256), (700, 256), (2, 512), (1, 1024), (33, 1536), (129, 2048), (1, 4096),
         (600, 4096), (5, 5120), (2, 8192), (70, 7168), (1, 16384), (3, 32768), (1, 65536)]


@pytest.mark.parametrize("rows,H", SIZES + ROUND)
def test_sizes(rows, H):
    run(rows, H, seed=H)
    run(rows, H, x="f32", residual="bf16", weight="f32", y=None, seed=H + 1, pad=3)
    run(rows, H, x="f16", residual=None, y="f32", q=None, seed=H + 2, pad=1, offset=1)
    run(rows, H, x="f32", residual="f32", weight=None, y="f16", q="int8", seed=H + 3, pad=8)


@pytest.mark.parametrize("rows,H", ROUND)
def test_mxfp8_sizes(rows, H):
    run(rows, H, q="mxfp8", seed=H)
    run(rows, H, x="f32", weight="f32", y=None, q="mxfp8", seed=H + 1, pad=3, offset=1)


@pytest.mark.parametrize("x", list(TYPES))
@pytest.mark.parametrize("residual", [None, "bf16", "f16", "f32"])
@pytest.mark.parametrize("q", [None, "int8", "mxfp8"])
def test_types(x, residual, q):
    for i, (y, weight) in enumerate([("bf16", "f32"), ("f16", "bf16"), ("f32", "f16"), (None if q else "f32", None)]):
        run(5, 352, x, residual, weight, y, q, seed=i)
        run(150, 96, x, residual, weight, y, q, seed=i, pad=5, offset=3)


def test_longest_row():
    run(2, 1 << 18, x="bf16", residual="f32", q="int8", seed=5)
    run(1, 1 << 18, x="f32", residual="bf16", y="f32", q="mxfp8", seed=6)


@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-12, 1e-5, 1.0, 1e30])
def test_eps(eps):
    run(6, 320, y="f32", eps=eps)


@pytest.mark.parametrize("std", [1e-30, 1e-20, 1e-6, 1e4, 1e15])
@pytest.mark.parametrize("q", ["int8", "mxfp8"])
def test_scales_of_the_inputs(std, q):
    """Rows far from one: their mean of squares lies beyond float32's range at both ends; eps rules the small ones."""
    run(5, 256, x="f32", residual="f32", weight="f32", y="f32", q=q, std=std)
    run(5, 2311 if q == "int8" else 2304, x="bf16", residual="bf16", y="f32", q=q, std=std)


def test_fp16_saturates():
    x = torch.full((2, 64), 60000.0, dtype=torch.float16)
    w = torch.full((64,), 60000.0, dtype=torch.float32)
    w[3] = 70000.0
    got = run(2, 64, data=(x, x.clone(), w), y="f16", q="int8")
    assert (got[0] == 65504).all() and got[1][0, 3] == 65504


def test_zero_rows():
    """A row of zeros: zeros, the least scale, zero codes; its neighbours are what they are alone."""
    x, r, w = inputs(4, 256)
    x[1] = 0
    r[1] = 0
    x[2] = -r[2]
    got = run(4, 256, data=(x, r, w), q="int8")
    assert (got[2][1:3] == 0).all() and (got[3][1:3] == SMALLEST).all() and (got[1][1:3] == 0).all()
    got = run(4, 256, data=(x, r, w), q="mxfp8")
    assert (got[2][1:3] & 0x7F == 0).all() and (got[3][1:3] == 0).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("H", [64, 1056, 4096, 40000])
@pytest.mark.parametrize("q", ["int8", "mxfp8"])
def test_not_finite_stays_in_its_row(bad, H, q):
    x, r, w = inputs(3, H, "f32", "bf16")
    x[1, H // 2] = bad
    gx, gr, gw = x.cuda(), r.cuda(), w.cuda()
    h, y, codes, scales = (t.cpu() for t in Q.moe_add_rmsnorm(gx, gw, gr, EPS, y_dtype=torch.float32, q_dtype={
        "int8": Q.MOE_I8, "mxfp8": Q.MOE_MXFP8}[q]))
    keep = [0, 2]
    check([t[keep] for t in (h, y, codes, scales)], x[keep], r[keep], w, EPS, "f32", q)
    assert torch.isnan(y[1, H // 2])
    if q == "int8":
        assert torch.isnan(scales[1]) and (codes[1] == 0).all()
    else:
        assert scales[1, H // 64] == 255 and (codes[1, H // 64 * 32: H // 64 * 32 + 32] == 0x7F).all()
        if math.isnan(bad):
            assert (scales[1] == 255).all()


def test_a_nan_in_the_weight_reaches_every_row():
    x, r, w = inputs(3, 128)
    w[5] = math.nan
    _, y, codes, scales = Q.moe_add_rmsnorm(x.cuda(), w.cuda(), r.cuda(), y_dtype=torch.bfloat16, q_dtype=Q.MOE_I8)
    assert torch.isnan(scales).all() and (codes == 0).all()
    assert torch.isnan(y[:, 5]).all() and torch.isfinite(y[:, :5]).all() and torch.isfinite(y[:, 6:]).all()


@pytest.mark.parametrize("H", [96, 2311, 4096, 40000])
def test_in_place(H):
    """sum over the residual, over x; y over x, over the residual; all with codes, which are read from h after it is written."""
    for x_type, r_type, sum_at, y_at in [("f32", "bf16", "r", None), ("bf16", "bf16", "x", "r"), ("bf16", "bf16", "r", "x"),
                                         ("f16", None, None, "x"), ("f32", "f16", None, "r")]:
        cx, cr, cw = inputs(5, H, x_type, r_type, seed=H)
        x, r, w = cx.cuda(), cr.cuda() if cr is not None else None, cw.cuda()
        at = {"x": x, "r": r, None: None}
        y = at[y_at]
        h, y, codes, scales = Q.moe_add_rmsnorm(x, w, r, EPS, sum_out=at[sum_at], y=y, y_dtype=torch.float32 if y is None else None,
                                                q_dtype=Q.MOE_I8)
        if sum_at:
            assert h.data_ptr() == at[sum_at].data_ptr()
        got = [h.cpu(), y.cpu(), codes.cpu(), scales.cpu()]
        name = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}[y.dtype]
        check(got, cx, cr, cw, EPS, name, "int8")


@pytest.mark.parametrize("H", [256, 4096, 40000])
def test_without_the_sum(H):
    """The C call with sum NULL: what is normed is the rounded sum all the same."""
    x, r, w = inputs(3, H, "f32", "bf16")
    gx, gr, gw = x.cuda(), r.cuda(), w.cuda()
    y = torch.empty((3, H), dtype=torch.float32, device="cuda")
    codes, scales = torch.empty((3, H), dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    st = B.load().moe_add_rmsnorm(3, H, gx.data_ptr(), B.MOE_F32, H, gr.data_ptr(), B.MOE_BF16, H, None, 0, gw.data_ptr(),
                                  B.MOE_BF16, EPS, y.data_ptr(), B.MOE_F32, H, codes.data_ptr(), B.MOE_I8, H,
                                  scales.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == B.MOE_OK
    check([None, y.cpu(), codes.cpu(), scales.cpu()], x, None, w, EPS, None, None)
    _, v, _ = normed(x, r, w, EPS)
    assert torch.equal(y.cpu(), v) and torch.equal(codes.cpu(), int8_rows(v)[0]) and torch.equal(gr.cpu(), r)


# ---- the int8 quantiser ----------------------------------------------------------------------

def quantise(v, pad=0, offset=0):
    gx, _ = placed(v, pad, offset)
    codes, buf = placed(torch.full(v.shape, 99, dtype=torch.int8), pad, offset, 99)
    _, scales = Q.moe_quantize_int8(gx, codes=codes)
    torch.cuda.synchronize()
    assert around(buf, codes, 99)
    want, ws = int8_rows(v.float())
    assert torch.equal(scales.cpu(), ws) or torch.equal(torch.isnan(scales.cpu()), torch.isnan(ws))
    good = torch.isfinite(ws)
    assert torch.equal(scales.cpu()[good], ws[good])
    assert torch.equal(codes.cpu(), want)
    return codes.cpu(), scales.cpu()


@pytest.mark.parametrize("rows,H", SIZES + ROUND)
@pytest.mark.parametrize("t", list(TYPES))
def test_quantise_sizes(rows, H, t):
    g = torch.Generator().manual_seed(H)
    v = (torch.randn((rows, H), generator=g) * torch.exp2(torch.randint(-9, 9, (rows, 1), generator=g))).to(TYPES[t])
    quantise(v)
    quantise(v, pad=5, offset=1)


def test_quantise_ties_and_their_neighbours():
    """Quotients at a half, and one float32 step to each side, for scales of every kind of mantissa."""
    g = torch.Generator().manual_seed(3)
    most = torch.cat([torch.tensor([127.0, 254.0, 1.0, 0.3, 3.0, 2.0 ** -100 * 1.7]), torch.rand(122, generator=g) + 0.5])
    scale = (most.double() / 127).float()
    k = torch.arange(-126, 127).double() + 0.5
    at = (k[None] * scale.double()[:, None]).float()
    rows = torch.cat([most[:, None], at, torch.nextafter(at, torch.full_like(at, 1e9)),
                      torch.nextafter(at, torch.full_like(at, -1e9))], 1)
    rows = rows.clamp(-most[:, None], most[:, None])
    quantise(rows)


@pytest.mark.parametrize("exponent", [-149, -140, -127, -126, -120, -119, -100, 0, 100, 127])
def test_quantise_over_the_whole_range(exponent):
    g = torch.Generator().manual_seed(200 + exponent)
    v = torch.ldexp((torch.rand((4, 300), generator=g) * 2 - 1).double(), torch.tensor(exponent)).float()
    codes, scales = quantise(v)
    if exponent >= -118:
        assert (codes.abs().amax(1) == 127).all()
    assert (scales >= SMALLEST).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_quantise_not_finite(bad):
    v = torch.randn((4, 700))
    v[2, 699] = bad
    codes, scales = quantise(v)
    assert torch.isnan(scales[2]) and (codes[2] == 0).all() and torch.isfinite(scales[[0, 1, 3]]).all()


# ---- many rows, offsets, streams, graphs --------------------------------------------------------

def test_offsets_past_32_bits():
    """Rows whose element offsets pass 2^31, in and out."""
    rows, H, ld = 70000, 64, 33000
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty((rows, ld), dtype=torch.bfloat16, device="cuda")[:, :H]
    x.copy_(torch.randn((rows, H), generator=g, device="cuda"))
    codes = torch.empty((rows, ld), dtype=torch.int8, device="cuda")[:, :H]
    y = torch.empty((rows, ld), dtype=torch.bfloat16, device="cuda")[:, :H]
    _, y, codes, scales = Q.moe_add_rmsnorm(x, y=y, codes=codes, q_dtype=Q.MOE_I8)
    check([None, y.cpu(), codes.cpu(), scales.cpu()], x.cpu(), None, None, EPS, "bf16", "int8")
    codes.zero_()
    _, scales = Q.moe_quantize_int8(x, codes=codes)
    want, ws = int8_rows(x.cpu().float())
    assert torch.equal(codes.cpu(), want) and torch.equal(scales.cpu(), ws)


def test_no_rows():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    h, y, codes, scales = Q.moe_add_rmsnorm(e, None, e.clone(), q_dtype=Q.MOE_MXFP8)
    assert h.shape == (0, 64) and y is None and codes.shape == (0, 64) and scales.shape == (0, 2)
    codes, scales = Q.moe_quantize_int8(e)
    assert codes.shape == (0, 64) and scales.shape == (0,)


@pytest.mark.parametrize("rows,H", [(1, 4096), (257, 4096), (40, 511), (3, 40000)])
def test_repeats_streams_and_replays(rows, H):
    """Bit for bit again, on two streams at once, and from a captured graph on new inputs."""
    def call(d, **kw):
        return Q.moe_add_rmsnorm(*d, EPS, y_dtype=torch.bfloat16, q_dtype=Q.MOE_I8, **kw)

    def new(seed):
        x, r, w = (t.cuda() for t in inputs(rows, H, "f32", "bf16", "f32", seed))
        return x, w, r
    data = [new(1), new(2)]
    first = [call(d) for d in data]
    streams = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i in range(2):
            got[i].append(call(data[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for g in got[i] for a, b in zip(g, first[i]))
    out = dict(zip(("sum_out", "y", "codes", "scales"), first[0]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Q.moe_add_rmsnorm(*data[0], EPS, q_dtype=Q.MOE_I8, **out)
    for i in range(4):
        for a, b in zip(data[0], new(10 + i)):
            a.copy_(b)
        eager = call(data[0])
        for v in out.values():
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out.values(), eager))
