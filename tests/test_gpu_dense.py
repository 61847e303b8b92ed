"""Dense products with a fused epilogue on the GPU against the definition in 64 bits."""
import math

import pytest
import torch

from moe_layer_03_amd import binding as B

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPI = {"none": B.MOE_EPI_NONE, "silu": B.MOE_EPI_SILU, "gelu": B.MOE_EPI_GELU, "gelu_tanh": B.MOE_EPI_GELU_TANH,
       "relu": B.MOE_EPI_RELU, "swiglu": B.MOE_EPI_SWIGLU}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def act64(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2))
    if act == "gelu_tanh":
        return v * torch.sigmoid(math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3))
    return v.clamp(min=0) if act == "relu" else v


def reference(a, w, bias, residual, act, c):
    """(value, bound): float32 sums of K products and a bias are off by at most (K + 2) u of their absolute sum, the
    activations have slopes up to 1.13 and a few u of their own (8 covers expf, erfcf and the division: the steepest,
    exp(-1.6 (z + 0.04 z^3)), has its argument's rounding times the argument, at most 8 where the value matters), and
    the result is rounded by half a step of c's type."""
    a = a.double()
    v = [a @ x.double() for x in w]
    mag = [a.abs() @ x.double().abs() for x in w]
    if bias is not None:
        v = [p + b.double() for p, b in zip(v, bias)]
        mag = [m + b.double().abs() for m, b in zip(mag, bias)]
    err = [(a.shape[1] + 2) * U * m for m in mag]
    if act == "swiglu":
        s = act64(v[0], "silu")
        out = s * v[1]
        e = 1.1 * err[0] * v[1].abs() + s.abs() * err[1] + 1.1 * err[0] * err[1] + 24 * U * out.abs()
    else:
        out = act64(v[0], act)
        e = 1.13 * err[0] + 24 * U * out.abs()
    if residual is not None:
        out = out + residual.double()
        e = e + U * out.abs()
    t = TYPES[c]
    if t == torch.float16:
        out = out.clamp(-65504, 65504)
    step = torch.finfo(t).eps / 2
    return out, e * (1 + step) + step * out.abs() + (2.0 ** -25 if t == torch.float16 else 2.0 ** -133)


def inputs(M, N, K, act, a="bf16", bias=False, residual=None, seed=0, pad=0, offset=0):
    g = torch.Generator().manual_seed(seed)
    n = 2 if act == "swiglu" else 1
    t = TYPES[a]

    def rows(cols, dtype, std=1.0):
        """[M, cols] inside a NaN buffer: rows cols + pad apart, starting `offset` elements in."""
        buf = torch.full((offset + M * (cols + pad),), float("nan"), dtype=dtype, device="cuda")
        v = buf[offset:].view(M, cols + pad)[:, :cols]
        v.copy_((torch.randn((M, cols), generator=g) * std).to(dtype))
        return v
    return dict(a=rows(K, t), w=[(torch.randn((K, N), generator=g) * 0.05).to(t).cuda() for _ in range(n)],
                bias=(torch.randn((n, N), generator=g)).cuda() if bias else None,
                residual=rows(N, TYPES[residual]) if residual else None)


def run(M, N, K, act="none", a="bf16", c="bf16", bias=False, residual=None, seed=0, pad=0, offset=0):
    d = inputs(M, N, K, act, a, bias, residual, seed, pad, offset)
    s = B.DenseShape(M, N, K, gated=act == "swiglu")
    packed = B.moe_pack_dense(s, *d["w"])
    buf = torch.full((M + 1, N + pad), 77.0, dtype=TYPES[c], device="cuda")
    got = B.moe_dense_gemm(s, d["a"], packed, EPI[act], bias=d["bias"], residual=d["residual"], c=buf[:M, :N])
    torch.cuda.synchronize()
    assert (buf[:M, N:] == 77).all() and (buf[M] == 77).all()
    ref, bound = reference(d["a"], d["w"], d["bias"], d["residual"], act, c)
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    assert (err <= bound).all(), f"{(err - bound).max().item():.3e} over the bound"
    if c == "f32":      # random rounding: 0.6 u sqrt(K) per product of the RMS, doubled for the longest chain's luck
        assert err.pow(2).mean().sqrt() <= max(3e-6, 4 * 0.6 * U * math.sqrt(K)) * ref.pow(2).mean().sqrt()
    return got


SIZES = [(1, 1, 1), (1, 64, 64), (2, 37, 8), (1, 1536, 1024), (3, 100, 72), (15, 256, 96), (16, 31, 128), (17, 128, 200),
         (32, 33, 64), (33, 512, 256), (63, 96, 320), (64, 65, 40), (65, 1000, 136), (96, 192, 1096), (127, 160, 64),
         (128, 256, 512), (129, 130, 264), (200, 1003, 96), (255, 320, 128), (256, 256, 256), (257, 257, 64),
         (300, 512, 192), (513, 640, 160), (1000, 192, 320)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("gated", [False, True])
def test_sizes(size, gated):
    run(*size, act="swiglu" if gated else "none", c="f32", seed=sum(size))
    run(*size, act="swiglu" if gated else "none", c="bf16", bias=True, residual="bf16", seed=1 + sum(size), pad=8)


# one size for each unit and tile shape, ungated and gated
SHAPES = [(5, 4100, 40), (17, 2050, 40), (17, 4100, 40), (48, 4100, 40), (200, 200, 40), (65, 16400, 264), (2050, 1000, 40),
          (2050, 4100, 40), (600, 16400, 40), (513, 70, 520), (513, 70, 40), (5, 4100, 131), (17, 2050, 131),
          (17, 4100, 131), (48, 4100, 1031), (128, 4100, 131)]
SHAPES_GATED = [(5, 2050, 40), (48, 2050, 40), (65, 8200, 264), (1030, 1000, 40), (300, 12300, 72), (200, 16400, 72),
                (200, 200, 40), (513, 70, 520), (513, 70, 40), (5, 2050, 131), (17, 2050, 131), (200, 200, 131),
                (48, 2050, 1031), (128, 2050, 131)]


@pytest.mark.parametrize("size,act", [(s, "relu") for s in SHAPES] + [(s, "swiglu") for s in SHAPES_GATED])
@pytest.mark.parametrize("a", ["bf16", "f16"])
def test_unit_and_tile_shapes(size, act, a):
    run(*size, act, a=a, c="f32", bias=True, residual="bf16", pad=8, seed=sum(size))


@pytest.mark.parametrize("act", list(EPI))
@pytest.mark.parametrize("a", ["bf16", "f16"])
@pytest.mark.parametrize("M", [5, 70, 300])
def test_epilogues_and_types(act, a, M):
    for i, (c, residual, bias) in enumerate([("f32", None, True), ("bf16", "f32", False), ("f16", "bf16", True),
                                             ("f32", "f16", False), ("f16", None, False)]):
        run(M, 136, 104, act=act, a=a, c=c, bias=bias, residual=residual, seed=i)


@pytest.mark.parametrize("M", [1, 20, 150])
@pytest.mark.parametrize("K,pad,offset", [(63, 0, 0), (65, 3, 0), (100, 4, 0), (64, 0, 3), (64, 1, 0), (7, 0, 1), (130, 6, 2)])
def test_rows_off_16_bytes(M, K, pad, offset):
    """Odd reductions, odd strides, odd starts: NaN lies between the rows."""
    run(M, 70, K, c="f32", bias=True, residual="f32", pad=pad, offset=offset, seed=K)
    run(M, 70, K, act="swiglu", a="f16", c="f16", residual="f16", pad=pad, offset=offset, seed=K)


@pytest.mark.parametrize("M", [1, 16, 40, 100, 512, 777])
def test_exact_on_integers(M):
    """Small integers: every order of summation is exact, whatever path the size takes."""
    g = torch.Generator().manual_seed(M)
    N, K = 320, 576
    a = torch.randint(-4, 5, (M, K), generator=g).bfloat16().cuda()
    w = torch.randint(-4, 5, (K, N), generator=g).bfloat16().cuda()
    s = B.DenseShape(M, N, K)
    got = B.moe_dense_gemm(s, a, B.moe_pack_dense(s, w), c_dtype=torch.float32)
    assert torch.equal(got.double(), a.double() @ w.double())


@pytest.mark.parametrize("M,c", [(4, "f32"), (33, "bf16"), (400, "f32"), (400, "f16")])
def test_residual_in_place(M, c):
    d = inputs(M, 200, 160, "none", residual=c, seed=M, pad=8)
    s = B.DenseShape(M, 200, 160)
    ref, bound = reference(d["a"], d["w"], None, d["residual"], "none", c)
    got = B.moe_dense_gemm(s, d["a"], B.moe_pack_dense(s, *d["w"]), residual=d["residual"], c=d["residual"])
    assert got.data_ptr() == d["residual"].data_ptr()
    assert ((got.double() - ref).abs() <= bound).all()


def test_float32_weights_are_packed_as_fp16():
    g = torch.Generator().manual_seed(1)
    a = torch.randn((9, 80), generator=g).half().cuda()
    w = (torch.randn((80, 50), generator=g) * 0.05).cuda()
    s = B.DenseShape(9, 50, 80)
    got = B.moe_dense_gemm(s, a, B.moe_pack_dense(s, w), c_dtype=torch.float32)
    assert torch.equal(got, B.moe_dense_gemm(s, a, B.moe_pack_dense(s, w.half()), c_dtype=torch.float32))


def test_fp16_output_saturates():
    a = torch.full((3, 64), 300.0, dtype=torch.float16, device="cuda")
    w = torch.full((64, 40), 300.0, dtype=torch.float16, device="cuda")
    s = B.DenseShape(3, 40, 64)
    packed = B.moe_pack_dense(s, w)
    assert (B.moe_dense_gemm(s, a, packed) == 65504).all()
    assert (B.moe_dense_gemm(s, -a, packed) == -65504).all()
    assert (B.moe_dense_gemm(s, a, packed, c_dtype=torch.float32) == 300.0 * 300.0 * 64).all()


def test_far_tails_of_the_activations():
    """Pre-activations from -60 to 60 through a bias."""
    N = 128
    s = B.DenseShape(2, N, 64)
    a = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    bias = torch.linspace(-60, 60, N, device="cuda")[None]
    packed = B.moe_pack_dense(s, torch.zeros((64, N), dtype=torch.bfloat16, device="cuda"))
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        got = B.moe_dense_gemm(s, a, packed, EPI[act], bias=bias, c_dtype=torch.float32)
        ref = act64(bias.double(), act).expand(2, -1)
        # exp(-y)'s relative error is its argument's rounding, |y| u; |y| up to 1.6 (60 + 0.0447 60^3) for gelu_tanh, but
        # only values above float32's smallest normal number are compared relatively, where |y| <= 100
        assert ((got.double() - ref).abs() <= 220 * U * ref.abs() + 2.0 ** -126).all(), act


def test_offsets_past_32_bits():
    """Rows of A, of the residual and of C whose element offsets pass 2^31."""
    M, K, N, ld = 70000, 64, 64, 33000
    g = torch.Generator(device="cuda").manual_seed(2)
    a = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")[:, :K]
    a.copy_(torch.randn((M, K), generator=g, device="cuda"))
    w = (torch.randn((K, N), generator=g, device="cuda") * 0.1).bfloat16()
    c = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")[:, :N]
    c.copy_(torch.randn((M, N), generator=g, device="cuda"))
    ref, bound = reference(a, [w], None, c, "none", "bf16")
    s = B.DenseShape(M, N, K)
    got = B.moe_dense_gemm(s, a, B.moe_pack_dense(s, w), residual=c, c=c)
    assert ((got.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("M,N,K,pad", [(1, 64, 40, 0), (5, 64, 72, 1), (100, 64, 104, 0), (70, 100, 33, 1),
                                       (130, 192, 40, 0), (300, 320, 104, 0), (1100, 512, 296, 0), (300, 100, 161, 3)])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_infinite_weights(M, N, K, pad, value):
    """An infinity in the last row of the weights reaches its own column only, as an infinity: what a kernel multiplies
    beyond K is zero on both sides."""
    g = torch.Generator().manual_seed(9)
    w = (torch.randn((K, N), generator=g) * 0.05).bfloat16()
    w[K - 1, 3::5] = value
    buf = torch.full((M, K + pad), math.nan, dtype=torch.bfloat16, device="cuda")
    a = buf[:, :K]
    a.copy_(torch.rand((M, K), generator=g) + 0.5)
    s = B.DenseShape(M, N, K)
    c = torch.empty((M, N), dtype=torch.float32, device="cuda")
    B.moe_dense_gemm(s, a, B.moe_pack_dense(s, w.cuda()), c=c)
    assert torch.isfinite(c[:, [j for j in range(N) if j % 5 != 3]]).all()
    assert (c[:, 3::5] == value).all()


@pytest.mark.parametrize("M,N,K,pad", [(3, 70, 72, 0), (20, 64, 33, 1), (100, 128, 64, 0), (130, 100, 65, 0),
                                       (300, 256, 96, 0)])
@pytest.mark.parametrize("c", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act", list(EPI))
def test_nan_stays_in_its_row(M, N, K, pad, c, act):
    """A NaN reaches its own row's outputs, whatever the activation and type, and no other row."""
    d = inputs(M, N, K, act, "f16", pad=pad, seed=8)
    d["a"][M // 2, K - 1] = math.nan
    s = B.DenseShape(M, N, K, gated=act == "swiglu")
    got = B.moe_dense_gemm(s, d["a"], B.moe_pack_dense(s, *d["w"]), EPI[act], c_dtype=TYPES[c])
    assert torch.isnan(got[M // 2]).all()
    assert torch.isfinite(got[: M // 2]).all() and torch.isfinite(got[M // 2 + 1:]).all()


def test_no_rows():
    s = B.DenseShape(0, 40, 64)
    packed = B.moe_pack_dense(s, torch.zeros((64, 40), dtype=torch.bfloat16, device="cuda"))
    assert B.moe_dense_gemm(s, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), packed).shape == (0, 40)


@pytest.mark.parametrize("M", [1, 48, 640])
def test_repeats_and_replays(M):
    """Bit for bit again, on another stream, and from a captured graph on new inputs."""
    d = inputs(M, 512, 256, "swiglu", bias=True, residual="bf16", seed=M)
    s = B.DenseShape(M, 512, 256, gated=True)
    packed = B.moe_pack_dense(s, *d["w"])

    def call(c=None, stream=None):
        return B.moe_dense_gemm(s, d["a"], packed, EPI["swiglu"], bias=d["bias"], residual=d["residual"], c=c,
                                stream=stream)
    first = call()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = torch.empty_like(first)
    call(other, st)
    torch.cuda.synchronize()
    assert torch.equal(first, call()) and torch.equal(first, other)
    c = torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c)
    for i in range(3):
        d["a"].copy_(inputs(M, 512, 256, "swiglu", seed=100 + i)["a"])
        eager = call()
        c.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, eager)
