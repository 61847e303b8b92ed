"""What the dense product does at the ends of its types: NaN of every payload, the 16-bit rounding, float32 activations
far from zero.  A is zero, so that the sum is the bias and the residual exactly."""
import math

import pytest
import torch

from moe_layer_03_amd import binding as B

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24
# M, N, K, extra elements per row of A: weight streaming (16-byte rows and others), tiles, any alignment
SIZES = [(3, 70, 64, 0), (20, 132, 65, 0), (130, 260, 64, 0), (700, 128, 264, 0), (600, 100, 65, 0)]
NANS = [0x7FC00000, 0x7FFFFFFF, 0x7F800001, 0xFFC00000, 0xFFFFFFFF, 0xFF800001]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def bits(values, dtype=torch.float32):
    """Tensor of the given bit patterns."""
    width = {torch.float32: torch.int32, torch.bfloat16: torch.int16, torch.float16: torch.int16}[dtype]
    size = 32 if width == torch.int32 else 16
    v = torch.as_tensor(values, dtype=torch.int64)
    return (v - ((v >> (size - 1)) << size)).to(width).view(dtype).cuda()


def zero_product(M, N, K, pad, **kw):
    s = B.DenseShape(M, N, K)
    a = torch.zeros((M, K + pad), dtype=torch.bfloat16, device="cuda")[:, :K]
    packed = B.moe_pack_dense(s, torch.zeros((K, N), dtype=torch.bfloat16, device="cuda"))
    return B.moe_dense_gemm(s, a, packed, **kw)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("c", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("through", ["f32", "f16", "bf16", "bias"])
def test_every_nan_stays_nan(size, c, through):
    """Whatever the payload, from a residual or a bias; its neighbours stay numbers."""
    M, N, K, pad = size
    if through == "bias":
        bias = torch.ones((1, N), device="cuda")
        bias[0, : 2 * len(NANS): 2] = bits(NANS)
        got = zero_product(M, N, K, pad, bias=bias, c_dtype=TYPES[c])
        nan = torch.isnan(bias).expand(M, -1)
    else:
        r = torch.ones((M, N), dtype=TYPES[through], device="cuda")
        wide = NANS if through == "f32" else [0x7FFF, 0xFFFF, 0x7FC1, 0xFFC1]
        r[M // 2, : 2 * len(wide): 2] = bits(wide, TYPES[through])
        r[M - 1, N - 1] = bits(wide[1:2], TYPES[through])[0]
        got = zero_product(M, N, K, pad, residual=r, c_dtype=TYPES[c])
        nan = torch.isnan(r)
    assert torch.equal(torch.isnan(got), nan)
    assert (got[~nan] == 1).all()


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("c", ["bf16", "f16"])
def test_rounding_to_16_bits(size, c):
    """To nearest, ties to even, for every exponent, subnormal results among them: torch's own conversion."""
    M, N, K, pad = size
    g = torch.Generator().manual_seed(M)
    v = torch.randint(0, 1 << 32, (M, N), generator=g)
    v[:, ::3] &= ~0xFFFF                                  # exact in bf16
    v[:, 1::3] = (v[:, 1::3] & ~0xFFFF) | 0x8000          # halfway between two bf16 values
    if c == "f16":                                        # exponents of fp16, halfway cases among them
        v = (v & 0x807FE000) | (v >> 9 & 1) << 12 | (torch.randint(98, 143, (M, N), generator=g) << 23)
    r = bits(v)
    r = torch.where(torch.isfinite(r), r, torch.ones_like(r))
    got = zero_product(M, N, K, pad, residual=r, c_dtype=TYPES[c])
    r = r.cpu() if c == "bf16" else r.cpu().clamp(-65504, 65504)
    assert torch.equal(got.cpu(), r.to(TYPES[c]))


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "swiglu"])
def test_float32_activations(size, act):
    """v / (1 + exp(-y)) to a few units of float32 (u = 2^-24) wherever it is a normal number.

    An exponential to an ulp (2 u) with a rounding, the sum, the reciprocal and the product: 6 u; below y = -80 exp(y)
    is taken as two factors exp(y / 2), 2 u each, with two products: 6 u (SwiGLU's product one more).  SiLU's y is v
    itself; tanh-GELU's y = c (v + d v^3) has seven roundings, of which exp makes 7 u |y|."""
    M, N, K, pad = size
    gated = act == "swiglu"
    v = torch.linspace(-100, 40, N) if act != "gelu_tanh" else torch.linspace(-11, 5, N)
    bias = torch.stack([v, torch.full((N,), 0.75)] if gated else [v]).cuda()
    s = B.DenseShape(M, N, K, gated=gated)
    a = torch.zeros((M, K + pad), dtype=torch.bfloat16, device="cuda")[:, :K]
    w = torch.zeros((K, N), dtype=torch.bfloat16, device="cuda")
    epi = {"silu": B.MOE_EPI_SILU, "gelu_tanh": B.MOE_EPI_GELU_TANH, "swiglu": B.MOE_EPI_SWIGLU}[act]
    got = B.moe_dense_gemm(s, a, B.moe_pack_dense(s, w, w if gated else None), epi, bias=bias, c_dtype=torch.float32)
    x = bias[0].double()
    y = math.sqrt(8 / math.pi) * (x + 0.044715 * x ** 3) if act == "gelu_tanh" else x
    ref = x * torch.where(y < -30, torch.exp(y) / (1 + torch.exp(y)), 1 / (1 + torch.exp(-y))) * (0.75 if gated else 1)
    units = (6 + gated + (7 * y.abs() if act == "gelu_tanh" else 0)) * 1.01     # 1.01: products of the small terms
    # below the normal numbers a result is off by its own spacing, times at most one more factor
    assert ((got.double() - ref).abs() <= units * U * ref.abs() + 2.0 ** -148).all()
