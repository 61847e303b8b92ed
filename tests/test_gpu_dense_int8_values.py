"""The int8 dense product on the GPU: scales of either sign, against the definition in 64 bits."""
import pytest
import torch

from moe_layer_03_amd import binding as B
from moe_layer_03_amd import quantized as Q
from test_gpu_dense_int8 import inputs, pack, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check(M, N, K, sa, sw, act, pad=0):
    """sa, sw: float32 on the CPU, of the rows and of each weight's columns."""
    d = inputs(M, N, K, act, seed=11, pad=pad)
    d["sa"], d["sw"] = sa.cuda(), [s.cuda() for s in sw]
    s = B.DenseShape(M, N, K, gated=act == "swiglu")
    got = Q.moe_dense_gemm_int8(s, d["a"], d["sa"], pack(s, d), B.MOE_EPI_SWIGLU if act == "swiglu" else B.MOE_EPI_NONE,
                                c_dtype=torch.float32)
    ref, bound = reference(d["a"], d["sa"], d["w"], d["sw"], None, None, act, "f32")
    assert torch.isfinite(got).all()
    assert ((got.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("M,K,pad", [(3, 144, 0), (100, 144, 0), (600, 144, 0), (600, 141, 0), (20, 130, 1)])
@pytest.mark.parametrize("sa,sw", [(-1e30, 1e-12), (-1e30, -1e-12), (1e30, -1e-12), (-1e36, 1e-36), (-1e-36, 1e36), (-1e-30, -1e30),
                                   (-1.0, 1e30), (-1.5, -1e30), (-(2.0 ** 115), 2.0 ** -126)])
@pytest.mark.parametrize("N", [70, 72])
def test_scales_of_either_sign(M, K, pad, sa, sw, N):
    """No product on the way overflows where the result does not: sums here reach 2^20 and some."""
    check(M, N, K, torch.full((M,), sa), [torch.full((N,), sw)], "none", pad)


@pytest.mark.parametrize("M", [3, 100, 600])
def test_scales_of_both_signs_in_a_call(M):
    """Large and small rows side by side, a lane's rows apart: each takes its own order."""
    g = torch.Generator().manual_seed(M)
    N, K = 136, 144
    sa = torch.where(torch.rand(M, generator=g) < 0.5, -1e34, 1e-6) * torch.where(torch.rand(M, generator=g) < 0.5, -1.0, 1.0)
    check(M, N, K, sa, [torch.where(torch.rand(N, generator=g) < 0.5, -1e-12, 1e-12)], "none")


@pytest.mark.parametrize("M", [3, 100, 600])
def test_negative_scales_of_a_gated_product(M):
    """Gate and up values of a few units each, from a row scale of -1e34."""
    g = torch.Generator().manual_seed(M)
    N, K = 136, 144
    sw = [(torch.rand(N, generator=g) - 0.5) * 1e-37 for _ in range(2)]
    check(M, N, K, torch.full((M,), -1e34), sw, "swiglu")
