"""Dense products whose rows of C and of the residual lie megabytes apart: the same bits as with rows side by side."""
import pytest
import torch

from moe_layer_03_amd import binding as B
from moe_layer_03_amd import quantized as Q
from test_gpu_dense import EPI, TYPES, inputs, reference
from test_gpu_dense_int8 import inputs as inputs8, pack as pack8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def apart(M, N, dtype, row_bytes):
    """[M, N], rows a little over row_bytes apart."""
    ld = row_bytes // dtype.itemsize + 8
    return torch.empty(((M - 1) * ld + N,), dtype=dtype, device="cuda").as_strided((M, N), (ld, 1))


def check(M, N, K, act, a, c, residual, far, row_bytes, in_place=False):
    d = inputs(M, N, K, act, a, True, residual, seed=M + N + K)
    s = B.DenseShape(M, N, K, gated=act == "swiglu")
    packed = B.moe_pack_dense(s, *d["w"])

    def call(r, out):
        return B.moe_dense_gemm(s, d["a"], packed, EPI[act], bias=d["bias"], residual=r, c=out)
    near = call(d["residual"], torch.empty((M, N), dtype=TYPES[c], device="cuda"))
    r, out = d["residual"], torch.empty((M, N), dtype=TYPES[c], device="cuda")
    if "r" in far:
        r = apart(M, N, TYPES[residual], row_bytes)
        r.copy_(d["residual"])
    if "c" in far:
        out = r if in_place else apart(M, N, TYPES[c], row_bytes)
    got = call(r, out)
    assert torch.equal(got, near)
    ref, bound = reference(d["a"], d["w"], d["bias"], d["residual"], act, c)
    assert ((got.double() - ref).abs() <= bound).all()


# over 8 MiB apart 256 rows pass the reach of a buffer.  A size for each tile shape, then for rows of A off 16 bytes.
SIZES = [(2050, 4100, 1032), (600, 12300, 264), (2050, 1000, 520), (700, 2052, 1032), (513, 1030, 1032), (513, 70, 1032),
         (700, 516, 1033), (700, 515, 1033)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("c,residual,far", [("bf16", "f32", "c"), ("f32", "bf16", "r"), ("f32", "f32", "cr")])
def test_rows_8_mib_apart(M, N, K, act, c, residual, far):
    check(M, N, K, act, "bf16", c, residual, far, 8 << 20, in_place=c == residual)


@pytest.mark.parametrize("M,N,K", [(600, 516, 520), (600, 515, 523)])
def test_fp16_rows_8_mib_apart(M, N, K):
    check(M, N, K, "silu", "f16", "f16", "f16", "cr", 8 << 20, in_place=True)


@pytest.mark.parametrize("M,N,K", [(40, 520, 264), (128, 4100, 1032), (128, 4099, 1091)])
def test_rows_128_mib_apart(M, N, K):
    """16 of them pass the reach of a buffer: an element at a time, in any order of k."""
    d = inputs(M, N, K, "silu", "bf16", True, "f32", seed=K)
    s = B.DenseShape(M, N, K)
    out = apart(M, N, torch.float32, 128 << 20)
    out.copy_(d["residual"])
    got = B.moe_dense_gemm(s, d["a"], B.moe_pack_dense(s, *d["w"]), EPI["silu"], bias=d["bias"], residual=out, c=out)
    ref, bound = reference(d["a"], d["w"], d["bias"], d["residual"], "silu", "f32")
    assert ((got.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("M,N,K,row_bytes", [(700, 1028, 272, 8 << 20), (700, 1027, 272, 8 << 20), (150, 1028, 272, 32 << 20),
                                             (40, 70, 261, 32 << 20), (70, 72, 130, 32 << 20), (5, 72, 144, 1 << 30)])
@pytest.mark.parametrize("act", ["relu", "swiglu"])
def test_int8_rows_far_apart(M, N, K, row_bytes, act):
    d = inputs8(M, N, K, act, True, "f32", seed=N)
    s = B.DenseShape(M, N, K, gated=act == "swiglu")
    packed = pack8(s, d)

    def call(r, out):
        return Q.moe_dense_gemm_int8(s, d["a"], d["sa"], packed, EPI[act], bias=d["bias"], residual=r, c=out)
    near = call(d["residual"], torch.empty((M, N), device="cuda"))
    out = apart(M, N, torch.float32, row_bytes)
    out.copy_(d["residual"])
    assert torch.equal(call(out, out), near)
