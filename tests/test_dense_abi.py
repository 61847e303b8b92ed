"""The dense product's refusals, on the host before any HIP call (no GPU needed)."""
import ctypes

import pytest
import torch

from moe_layer_03_amd import binding as B

P = ctypes.c_void_p(0x1000)
BAD, UNS = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED


def _at(n):
    return ctypes.c_void_p(0x1000 + n)


def _gemm(M=8, N=40, K=64, gated=0, a=P, ad=B.MOE_BF16, lda=64, packed=P, epi=0, bias=None, r=None, rd=0, ldr=40, c=P,
          cd=B.MOE_BF16, ldc=40):
    s = B._CDenseShape(M, N, K, gated)
    return B.load().moe_dense_gemm(ctypes.byref(s), a, ad, lda, packed, epi, bias, r, rd, ldr, c, cd, ldc, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), BAD), (dict(N=0), BAD), (dict(K=0), BAD), (dict(gated=2), BAD),
    (dict(M=(1 << 21) + 1), UNS), (dict(N=(1 << 18) + 1, ldc=1 << 20), UNS), (dict(K=(1 << 18) + 1, lda=1 << 20), UNS),
    (dict(epi=6), BAD), (dict(epi=-1), BAD), (dict(epi=B.MOE_EPI_SWIGLU), BAD), (dict(gated=1), BAD),
    (dict(gated=1, epi=B.MOE_EPI_SILU), BAD),
    (dict(ad=B.MOE_F32), UNS), (dict(ad=B.MOE_MXFP8), UNS), (dict(cd=B.MOE_MXFP8), UNS), (dict(r=P, rd=9), UNS),
    (dict(lda=63), BAD), (dict(ldc=39), BAD), (dict(r=P, ldr=39), BAD),
    (dict(a=None), BAD), (dict(packed=None), BAD), (dict(c=None), BAD),
    (dict(a=_at(1)), BAD), (dict(packed=_at(8)), BAD), (dict(c=_at(1)), BAD), (dict(c=_at(2), cd=B.MOE_F32), BAD),
    (dict(r=_at(1), rd=B.MOE_BF16), BAD), (dict(r=_at(2), rd=B.MOE_F32), BAD), (dict(bias=_at(2)), BAD),
    (dict(r=P, rd=B.MOE_F32), BAD),                     # in place in another type
    (dict(r=P, rd=B.MOE_BF16, ldr=48), BAD),            # in place with another stride
    (dict(M=0, a=None, c=None, packed=None), B.MOE_OK),
])
def test_gemm_refusals(kw, status):
    assert _gemm(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), BAD), (dict(w=_at(1)), BAD), (dict(w=_at(2), dt=B.MOE_F32), BAD), (dict(packed=_at(8)), BAD),
    (dict(w_up=P), BAD), (dict(gated=1), BAD), (dict(dt=B.MOE_MXFP8), UNS), (dict(N=0), BAD),
])
def test_pack_refusals(kw, status):
    v = dict(M=1, N=40, K=64, gated=0, w=P, w_up=None, dt=B.MOE_BF16, packed=P)
    v.update(kw)
    s = B._CDenseShape(v["M"], v["N"], v["K"], v["gated"])
    assert B.load().moe_pack_dense(ctypes.byref(s), v["w"], v["w_up"], v["dt"], v["packed"], None) == status


def test_packed_bytes():
    """Columns in whole 64-column pairs (32 of each weight when gated), the reduction in multiples of 64."""
    assert B.moe_packed_dense_bytes(B.DenseShape(5, 64, 64)) == 64 * 64 * 2
    assert B.moe_packed_dense_bytes(B.DenseShape(0, 65, 1)) == 128 * 64 * 2
    assert B.moe_packed_dense_bytes(B.DenseShape(5, 33, 65, gated=True)) == 128 * 128 * 2
    assert B.moe_packed_dense_bytes(B.DenseShape(5, 0, 64)) == 0


def test_binding_refuses_host_tensors():
    s = B.DenseShape(2, 64, 64)
    with pytest.raises(ValueError):
        B.moe_dense_gemm(s, torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros(64 * 64 * 2, dtype=torch.uint8))
    with pytest.raises(ValueError):
        B.moe_dense_gemm(s, torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros(64, dtype=torch.uint8))


@pytest.mark.parametrize("M", [-1, -(1 << 31), (1 << 21) + 1, (1 << 31) - 1])
def test_weights_do_not_depend_on_the_rows(M):
    """The size query and the packer look at N, K and gated only; the product refuses such an M."""
    assert B.moe_packed_dense_bytes(B.DenseShape(M, 65, 1)) == 128 * 64 * 2
    s = B._CDenseShape(M, 40, 64, 0)
    pack = B.load().moe_pack_dense
    # what comes after the shape is what is refused, before any HIP call
    assert pack(ctypes.byref(s), P, None, B.MOE_MXFP8, P, None) == UNS
    assert pack(ctypes.byref(s), None, None, B.MOE_BF16, P, None) == BAD
    assert _gemm(M=M) == (BAD if M < 0 else UNS)


def test_binding_refuses_an_output_of_another_type():
    s = B.DenseShape(2, 64, 64)
    a, packed = torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros(64 * 64 * 2, dtype=torch.uint8)
    with pytest.raises(TypeError, match="c_dtype"):
        B.moe_dense_gemm(s, a, packed, c=torch.zeros((2, 64), dtype=torch.float16), c_dtype=torch.float32)
    with pytest.raises(ValueError, match="GPU"):         # the same type is no conflict: the host tensors are refused
        B.moe_dense_gemm(s, a, packed, c=torch.zeros((2, 64)), c_dtype=torch.float32)
