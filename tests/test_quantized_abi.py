"""The norm's, the int8 quantiser's and the int8 product's refusals, on the host before any HIP call (no GPU needed)."""
import contextlib
import ctypes
import math

import pytest
import torch

from moe_layer_03_amd import binding as B
from moe_layer_03_amd import quantized as Q

P = ctypes.c_void_p(0x1000)
BAD, UNS, OK = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_OK
F32, BF16, F16, MX, I8 = B.MOE_F32, B.MOE_BF16, B.MOE_F16, B.MOE_MXFP8, B.MOE_I8


def _at(n):
    return ctypes.c_void_p(0x1000 + n)


X, R, S, W, Y, C, SC = (ctypes.c_void_p(0x10000 * i) for i in range(1, 8))


def _norm(rows=4, H=64, x=X, xd=BF16, ldx=64, r=R, rd=BF16, ldr=64, t=S, lds=64, w=W, wd=BF16, eps=1e-6, y=Y, yd=BF16,
          ldy=64, q=C, qd=I8, ldq=64, sc=SC):
    return B.load().moe_add_rmsnorm(rows, H, x, xd, ldx, r, rd, ldr, t, lds, w, wd, eps, y, yd, ldy, q, qd, ldq, sc, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), BAD), (dict(H=0), BAD), (dict(H=-3), BAD), (dict(rows=(1 << 21) + 1), UNS),
    (dict(H=(1 << 18) + 1), UNS),
    (dict(xd=MX), UNS), (dict(xd=I8), UNS), (dict(rd=7), UNS), (dict(wd=I8), UNS), (dict(yd=MX), UNS),
    (dict(qd=BF16), UNS), (dict(qd=0), UNS), (dict(qd=MX, H=48), UNS),
    (dict(eps=0.0), BAD), (dict(eps=-1e-6), BAD), (dict(eps=math.nan), BAD), (dict(eps=math.inf), BAD), (dict(eps=1e-40), BAD),
    (dict(ldx=63), BAD), (dict(ldr=63), BAD), (dict(lds=63), BAD), (dict(ldy=63), BAD), (dict(ldq=63), BAD),
    (dict(x=None), BAD), (dict(r=None), BAD),            # a sum without a residual
    (dict(y=None, q=None), BAD), (dict(sc=None), BAD),
    (dict(x=_at(1)), BAD), (dict(x=_at(2), xd=F32), BAD), (dict(r=_at(1)), BAD), (dict(t=_at(1)), BAD),
    (dict(w=_at(1)), BAD), (dict(w=_at(2), wd=F32), BAD), (dict(y=_at(1)), BAD), (dict(y=_at(2), yd=F32), BAD),
    (dict(sc=_at(2)), BAD),
    (dict(t=X, rd=F32), BAD), (dict(t=X, lds=72), BAD), (dict(t=R, ldr=72), BAD), (dict(t=Y), BAD),
    (dict(y=X, yd=F32), BAD), (dict(y=X, ldy=72), BAD), (dict(y=R, rd=F32), BAD), (dict(y=R, ldr=72), BAD),
    (dict(rows=0, x=None, r=None, t=None, y=None, q=None), OK),
])
def test_norm_refusals(kw, status):
    assert _norm(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), BAD), (dict(K=0), BAD), (dict(rows=(1 << 21) + 1), UNS), (dict(K=(1 << 18) + 1), UNS),
    (dict(xd=MX), UNS), (dict(ldx=63), BAD), (dict(ldq=63), BAD), (dict(x=None), BAD), (dict(q=None), BAD),
    (dict(sc=None), BAD), (dict(x=_at(1)), BAD), (dict(xd=F32, x=_at(2)), BAD), (dict(sc=_at(2)), BAD),
    (dict(rows=0, x=None, q=None, sc=None), OK),
])
def test_quantise_refusals(kw, status):
    v = dict(rows=4, K=64, x=X, xd=BF16, ldx=64, q=C, ldq=64, sc=SC)
    v.update(kw)
    assert B.load().moe_quantize_int8(v["rows"], v["K"], v["x"], v["xd"], v["ldx"], v["q"], v["ldq"], v["sc"],
                                      None) == status


def _gemm(M=8, N=40, K=64, gated=0, a=P, lda=64, sa=P, packed=P, epi=0, bias=None, r=None, rd=0, ldr=40, c=C, cd=BF16,
          ldc=40):
    s = B._CDenseShape(M, N, K, gated)
    return B.load().moe_dense_gemm_int8(ctypes.byref(s), a, lda, sa, packed, epi, bias, r, rd, ldr, c, cd, ldc, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), BAD), (dict(N=0), BAD), (dict(K=0), BAD), (dict(gated=2), BAD),
    (dict(M=(1 << 21) + 1), UNS), (dict(N=(1 << 18) + 1, ldc=1 << 20), UNS), (dict(K=131072, lda=1 << 20), UNS),
    (dict(epi=6), BAD), (dict(epi=-1), BAD), (dict(epi=B.MOE_EPI_SWIGLU), BAD), (dict(gated=1), BAD),
    (dict(gated=1, epi=B.MOE_EPI_SILU), BAD), (dict(cd=MX), UNS), (dict(cd=I8), UNS), (dict(r=R, rd=9), UNS),
    (dict(lda=63), BAD), (dict(ldc=39), BAD), (dict(r=R, ldr=39), BAD),
    (dict(a=None), BAD), (dict(sa=None), BAD), (dict(packed=None), BAD), (dict(c=None), BAD),
    (dict(sa=_at(2)), BAD), (dict(packed=_at(8)), BAD), (dict(c=_at(1)), BAD), (dict(c=_at(2), cd=F32), BAD),
    (dict(r=_at(1), rd=BF16), BAD), (dict(r=_at(2), rd=F32), BAD), (dict(bias=_at(2)), BAD),
    (dict(r=C, rd=F32), BAD), (dict(r=C, rd=BF16, ldr=48), BAD),
    (dict(M=0, a=None, sa=None, c=None, packed=None), OK),
])
def test_gemm_refusals(kw, status):
    assert _gemm(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), BAD), (dict(dt=BF16, s=None, w=_at(1)), BAD), (dict(dt=F32, s=None, w=_at(2)), BAD),
    (dict(packed=_at(8)), BAD), (dict(w_up=P), BAD), (dict(gated=1), BAD), (dict(gated=1, w_up=P), BAD),
    (dict(dt=MX), UNS), (dict(N=0), BAD), (dict(K=131072), UNS), (dict(s=None), BAD), (dict(s=_at(2)), BAD),
    (dict(us=P), BAD), (dict(dt=BF16), BAD), (dict(dt=BF16, s=None, us=P), BAD),
])
def test_pack_refusals(kw, status):
    v = dict(M=1, N=40, K=64, gated=0, w=P, w_up=None, dt=I8, s=P, us=None, packed=P)
    v.update(kw)
    s = B._CDenseShape(v["M"], v["N"], v["K"], v["gated"])
    assert B.load().moe_pack_dense_int8(ctypes.byref(s), v["w"], v["w_up"], v["dt"], v["s"], v["us"], v["packed"],
                                        None) == status


def test_packed_bytes():
    """A byte a code, columns in whole pairs, the reduction in multiples of 128; a float32 scale per packed column."""
    size = Q.moe_packed_dense_bytes_int8
    assert size(B.DenseShape(5, 64, 128)) == 64 * 128 + 64 * 4
    assert size(B.DenseShape(0, 65, 1)) == 128 * 128 + 128 * 4
    assert size(B.DenseShape(-7, 33, 129, gated=True)) == 128 * 256 + 128 * 4
    assert size(B.DenseShape(5, 0, 64)) == 0
    assert size(B.DenseShape(5, 64, 131072)) == 0 and size(B.DenseShape(5, 64, 131071)) == 64 * 131072 + 256


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


D = B.DenseShape(4, 64, 64)
PACKED = t(1 << 16, dtype=torch.uint8)
A8, SA = t(4, 64, dtype=torch.int8), t(4, dtype=torch.float32)
CALLS = {
    "moe_add_rmsnorm": (lambda **k: Q.moe_add_rmsnorm(t(4, 64), t(64), t(4, 64), y_dtype=torch.float32, q_dtype=Q.MOE_I8,
                                                      **k), 4),
    "moe_quantize_int8": (lambda **k: Q.moe_quantize_int8(t(4, 64), **k), 2),
    "moe_pack_dense_int8": (lambda **k: Q.moe_pack_dense_int8(D, t(64, 64), **k), 1),
    "moe_dense_gemm_int8": (lambda **k: Q.moe_dense_gemm_int8(D, A8, SA, PACKED, **k), 1),
}


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("stream", [None, "side"])
def test_binding_refuses_host_tensors(name, stream, monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        CALLS[name][0](stream=stream)


class OnGpu(torch.Tensor):
    """A host tensor that says it is on the first GPU: what is refused here is refused before anything is launched."""
    is_cuda = True

    def get_device(self):
        return 0


def g(*shape, dtype=torch.bfloat16):
    return t(*shape, dtype=dtype).as_subclass(OnGpu)


@pytest.mark.parametrize("call,error", [
    (lambda: Q.moe_add_rmsnorm(g(4, 64), y=g(4, 64), codes=g(4, 64, dtype=torch.int8)), ValueError),
    (lambda: Q.moe_add_rmsnorm(g(4, 64), q_dtype=B.MOE_BF16), ValueError),
    (lambda: Q.moe_add_rmsnorm(g(4, 64), sum_out=g(4, 64)), ValueError),
    (lambda: Q.moe_add_rmsnorm(g(4, 64), None, g(4, 64), sum_out=g(4, 64, dtype=torch.float32)), TypeError),
    (lambda: Q.moe_add_rmsnorm(g(4, 64), None, g(4, 32)), ValueError),
    (lambda: Q.moe_add_rmsnorm(g(4, 64), None, t(4, 64)), ValueError),
    (lambda: Q.moe_add_rmsnorm(g(4, 64), g(32)), ValueError),
    (lambda: Q.moe_add_rmsnorm(g(4, 64), g(128)[::2]), ValueError),
    (lambda: Q.moe_add_rmsnorm(g(4, 64), g(64, dtype=torch.float64)), TypeError),
    (lambda: Q.moe_add_rmsnorm(g(64, 4).t(), y=g(4, 64)), ValueError),
    (lambda: Q.moe_add_rmsnorm(g(4, 64), y=g(1, 64).expand(4, 64)), ValueError),
    (lambda: Q.moe_add_rmsnorm(g(4, 64), y=g(4, 64), y_dtype=torch.float32), TypeError),
    (lambda: Q.moe_add_rmsnorm(g(4, 64), q_dtype=Q.MOE_I8, codes=g(4, 64, dtype=torch.uint8)), TypeError),
    (lambda: Q.moe_add_rmsnorm(g(4, 64), q_dtype=Q.MOE_I8, codes=g(4, 64, dtype=torch.int8),
                               scales=g(3, dtype=torch.float32)), ValueError),
    (lambda: Q.moe_add_rmsnorm(g(4, 64, dtype=torch.int8), y=g(4, 64)), TypeError),
    (lambda: Q.moe_quantize_int8(g(4, 64), codes=g(4, 64, dtype=torch.uint8)), TypeError),
    (lambda: Q.moe_quantize_int8(g(4, 64), codes=g(4, 64, dtype=torch.int8), scales=g(4)), TypeError),
    (lambda: Q.moe_dense_gemm_int8(D, g(4, 64), SA, PACKED), TypeError),
    (lambda: Q.moe_dense_gemm_int8(D, g(4, 64, dtype=torch.int8), SA, g(64, dtype=torch.uint8)), ValueError),
    (lambda: Q.moe_dense_gemm_int8(D, g(4, 64, dtype=torch.int8), SA, PACKED, c=g(4, 64), c_dtype=torch.float32), TypeError),
    (lambda: Q.moe_dense_gemm_int8(D, g(4, 64, dtype=torch.int8), SA, PACKED, c=g(4, 64), bias=g(64)), TypeError),
    (lambda: Q.moe_dense_gemm_int8(D, g(4, 32, dtype=torch.int8), SA, PACKED, c=g(4, 64)), ValueError),
    (lambda: Q.moe_pack_dense_int8(D, t(64, 64), packed=t(64, dtype=torch.uint8)), ValueError),
])
def test_binding_refusals(call, error):
    with pytest.raises(error):
        call()


class Recorded(torch.Tensor):
    is_cuda = True

    def record_stream(self, stream):
        self.recorded = getattr(self, "recorded", []) + [stream]


@pytest.mark.parametrize("stream", [None, "side"])
@pytest.mark.parametrize("name", list(CALLS))
def test_what_a_call_allocates_belongs_to_its_stream(name, stream, monkeypatch):
    real, empty, log, active = B.load(), torch.empty, [], []

    class Library:
        def __getattr__(self, fn):
            return getattr(real, fn) if "_bytes" in fn else lambda *a: OK

    @contextlib.contextmanager
    def on(s):
        active.append(s)
        yield
        active.pop()

    def allocate(n, dtype=None, device=None):
        v = empty(n, dtype=dtype).as_subclass(Recorded)
        log.append((active[-1] if active else None, v))
        return v
    monkeypatch.setattr(B, "load", Library)
    for module, fn in ((B, "_ptr"), (B, "_stream_on"), (B, "_same_device"), (Q, "_flat"), (Q, "_stream")):
        monkeypatch.setattr(module, fn, lambda *a, **k: None)
    monkeypatch.setattr(Q, "_rows", lambda *a: (None, 0))
    monkeypatch.setattr(Q, "_index", lambda *a: 0)
    monkeypatch.setattr(Q, "_dense_int8_of", Q._dense_int8_of.__wrapped__)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: "current")
    monkeypatch.setattr(torch, "empty", allocate)
    call, count = CALLS[name]
    call(stream=stream)
    assert [s for s, _ in log] == [stream] * count
    assert all(getattr(v, "recorded", None) == (["current"] if stream else None) for _, v in log)


@pytest.mark.parametrize("current,stream,good", [(0, None, True), (0, 0, True), (0, 1, False), (1, None, False), (1, 0, False)])
def test_the_stream_is_on_the_tensors_device(current, stream, good, monkeypatch):
    """Tensors on cuda:0, whatever the current device and the stream's."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current)
    monkeypatch.setattr(Q, "_current_device", lambda: current)
    monkeypatch.setattr(Q, "_current_stream", lambda i: 0x40 + i)
    given = None if stream is None else type("Stream", (), {"cuda_stream": 0x40, "device": torch.device("cuda", stream)})()
    if good:
        assert Q._stream(0, given) == 0x40
    else:
        with pytest.raises(ValueError, match="tensors are on cuda:0"):
            Q._stream(0, given)


def test_every_entry_point_is_here():
    assert {n for n in B.EXPORTED if hasattr(Q, n) and "_bytes" not in n} == set(CALLS)
    assert all(hasattr(B, n) or hasattr(Q, n) or n in (
        "moe_status_string", "moe_last_hip_error", "moe_probe_mfma_bf16_flops") for n in B.EXPORTED)
