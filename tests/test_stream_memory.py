"""Memory that the binding allocates itself belongs to the stream that the call runs on (no GPU needed): each entry
point is called with everything optional left out, its library replaced by one that does nothing."""
import contextlib

import pytest
import torch

from moe_layer_03_amd import binding as B

S = B.Shape(4, 256, 8, 2, 256, 0, 8)
D = B.DenseShape(4, 64, 64)


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


X, WR, W, PACKED = t(4, 256), t(256, 8), t(8, 256, 256), t(1 << 23, dtype=torch.uint8)
IDX, TW, OFF = t(4, 2, dtype=torch.int32), t(4, 2, dtype=torch.float32), t(9, dtype=torch.int32)

CALLS = {
    "moe_pack_weights": (lambda **k: B.moe_pack_weights(S, W, W, W, **k), 1),
    "moe_route": (lambda **k: B.moe_route(S, X, WR, want_logits=True, **k), 4),
    "moe_route_from_logits": (lambda **k: B.moe_route_from_logits(S, t(4, 8, dtype=torch.float32), **k), 2),
    "moe_dispatch": (lambda **k: B.moe_dispatch(S, IDX, X, **k), 7),
    "moe_grouped_gemm": (lambda **k: B.moe_grouped_gemm(S, t(8, 256), OFF, PACKED, B.MOE_GEMM_GATE_UP, **k), 1),
    "moe_combine": (lambda **k: B.moe_combine(S, X, IDX, TW, **k), 1),
    "moe_layer": (lambda **k: B.moe_layer(S, X, WR, PACKED, **k), 2),
    "moe_layer_noalloc": (lambda **k: B.moe_layer_noalloc(S, X, WR, PACKED, **k), 1),
    "moe_pack_weights_mxfp8": (lambda **k: B.moe_pack_weights_mxfp8(S, W, W, W, **k), 1),
    "moe_quantize_mxfp8": (lambda **k: B.moe_quantize_mxfp8(X, **k), 2),
    "moe_grouped_gemm_mxfp8": (lambda **k: B.moe_grouped_gemm_mxfp8(
        S, t(4, 256, dtype=torch.uint8), t(4, 8, dtype=torch.uint8), OFF, PACKED, B.MOE_GEMM_GATE_UP,
        B.MOE_EPI_SWIGLU, c_dtype=torch.uint8, **k), 2),
    "moe_layer_mxfp8": (lambda **k: B.moe_layer_mxfp8(S, X, WR, PACKED, **k), 2),
    "moe_layer_few_tokens": (lambda **k: B.moe_layer_few_tokens(S, X, WR, PACKED, **k), 2),
    "moe_layer_few_tokens_mxfp8": (lambda **k: B.moe_layer_few_tokens_mxfp8(S, X, WR, PACKED, **k), 2),
    "moe_pack_dense": (lambda **k: B.moe_pack_dense(D, t(64, 64), **k), 1),
    "moe_dense_gemm": (lambda **k: B.moe_dense_gemm(D, t(4, 64), PACKED, **k), 1),
}


class Recorded(torch.Tensor):
    """A tensor that notes which streams it is recorded for, and says that it is on the GPU."""
    is_cuda = True

    def record_stream(self, stream):
        self.recorded = getattr(self, "recorded", []) + [stream]


@pytest.fixture
def allocations(monkeypatch):
    """[(stream in force, tensor)] of every torch.empty, the library's launches and the GPU checks taken out."""
    real, empty = B.load(), torch.empty
    log, active = [], []

    class Library:
        def __getattr__(self, name):
            return getattr(real, name) if "_bytes" in name else lambda *a: B.MOE_OK

    @contextlib.contextmanager
    def on(stream):
        active.append(stream)
        yield
        active.pop()

    def allocate(n, dtype=None, device=None):
        v = empty(n, dtype=dtype).as_subclass(Recorded)
        log.append((active[-1] if active else None, v))
        return v
    monkeypatch.setattr(B, "load", Library)
    for name in ("_ptr", "_stream", "_stream_on", "_same_device"):
        monkeypatch.setattr(B, name, lambda *a, **k: None)
    monkeypatch.setattr(B, "_rows", lambda *a: (None, 0))
    for name in ("_few_tokens_of", "_dense_of"):         # past their caches, which outlive this test
        monkeypatch.setattr(B, name, getattr(B, name).__wrapped__)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: "current")
    monkeypatch.setattr(torch, "empty", allocate)
    return log


def test_every_entry_point_is_here():
    other = {"moe_route_screen_layout", "moe_probe_mfma_bf16"}          # nothing of theirs is allocated
    assert {n for n in B.EXPORTED if hasattr(B, n) and "_bytes" not in n} - other == set(CALLS)


@pytest.mark.parametrize("name", list(CALLS))
def test_allocated_on_the_call_s_stream(name, allocations):
    call, count = CALLS[name]
    r = call(stream="side")
    assert len(allocations) == count
    assert [s for s, _ in allocations] == ["side"] * count
    # what the caller gets is also kept from reuse until the current stream has read it
    results = {id(v) for v in (r if isinstance(r, tuple) else r.values() if isinstance(r, dict) else (r,))}
    for _, v in allocations:
        assert (id(v) in results) == (getattr(v, "recorded", []) == ["current"])


def test_host_tensors_are_refused_with_a_stream_too(monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    for call in (lambda: B.moe_layer(S, X, WR, PACKED, stream="side"),
                 lambda: B.moe_dense_gemm(D, t(4, 64), PACKED, stream="side")):
        with pytest.raises(ValueError, match="must be a GPU tensor"):
            call()


@pytest.mark.parametrize("name", list(CALLS))
def test_allocated_on_the_current_stream(name, allocations):
    CALLS[name][0]()
    assert [s for s, _ in allocations] == [None] * CALLS[name][1]
    assert not any(hasattr(v, "recorded") for _, v in allocations)


@pytest.mark.parametrize("current,stream,good", [(0, 0, True), (0, 1, False), (1, 0, False)])
def test_the_stream_is_on_the_tensors_device(current, stream, good, monkeypatch):
    """Tensors on cuda:0, whatever the current device and the stream's."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current)
    given = type("Stream", (), {"cuda_stream": 0x40, "device": torch.device("cuda", stream)})()
    if good:
        assert B._stream_on(torch.device("cuda", 0), given) == 0x40
    else:
        with pytest.raises(ValueError, match="tensors are on cuda:0"):
            B._stream_on(torch.device("cuda", 0), given)
