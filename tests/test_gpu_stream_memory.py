"""Calls on a stream of their own that leave the workspace and the results to the binding."""
import pytest
import torch

from few_reference import make, pack
from moe_layer_03_amd import binding as B

pytestmark = pytest.mark.gpu

S = B.Shape(8, 512, 64, 4, 256, 0, 64)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def calls(mx, seed):
    d = make(S, mx=mx, seed=seed)
    packed = pack(S, d, mx=mx)
    layer, few = (B.moe_layer_mxfp8, B.moe_layer_few_tokens_mxfp8) if mx else (B.moe_layer, B.moe_layer_few_tokens)
    dense = B.DenseShape(S.T, 320, S.H, gated=True)
    w = B.moe_pack_dense(dense, d["gate"][0][:, :1].bfloat16().expand(-1, 320).contiguous(),
                         d["up"][0][:, :1].bfloat16().expand(-1, 320).contiguous())
    return [lambda **k: layer(S, d["x"], d["w_router"], packed, **k),
            lambda **k: few(S, d["x"], d["w_router"], packed, **k),
            lambda **k: B.moe_dense_gemm(dense, d["x"], w, B.MOE_EPI_SWIGLU, **k)]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("which", [0, 1, 2])
def test_the_current_stream_allocates_meanwhile(mx, which):
    """The side stream is behind; what the current stream allocates and fills right after the call is other memory."""
    call = calls(mx, 60)[which]
    ref = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = call(stream=side)
    size = max(B.moe_layer_workspace_bytes(S), B.moe_layer_workspace_bytes_mxfp8(S),
               B.moe_layer_few_tokens_workspace_bytes(S))
    junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (size, size // 2, size // 8) * 4]
    torch.cuda.synchronize()
    assert torch.equal(got, ref) and len(junk) == 12


@pytest.mark.parametrize("mx", [False, True])
def test_two_streams_leave_everything_to_the_call(mx):
    both = [calls(mx, 61), calls(mx, 62)]
    for which in range(3):
        ref = [c[which]() for c in both]
        streams = [torch.cuda.Stream() for _ in both]
        torch.cuda.synchronize()
        got = [[], []]
        for _ in range(10):
            for i, (c, st) in enumerate(zip(both, streams)):
                got[i].append(c[which](stream=st))
        torch.cuda.synchronize()
        assert all(torch.equal(r, g) for r, gs in zip(ref, got) for g in gs)


def test_a_result_outlives_its_reader():
    """A result that the current stream still reads when it is dropped is not handed to the side stream's next call."""
    call, other = calls(False, 63)[1], calls(False, 64)[1]
    ref = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(20_000_000)
    copy = got.clone()
    del got
    for _ in range(4):
        other(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy, ref)


def test_captured_on_its_own_stream():
    """A capture whose call names the capturing stream and leaves everything to the binding, replayed between eager
    calls."""
    call = calls(False, 65)[1]
    ref = call()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = call(stream=torch.cuda.current_stream())
    for _ in range(3):
        got.fill_(float("nan"))
        g.replay()
        assert torch.equal(call(), ref)
        torch.cuda.synchronize()
        assert torch.equal(got, ref)
