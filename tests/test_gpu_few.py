"""The few-token layer on the GPU against the definition in 64 bits."""
import pytest
import torch

from few_reference import check, make, pack, reference
from moe_layer_03_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def call(s, d, packed, mx=False, **kw):
    idx = torch.full((s.T, s.K), -7, dtype=torch.int32, device="cuda")
    w = torch.full((s.T, s.K), float("nan"), device="cuda")
    out = torch.full((s.T + 2, s.H), float("nan"), device="cuda")
    ws = torch.full((B.moe_layer_few_tokens_workspace_bytes(s),), 0xFF, dtype=torch.uint8, device="cuda")
    f = B.moe_layer_few_tokens_mxfp8 if mx else B.moe_layer_few_tokens
    r = f(s, d["x"], d["w_router"], packed, d["bias"], out=out[: s.T], ws=ws, topk_idx=idx, topk_w=w, **kw)
    torch.cuda.synchronize()
    assert torch.isnan(out[s.T:]).all()         # rows behind the last token are left alone
    return r, idx, w


def run(s, dtype="bf16", mx=False, **kw):
    d = make(s, dtype, mx, **kw)
    got, idx, w = call(s, d, pack(s, d, dtype, mx), mx)
    check(s, d, got, idx, w)


SHAPES = [  # T, H, E, K, I, e_begin, e_end
    (1, 64, 4, 1, 64, 0, 4),
    (1, 256, 8, 2, 128, 0, 8),
    (2, 64, 5, 5, 64, 1, 3),
    (3, 192, 17, 3, 320, 0, 17),
    (5, 512, 128, 8, 192, 16, 24),
    (15, 128, 33, 4, 64, 3, 30),
    (16, 1024, 128, 8, 128, 0, 128),
    (17, 320, 130, 8, 64, 2, 100),
    (31, 64, 8, 8, 448, 0, 8),
    (32, 256, 64, 2, 256, 8, 40),
    (7, 128, 300, 64, 64, 100, 300),
    (4, 64, 1000, 7, 64, 0, 1000),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer(shape, dtype):
    run(B.Shape(*shape), dtype, seed=sum(shape), bias=shape[0] % 2 == 1)


@pytest.mark.parametrize("shape", [(1, 256, 4, 1, 256, 0, 4), (3, 512, 17, 3, 256, 2, 11), (16, 256, 128, 8, 512, 0, 128),
                                   (19, 1024, 16, 4, 256, 0, 16), (32, 256, 8, 8, 768, 4, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_mxfp8(shape, dtype):
    run(B.Shape(*shape), dtype, mx=True, seed=sum(shape), bias=shape[0] % 2 == 1)


def test_layer_full_width():
    """Hidden 4096, expert 1536, top-8 of 128, both weight formats; 4096 / 8 additions a wave."""
    s = B.Shape(6, 4096, 128, 8, 1536, 40, 60)
    run(s, "bf16", seed=1)
    run(s, "bf16", mx=True, seed=2)


def test_limits_of_the_tables():
    """The largest routing tables: 32 tokens, 64 of 1024 experts each."""
    run(B.Shape(32, 64, 1024, 64, 64, 0, 1024), seed=3)


def test_ties_go_to_the_lower_index():
    s = B.Shape(9, 128, 40, 6, 64, 0, 40)
    d = make(s, seed=4)
    d["w_router"][:, 20:] = d["w_router"][:, :20]          # pairs of equal logits
    got, idx, w = call(s, d, pack(s, d))
    check(s, d, got, idx, w)
    d["w_router"].zero_()                                   # all equal
    got, idx, w = call(s, d, pack(s, d))
    assert (idx.cpu() == torch.arange(6, dtype=torch.int32)).all()
    check(s, d, got, idx, w)


def test_signed_zero_logits_tie():
    s = B.Shape(1, 64, 4, 2, 64, 0, 4)
    d = make(s, seed=5)
    d["x"].zero_()
    d["bias"] = torch.tensor([-0.0, 0.0, -0.0, 0.0], device="cuda")
    _, idx, w = call(s, d, pack(s, d))
    assert idx.cpu().tolist() == [[0, 1]]
    assert w.cpu().tolist() == [[0.5, 0.5]]


def test_near_ties_are_decided_in_double():
    """Logits a float32 sum cannot tell apart: 1 + 2^-24-sized differences in the products."""
    s = B.Shape(1, 64, 4, 1, 64, 0, 4)
    d = make(s, seed=6)
    d["x"] = torch.zeros_like(d["x"])
    d["x"][0, :3] = torch.tensor([1.0, 2.0 ** -20, 2.0 ** -20])
    d["w_router"].zero_()
    d["w_router"][0] = 1.0
    d["w_router"][1] = torch.tensor([0.0, 2.0 ** -6, 2.0 ** -5, 2.0 ** -7])
    _, idx, _ = call(s, d, pack(s, d))
    assert idx.item() == 2


def test_no_local_expert():
    """Tokens whose experts are all elsewhere: exact zeros, for some tokens and for all."""
    s = B.Shape(12, 128, 64, 2, 64, 60, 64)
    run(s, seed=7)
    d = make(s, seed=8)
    d["bias"] = torch.zeros(64, device="cuda")
    d["bias"][:30] = 1000.0
    got, idx, w = call(s, d, pack(s, d))
    assert (idx < 30).all() and (got == 0).all()


def test_every_token_one_expert():
    s = B.Shape(32, 256, 8, 1, 128, 2, 6)
    d = make(s, seed=9)
    d["bias"] = torch.zeros(8, device="cuda")
    d["bias"][4] = 1000.0
    got, idx, w = call(s, d, pack(s, d))
    assert (idx == 4).all() and (w == 1).all()
    check(s, d, got, idx, w)


def test_no_tokens():
    s = B.Shape(0, 128, 8, 2, 64, 0, 8)
    x = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    d = make(B.Shape(1, 128, 8, 2, 64, 0, 8), seed=10)
    out = B.moe_layer_few_tokens(s, x, d["w_router"], pack(s, d))
    assert out.shape == (0, 128)


def test_agrees_with_moe_layer():
    """The same experts as moe_layer, and its output within the fp16 roundings that moe_layer makes."""
    s = B.Shape(24, 512, 128, 8, 256, 0, 64)
    d = make(s, seed=11)
    packed = pack(s, d)
    got, idx, w = call(s, d, packed)
    i2 = torch.empty_like(idx)
    w2 = torch.empty_like(w)
    ref = B.moe_layer(s, d["x"], d["w_router"], packed, topk_idx=i2, topk_w=w2)
    assert torch.equal(idx, i2)
    assert (w - w2).abs().max().item() <= 2e-6
    assert (got - ref).abs().max().item() <= 2e-2 * ref.pow(2).mean().sqrt().item()


def test_shards_add_up():
    d = make(B.Shape(10, 256, 32, 4, 128, 0, 32), seed=12)
    total = 0.0
    for b in (0, 5, 6, 20):
        e = {0: 5, 5: 6, 6: 20, 20: 32}[b]
        s = B.Shape(10, 256, 32, 4, 128, b, e)
        part = dict(d, **{k: d[k][b:e].contiguous() for k in ("gate", "up", "down")})
        total = total + call(s, part, pack(s, part))[0].double()
    ref, _, _, bound = reference(B.Shape(10, 256, 32, 4, 128, 0, 32), d)
    assert ((total - ref).abs() <= bound + 4 * 2.0 ** -24 * ref.abs()).all()


@pytest.mark.parametrize("T", [1, 4, 6, 13, 27])
@pytest.mark.parametrize("mx,dtype", [(False, "bf16"), (False, "f32"), (True, "bf16"), (True, "f32")])
def test_nan_stays_in_its_token(T, mx, dtype):
    s = B.Shape(T, 256, 24, 4, 256, 0, 24)
    d = make(s, dtype, mx, seed=31)
    d["x"][T // 2, 5] = float("nan")
    got, idx, w = call(s, d, pack(s, d, dtype, mx), mx)
    assert ((idx >= 0) & (idx < s.E)).all() and all(len(set(r)) == s.K for r in idx.tolist())
    rest = [t for t in range(T) if t != T // 2]
    assert torch.isnan(got[T // 2]).all() and torch.isnan(w[T // 2]).all()
    assert torch.isfinite(got[rest]).all() and torch.isfinite(w[rest]).all()


@pytest.mark.parametrize("mx", [False, True])
def test_repeats_bit_for_bit(mx):
    s = B.Shape(20, 512, 128, 8, 256, 0, 128)
    d = make(s, mx=mx, seed=13)
    packed = pack(s, d, mx=mx)
    first = call(s, d, packed, mx)
    for _ in range(5):
        again = call(s, d, packed, mx)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_two_streams_at_once():
    """Overlapping calls with workspaces of their own."""
    s = B.Shape(8, 1024, 128, 8, 512, 0, 128)
    d = [make(s, seed=20 + i) for i in range(2)]
    packed = [pack(s, v) for v in d]
    ref = [call(s, v, p)[0] for v, p in zip(d, packed)]
    streams = [torch.cuda.Stream() for _ in d]
    n = B.moe_layer_few_tokens_workspace_bytes(s)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in d]
    outs = [torch.empty((s.T, s.H), device="cuda") for _ in d]
    torch.cuda.synchronize()
    for _ in range(20):
        for v, p, q, o, st in zip(d, packed, ws, outs, streams):
            B.moe_layer_few_tokens(s, v["x"], v["w_router"], p, out=o, ws=q, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, outs))


def test_captured_and_replayed():
    """A captured call replayed on new inputs, eager calls between the replays."""
    s = B.Shape(4, 512, 64, 4, 256, 0, 64)
    d = make(s, seed=30)
    packed = pack(s, d)
    ws = torch.empty(B.moe_layer_few_tokens_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    out = torch.empty((s.T, s.H), device="cuda")
    call(s, d, packed)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.moe_layer_few_tokens(s, d["x"], d["w_router"], packed, out=out, ws=ws)
    for i in range(4):
        d["x"].copy_(make(s, seed=31 + i)["x"])
        eager = call(s, d, packed)[0]
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


@pytest.mark.parametrize("dtype,mx", [("bf16", False), ("f32", False), ("bf16", True), ("f32", True)])
@pytest.mark.parametrize("T", [9, 17, 32])
def test_crowded_experts(dtype, mx, T):
    """Experts that more tokens choose than an MFMA tile has rows, beside experts with one token: several row
    segments of one expert, shared out over workgroups."""
    s = B.Shape(T, 256, 96, 4, 256, 0, 90)
    d = make(s, dtype, mx, seed=40 + T)
    d["bias"] = torch.zeros(96, device="cuda")
    d["bias"][torch.tensor([3, 64, 91])] = torch.tensor([2.0, 1.2, 1.5], device="cuda")
    got, idx, w = call(s, d, pack(s, d, dtype, mx), mx)
    check(s, d, got, idx, w)


def test_every_token_every_expert():
    """32 tokens that all choose the same 8 experts."""
    run(B.Shape(32, 320, 8, 8, 192, 0, 8), seed=44)
    run(B.Shape(32, 256, 8, 8, 512, 0, 8), mx=True, seed=45)
