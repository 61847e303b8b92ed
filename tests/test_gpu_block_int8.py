"""8-bit rows as a server uses them: the norm before the feed-forward half, its rows to the router and the experts, a
shared expert in int8 added onto their sum, eager and captured."""
import pytest
import torch

from few_reference import make, pack
from moe_layer_03_amd import binding as B
from moe_layer_03_amd import quantized as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("T", [1, 40, 300])
def test_normed_rows_through_the_mxfp8_experts(T):
    """The norm's MXFP8 rows, gathered by the grouped product, and its y for the router: what moe_layer_mxfp8 makes of y
    where y holds the normed rows whole (float32 rows whose values bf16 holds)."""
    H, E, K, I = 512, 16, 4, 256
    s = B.Shape(T, H, E, K, I, 0, E)
    d = make(s, mx=True, seed=T)
    packed = pack(s, d, mx=True)
    g = torch.Generator().manual_seed(T)
    # rows of +-1 times a power of two have a mean square of a power of four, so y is exact in bf16; eps vanishes
    sign = torch.randint(0, 2, (T, H), generator=g) * 2.0 - 1
    x = (sign * 2.0 ** 20).bfloat16().cuda()
    w = (torch.randint(-8, 9, (H,), generator=g) / 8.0).bfloat16().cuda()
    _, y, codes, scales = Q.moe_add_rmsnorm(x, w, eps=2.0 ** -126, y_dtype=torch.bfloat16, q_dtype=Q.MOE_MXFP8)
    assert torch.equal(y.float(), (x.float() / 2.0 ** 20) * w.float())
    ref = B.moe_layer_mxfp8(s, y, d["w_router"], packed)
    idx, tw, _ = B.moe_route(s, y, d["w_router"])
    m = B.moe_dispatch(s, idx)
    hc, hs = B.moe_grouped_gemm_mxfp8(s, codes, scales, m["offsets"], packed, B.MOE_GEMM_GATE_UP, B.MOE_EPI_SWIGLU,
                                      c_dtype=torch.uint8, a_rows=m["row_token"])
    out = B.moe_combine(s, B.moe_grouped_gemm_mxfp8(s, hc, hs, m["offsets"], packed, B.MOE_GEMM_DOWN), m["slot_row"], tw)
    assert torch.equal(out, ref)


class Block:
    """Norm, routed experts of y, shared expert of the codes onto their sum, and the sum into the stream's next norm."""

    def __init__(self, T, seed):
        H, I = 512, 256
        self.s = B.Shape(T, H, 64, 4, I, 0, 64)
        self.d = make(self.s, seed=seed)
        g = torch.Generator().manual_seed(seed + 1)
        mk = lambda *n, std=1.0: (torch.randn(n, generator=g) * std).bfloat16().cuda()   # noqa: E731
        self.attn, self.stream = mk(T, H), mk(T, H)
        self.w1, self.w2 = mk(H), mk(H)
        self.wg, self.wu, self.wd = mk(H, I, std=0.04), mk(H, I, std=0.04), mk(I, H, std=0.04)
        self.gu, self.dn = B.DenseShape(T, I, H, gated=True), B.DenseShape(T, H, I)
        self.experts = pack(self.s, self.d)
        self.p_gu = Q.moe_pack_dense_int8(self.gu, self.wg, self.wu)
        self.p_dn = Q.moe_pack_dense_int8(self.dn, self.wd)

    def step(self):
        h, y, codes, scales = Q.moe_add_rmsnorm(self.attn, self.w1, self.stream, y_dtype=torch.bfloat16, q_dtype=Q.MOE_I8)
        out = B.moe_layer_few_tokens(self.s, y, self.d["w_router"], self.experts) if self.s.T <= 32 else B.moe_layer(
            self.s, y, self.d["w_router"], self.experts)
        if not torch.cuda.is_current_stream_capturing():
            self.routed = out.clone()
        self.g = Q.moe_dense_gemm_int8(self.gu, codes, scales, self.p_gu, B.MOE_EPI_SWIGLU)
        self.h, self.y, self.codes, self.scales = h, y, codes, scales
        Q.moe_dense_gemm_int8(self.dn, *Q.moe_quantize_int8(self.g), self.p_dn, residual=out, c=out)
        return out, Q.moe_add_rmsnorm(out, self.w2, h, q_dtype=Q.MOE_I8)


@pytest.mark.parametrize("T", [1, 7, 32, 200])
def test_step(T):
    b = Block(T, seed=T)
    out, (h2, _, _, _) = b.step()
    # the shared expert against its unquantised form.  A code is off by a uniform +-0.5, 0.29 as a standard deviation, of
    # 1 / 127 of the largest of 512 (256) values: 3.3 (3.0) standard deviations of normal ones, 0.8 % of one each for rows
    # and columns, 1.1 % for a product.  Gate and up make 1.6 % of the SwiGLU rows (2 % with silu's slope), whose largest
    # is some 8 of their standard deviations: 1.8 % more, and 0.7 % for the last columns: 3 % in all, and some spread
    y = b.y.double()
    a, u = y @ b.wg.double(), y @ b.wu.double()
    shared = (a * torch.sigmoid(a) * u) @ b.wd.double()
    got = out.double() - b.routed.double()
    assert (got - shared).pow(2).mean().sqrt() <= 0.05 * shared.pow(2).mean().sqrt()
    assert torch.equal(h2, (out + b.h.float()).bfloat16())


def test_step_captured():
    """One graph of the whole step, replayed on new inputs with eager steps between."""
    b = Block(5, seed=50)
    b.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, nxt = b.step()
    kept = [out, nxt[0], nxt[2], nxt[3]]
    for i in range(4):
        n = Block(5, seed=51 + i)
        b.attn.copy_(n.attn)
        b.stream.copy_(n.stream)
        out, nxt = b.step()
        eager = [t.clone() for t in (out, nxt[0], nxt[2], nxt[3])]
        for t in kept:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(kept, eager))
