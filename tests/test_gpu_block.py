"""The feed-forward half of a decode step as a server runs it: an output projection with its residual, the routed
experts of the result, a shared expert's two dense products added onto their sum."""
import pytest
import torch

from few_reference import make, pack, reference
from moe_layer_03_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Block:
    def __init__(self, T, mx, seed):
        H, I, D = 512, 256, 384
        self.s = B.Shape(T, H, 64, 4, I, 0, 64)
        self.mx = mx
        self.d = make(self.s, mx=mx, seed=seed)
        g = torch.Generator().manual_seed(seed + 1)
        mk = lambda *n, std=1.0: (torch.randn(n, generator=g) * std).bfloat16().cuda()
        self.attn, self.hidden = mk(T, D), mk(T, H)
        self.w_o, self.wg, self.wu, self.wd = mk(D, H, std=0.04), mk(H, I, std=0.04), mk(H, I, std=0.04), mk(I, H, std=0.04)
        self.bias_o = torch.randn((1, H), generator=g).cuda()
        self.so, self.sgu, self.sd = B.DenseShape(T, H, D), B.DenseShape(T, I, H, gated=True), B.DenseShape(T, H, I)
        self.packed = pack(self.s, self.d, mx=mx)
        self.p_o = B.moe_pack_dense(self.so, self.w_o)
        self.p_gu = B.moe_pack_dense(self.sgu, self.wg, self.wu)
        self.p_d = B.moe_pack_dense(self.sd, self.wd)
        self.ws = torch.empty(B.moe_layer_few_tokens_workspace_bytes(self.s), dtype=torch.uint8, device="cuda")
        self.x = torch.empty_like(self.hidden)
        self.h = torch.empty((T, I), dtype=torch.bfloat16, device="cuda")
        self.out = torch.empty((T, H), device="cuda")

    def step(self):
        layer = B.moe_layer_few_tokens_mxfp8 if self.mx else B.moe_layer_few_tokens
        B.moe_dense_gemm(self.so, self.attn, self.p_o, bias=self.bias_o, residual=self.hidden, c=self.x)
        layer(self.s, self.x, self.d["w_router"], self.packed, out=self.out, ws=self.ws)
        B.moe_dense_gemm(self.sgu, self.x, self.p_gu, B.MOE_EPI_SWIGLU, c=self.h)
        B.moe_dense_gemm(self.sd, self.h, self.p_d, residual=self.out, c=self.out)
        return self.out


@pytest.mark.parametrize("T", [1, 7, 32])
@pytest.mark.parametrize("mx", [False, True])
def test_step(T, mx):
    b = Block(T, mx, seed=T)
    got = b.step()
    torch.cuda.synchronize()
    x = b.attn.double() @ b.w_o.double() + b.bias_o.double() + b.hidden.double()
    assert ((b.x.double() - x).abs() <= (2.0 ** -8 + 2.0 ** -12) * x.abs() + 1e-4).all()   # one bf16 rounding
    # from the rounded rows on: the experts to float32, the shared expert through a bf16 h
    ref, _, _, bound = reference(b.s, dict(b.d, x=b.x))
    a, u = b.x.double() @ b.wg.double(), b.x.double() @ b.wu.double()
    h = a * torch.sigmoid(a) * u
    assert ((b.h.double() - h).abs() <= (2.0 ** -8 + 2.0 ** -12) * h.abs() + 1e-4).all()
    ref = ref + b.h.double() @ b.wd.double()
    # float32 sums of I products and one addition
    bound = bound + (b.s.I + 2) * 2.0 ** -24 * (b.h.double().abs() @ b.wd.double().abs() + ref.abs())
    assert ((got.double() - ref).abs() <= bound).all()


def test_step_captured():
    """One graph of the whole step, replayed on new inputs with eager steps between."""
    b = Block(3, False, seed=50)
    b.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.step()
    for i in range(4):
        n = Block(3, False, seed=51 + i)
        b.attn.copy_(n.attn)
        b.hidden.copy_(n.hidden)
        eager = b.step().clone()
        b.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.out, eager)
