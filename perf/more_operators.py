"""The norm with the residual's sum and 8-bit rows, the int8 row quantiser and the int8 product: cases, inputs, plain
forms and exact values.

``listed()`` and ``draw(rng)`` give the cases, ``prepare`` their inputs, ``run`` one pass (the plain form in elementary
torch operations, or the library's call where ``own`` is true), ``work`` the bytes and operations a pass cannot do
without, ``exact`` the outputs from the definition in 64 bits.

Norm cases ("norm"): h = x + residual rounded to the residual's type (no residual: x), s = 1 / sqrt(mean(h^2) + eps)
in double, rounded to float32, v = (h s) w in float32; y is v rounded, and the codes are v's: "int8" with a scale per
row, "mxfp8" E4M3 codes with a power-of-two scale per 32.

Quantiser cases ("quantise"): int8 codes of given rows; scale = largest |v| / 127 in float32 (2^-126 at least), codes
v / scale to the nearest integer.

Product cases ("product"): C = act((A W) sa sw + bias) + residual with codes A [M, K], W [K, N], a scale per row of A
and per column of W; "swiglu" has a gate and an up weight.

``pad`` is the extra length of the rows of x, the residual and A in memory.
"""
import math

import torch

own = False

EPS = 1e-6
SMALLEST = 2.0 ** -126            # least scale of int8 rows
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}


def _norm(name, rows, H, x="bf16", residual="bf16", y="bf16", q="int8", pad=0):
    return {"name": name, "op": "norm", "rows": rows, "H": H, "x": x, "residual": residual, "y": y, "q": q, "pad": pad}


def _quantise(name, rows, K, x="bf16", pad=0):
    return {"name": name, "op": "quantise", "rows": rows, "K": K, "x": x, "pad": pad}


def _product(name, M, N, K, act="none", c="bf16", bias=False, residual="none", pad=0):
    return {"name": name, "op": "product", "M": M, "N": N, "K": K, "act": act, "c": c, "bias": bias,
            "residual": residual, "pad": pad}


def listed():
    return [
        # one sequence being decoded: the sum goes on as the residual stream, the codes into the next product
        _norm("norm 1 row int8", 1, 4096, y="none"),
        # the tiny workload's float32 rows, the norm alone
        _norm("norm 64 rows f32", 64, 256, x="f32", residual="none", y="f32", q="none"),
        # a decode batch: the experts' float32 sum is added, the router reads y and MXFP8 experts the codes
        _norm("norm 128 rows mxfp8", 128, 4096, x="f32", q="mxfp8"),
        # an odd size, fp16 rows apart in memory
        _norm("norm odd rows f16", 1001, 2311, x="f16", residual="f16", y="f16", pad=5),
        # the prefill batch, everything written
        _norm("norm 6000 rows int8", 6000, 4096),
        # the SwiGLU rows of a decode batch between a shared expert's products
        _quantise("quantise 128 rows", 128, 1536),
        # the same rows of the skewed prefill batch
        _quantise("quantise 16384 rows", 16384, 1536),
        # a shared expert's gate and up projection for one token
        _product("product 1 row swiglu", 1, 1536, 4096, act="swiglu"),
        # its down projection for a small batch, added onto the routed experts' float32 sum
        _product("product 16 rows add f32", 16, 4096, 1536, c="f32", residual="f32"),
        # a decode batch through an output projection with bias and residual
        _product("product 128 rows residual", 128, 4096, 4096, bias=True, residual="bf16"),
        # an odd size all round over a ragged batch
        _product("product odd f16 gelu", 1000, 1003, 1100, act="gelu", c="f16", bias=True, pad=4),
        # the prefill batch through a dense MLP's first projection
        _product("product 6000 rows silu", 6000, 4096, 4096, act="silu", bias=True),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    """One more case of the ranges that the listed ones stand for."""
    kind = rng.random()
    if kind < 0.65:
        H = _spread(rng, 64, 8192)
        if rng.random() < 0.75:       # most hidden sizes are round ones
            H = (H + 63) // 64 * 64
        rows = _spread(rng, 1, 6000 * 4096 // max(H, 4096))
        pad = rng.choice([0, 0, 0, 8, rng.randint(1, 9)])
        if kind < 0.2:
            return {"op": "quantise", "rows": rows, "K": H, "x": rng.choice(["bf16", "f16", "f32"]), "pad": pad}
        q = rng.choice(["none", "int8", "int8", "mxfp8"])
        if q == "mxfp8":
            H = (H + 31) // 32 * 32
        return {"op": "norm", "rows": rows, "H": H, "x": rng.choice(["bf16", "f16", "f32"]),
                "residual": rng.choice(["none", "bf16", "bf16", "f16", "f32"]),
                "y": rng.choice(["bf16", "f16", "f32"] + (["none"] if q != "none" else [])), "q": q, "pad": pad}
    act = rng.choice(["none", "none", "silu", "gelu", "gelu_tanh", "relu", "swiglu", "swiglu"])
    N = _spread(rng, 32, 4096 if act != "swiglu" else 2048)
    if rng.random() < 0.7:
        N = (N + 63) // 64 * 64
    K = 16 * _spread(rng, 4, 256)
    pad = 16 * rng.randint(0, 4)
    if rng.random() < 0.15:           # rows that start off a 16-byte boundary
        K += rng.randint(1, 15)
        pad = rng.randint(0, 9)
    return {"op": "product", "M": _spread(rng, 1, 6000), "N": N, "K": K, "act": act, "c": rng.choice(["bf16", "f16", "f32"]),
            "bias": rng.random() < 0.5, "residual": rng.choice(["none", "none", "f32", "bf16", "f16"]), "pad": pad}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _rows(gen, rows, cols, pad, dtype, std=1.0):
    """[rows, cols] of normal values, cols + pad apart."""
    return (torch.randn((rows, cols + pad), generator=gen, device="cuda") * std).to(TYPES[dtype])[:, :cols]


def _codes(gen, shape, dim):
    """int8 codes of normal values with a largest value of 127 along dim, as a quantiser writes them, and float32 scales."""
    v = torch.randn(shape, generator=gen, device="cuda")
    scale = v.abs().amax(dim, keepdim=True) / 127
    return torch.round(v / scale).to(torch.int8), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    st = {"case": c}
    if c["op"] == "norm":
        rows, H = c["rows"], c["H"]
        st["x"] = _rows(gen, rows, H, c["pad"], c["x"])
        # the residual stream has a few channels far larger than the rest
        st["residual"] = None
        if c["residual"] != "none":
            loud = 1 + 30 * (torch.rand((H + c["pad"],), generator=gen, device="cuda") < 0.002)
            r = torch.randn((rows, H + c["pad"]), generator=gen, device="cuda") * 2 * loud
            st["residual"] = r.to(TYPES[c["residual"]])[:, :H]
        st["weight"] = (1 + 0.2 * torch.randn((H,), generator=gen, device="cuda")).to(
            torch.float32 if c["x"] == "f32" else TYPES[c["x"]])
        if own:
            from moe_layer_03_amd import quantized as Q
            new = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")   # noqa: E731
            out = {"sum_out": new(rows, H, dtype=TYPES[c["residual"]]) if c["residual"] != "none" else None,
                   "y": new(rows, H, dtype=TYPES[c["y"]]) if c["y"] != "none" else None}
            if c["q"] == "int8":
                out |= {"codes": new(rows, H, dtype=torch.int8), "scales": new(rows, dtype=torch.float32),
                        "q_dtype": Q.MOE_I8}
            elif c["q"] == "mxfp8":
                out |= {"codes": new(rows, H, dtype=torch.uint8), "scales": new(rows, H // 32, dtype=torch.uint8),
                        "q_dtype": Q.MOE_MXFP8}
            st["out"] = out
    elif c["op"] == "quantise":
        st["x"] = _rows(gen, c["rows"], c["K"], c["pad"], c["x"])
        st["x"] *= torch.exp2(torch.randint(-6, 7, (c["rows"], 1), generator=gen, device="cuda")).to(st["x"].dtype)
        if own:
            st["codes"] = torch.empty((c["rows"], c["K"]), dtype=torch.int8, device="cuda")
            st["scales"] = torch.empty((c["rows"],), dtype=torch.float32, device="cuda")
    else:
        M, N, K = c["M"], c["N"], c["K"]
        a, sa = _codes(gen, (M, K + c["pad"]), 1)
        st["a"], st["sa"] = a[:, :K], sa[:, 0].contiguous()
        parts = 2 if c["act"] == "swiglu" else 1
        w = [_codes(gen, (K, N), 0) for _ in range(parts)]
        w = [(q, s[0] * 0.02) for q, s in w]          # weights of std 0.02, as in the package's workloads
        st["bias"] = torch.randn((parts, N), generator=gen, device="cuda") * 0.1 if c["bias"] else None
        st["residual"] = _rows(gen, M, N, c["pad"], c["residual"]) if c["residual"] != "none" else None
        if own:
            from moe_layer_03_amd import binding as B
            from moe_layer_03_amd import quantized as Q
            st["shape"] = B.DenseShape(M, N, K, gated=parts == 2)
            st["packed"] = Q.moe_pack_dense_int8(st["shape"], *(q for q, _ in w), scales=w[0][1],
                                                 up_scales=w[1][1] if parts == 2 else None)
            st["epilogue"] = {"none": B.MOE_EPI_NONE, "swiglu": B.MOE_EPI_SWIGLU, "silu": B.MOE_EPI_SILU,
                              "gelu": B.MOE_EPI_GELU, "gelu_tanh": B.MOE_EPI_GELU_TANH,
                              "relu": B.MOE_EPI_RELU}[c["act"]]
            st["c"] = torch.empty((M, N), dtype=TYPES[c["c"]], device="cuda")
        else:
            st["w"] = w
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _plain_int8(v):
    """Codes and scales of float32 rows; the quotient in double, since a code turns on which side of a half it lies."""
    scale = torch.clamp((v.abs().amax(1, keepdim=True).double() / 127).float(), min=SMALLEST)
    return torch.round(v.double() / scale.double()).to(torch.int8), scale[:, 0]


def _plain_mxfp8(v):
    """E4M3 codes and E8M0 scale bytes of float32 rows, 32 values to a scale."""
    b = v.view(v.shape[0], -1, 32)
    most = b.abs().amax(2)
    shared = torch.frexp(most).exponent - 9             # floor(log2) - 8
    shared = torch.where(most > 0, torch.clamp(shared, -127, 127), torch.full_like(shared, -127))
    inverse = ((127 - shared) << 23).view(torch.float32)     # 2^-shared; shared stays below 127 here
    q = (b * inverse[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(v.shape), (shared + 127).to(torch.uint8)


def _plain_norm(st):
    c, x = st["case"], st["x"]
    h = x if st["residual"] is None else (x.float() + st["residual"].float()).to(st["residual"].dtype)
    # the mean of the squares in double: a last digit of the row's factor moves codes that lie next to a half
    s = (1 / torch.sqrt((h.double() ** 2).mean(1, keepdim=True) + EPS)).float()
    v = h.float() * s * st["weight"].float()
    out = {"sum": None if st["residual"] is None else h, "y": v.to(TYPES[c["y"]]) if c["y"] != "none" else None}
    if c["q"] != "none":
        out["codes"], out["scales"] = _plain_int8(v) if c["q"] == "int8" else _plain_mxfp8(v)
    return out


def _activation(v, act):
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return torch.clamp(v, min=0) if act == "relu" else v


def _plain_product(st):
    c = st["case"]
    a, sa = st["a"].float(), st["sa"][:, None]
    v = [(a @ q.float()) * sa * s for q, s in st["w"]]
    if st["bias"] is not None:
        v = [p + b for p, b in zip(v, st["bias"])]
    v = _activation(v[0], "silu") * v[1] if c["act"] == "swiglu" else _activation(v[0], c["act"])
    if st["residual"] is not None:
        v = v + st["residual"].float()
    return v.to(TYPES[c["c"]])


def run(st):
    c = st["case"]
    if c["op"] == "norm":
        if not own:
            return _plain_norm(st)
        from moe_layer_03_amd import quantized as Q
        total, y, codes, scales = Q.moe_add_rmsnorm(st["x"], st["weight"], st["residual"], EPS, **st["out"])
        out = {"sum": total if st["residual"] is not None else None, "y": y}
        if c["q"] != "none":
            out["codes"], out["scales"] = codes.view(torch.float8_e4m3fn) if c["q"] == "mxfp8" else codes, scales
        return out
    if c["op"] == "quantise":
        if not own:
            codes, scales = _plain_int8(st["x"].float())
        else:
            from moe_layer_03_amd import quantized as Q
            codes, scales = Q.moe_quantize_int8(st["x"], codes=st["codes"], scales=st["scales"])
        return {"codes": codes, "scales": scales}
    if not own:
        return _plain_product(st)
    from moe_layer_03_amd import quantized as Q
    return Q.moe_dense_gemm_int8(st["shape"], st["a"], st["sa"], st["packed"], st["epilogue"], bias=st["bias"],
                                 residual=st["residual"], c=st["c"])


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["rows"] * c["H"]
        code = {"none": 0, "int8": 1, "mxfp8": 1 + 1 / 32}[c["q"]]
        return {"bytes": n * (SIZE[c["x"]] + 2 * SIZE[c["residual"]] + SIZE[c["y"]] + code)
                + c["H"] * SIZE[c["x"]] + (4 * c["rows"] if c["q"] == "int8" else 0), "flops": 6 * n}
    if c["op"] == "quantise":
        n = c["rows"] * c["K"]
        return {"bytes": n * (SIZE[c["x"]] + 1) + 4 * c["rows"], "flops": 3 * n}
    parts = 2 if c["act"] == "swiglu" else 1
    return {"bytes": c["M"] * (c["K"] + 4) + parts * (c["K"] + 4) * c["N"] + (4 * parts * c["N"] if c["bias"] else 0)
            + c["M"] * c["N"] * (SIZE[c["c"]] + SIZE[c["residual"]]),
            "flops": 2 * parts * c["M"] * c["N"] * c["K"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_norm(st):
    c = st["case"]
    total = st["x"].double()
    h = total
    if st["residual"] is not None:
        total = total + st["residual"].double()
        # what is normed is the sum that is written: float32's, in the residual's type
        h = total.float().to(st["residual"].dtype).double()
    v = h * torch.rsqrt(h.pow(2).sum(1) / c["H"] + EPS)[:, None] * st["weight"].double()
    out = {"sum": None if st["residual"] is None else total, "y": v if c["y"] != "none" else None}
    if c["q"] != "none":
        out["codes"] = None
        out["scales"] = v.abs().max(1).values / 127 if c["q"] == "int8" else None
    return out


def _exact_product(st):
    c, a = st["case"], st["a"].double()
    v = torch.stack([torch.mm(a, q.double()) * torch.outer(st["sa"].double(), s.double()) for q, s in st["w"]])
    if st["bias"] is not None:
        v += st["bias"].double()[:, None]
    if c["act"] == "swiglu":
        v = v[0] * torch.sigmoid(v[0]) * v[1]
    elif c["act"] == "silu":
        v = v[0] * torch.sigmoid(v[0])
    elif c["act"] == "gelu":
        v = v[0] * (1 - 0.5 * torch.erfc(v[0] / math.sqrt(2)))
    elif c["act"] == "gelu_tanh":      # (1 + tanh z) / 2 = sigmoid(2 z)
        v = v[0] * torch.sigmoid(math.sqrt(8 / math.pi) * (v[0] + 0.044715 * v[0] ** 3))
    elif c["act"] == "relu":
        v = torch.where(v[0] > 0, v[0], torch.zeros_like(v[0]))
    else:
        v = v[0]
    return v if st["residual"] is None else v + st["residual"].double()


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "norm":
        return _exact_norm(st)
    if case["op"] == "quantise":
        return {"codes": None, "scales": st["x"].double().abs().max(1).values / 127}
    return _exact_product(st)
