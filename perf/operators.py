"""The few-token MoE layer and the dense product with a fused epilogue: cases, inputs, plain forms and exact values.

``listed()`` and ``draw(rng)`` give the cases, ``prepare`` their inputs, ``run`` one pass (the plain form in elementary
torch operations, or the library's call where ``own`` is true), ``work`` the bytes and operations a pass cannot do
without, ``exact`` the outputs from the definition in 64 bits.

Layer cases ("layer"): T tokens through E experts, the K best of each token, experts [e_begin, e_end) held here, hidden
size H, expert size I.  Weights of a "f32" layer are values that fp16 holds, since that is what such a layer packs.
Weights of an "mxfp8" layer are E4M3 codes with a power-of-two scale per 32 along the reduction.

Dense cases ("dense"): C = act(A W + bias) + residual with A [M, K] and W [K, N]; "swiglu" has a gate and an up weight.
``pad`` is the extra length of A's and the residual's rows in memory.
"""
import math

import torch

own = False

STD_W = 0.02                      # weights, as in the package's workloads (inputs have std 1)
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _layer(name, T, e_begin, e_end, dtype="bf16", H=4096, E=128, K=8, I=1536, bias=False):
    return {"name": name, "op": "layer", "T": T, "H": H, "E": E, "K": K, "I": I, "e_begin": e_begin, "e_end": e_end,
            "dtype": dtype, "bias": bias}


def _dense(name, M, N, K, act="none", a="bf16", c="bf16", bias=False, residual="none", pad=0):
    return {"name": name, "op": "dense", "M": M, "N": N, "K": K, "act": act, "a": a, "c": c, "bias": bias,
            "residual": residual, "pad": pad}


def listed():
    return [
        # the tiny workload's layer with a handful of tokens: launch latency is all there is
        _layer("layer tiny 5 tokens f32", 5, 0, 8, dtype="f32", H=256, E=8, K=2, I=128),
        # one sequence being decoded, every expert on this GPU
        _layer("layer 1 token whole", 1, 0, 128),
        # eight sequences on one rank of a 16-way expert split: half of them find none of their experts here
        _layer("layer 8 tokens ep16", 8, 0, 8, bias=True),
        # a small decode batch on one rank of a 4-way split
        _layer("layer 16 tokens ep4", 16, 32, 64),
        # the largest batch the few-token layer takes, every expert on this GPU
        _layer("layer 32 tokens whole", 32, 0, 128),
        # the deployed weight format, one sequence and a batch of them
        _layer("mxfp8 1 token whole", 1, 0, 128, dtype="mxfp8"),
        _layer("mxfp8 13 tokens ep16", 13, 16, 24, dtype="mxfp8"),
        # a shared expert's gate and up projection for one token
        _dense("dense 1 row swiglu", 1, 1536, 4096, act="swiglu"),
        # a shared expert's down projection, added onto the routed experts' float32 sum
        _dense("dense 16 rows add f32", 16, 4096, 1536, c="f32", residual="f32"),
        # a decode batch through an output projection with bias and residual
        _dense("dense 128 rows residual", 128, 4096, 4096, bias=True, residual="bf16"),
        # an odd size all round: a classifier-like head over a ragged batch
        _dense("dense odd f16 gelu", 1000, 1003, 1096, act="gelu", a="f16", c="f16", bias=True, pad=8),
        # the prefill batch through a dense MLP's first projection
        _dense("dense 6000 rows silu", 6000, 4096, 4096, act="silu", bias=True),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    """One more case of the ranges that the listed ones stand for."""
    if rng.random() < 0.5:
        dtype = rng.choice(["bf16", "bf16", "bf16", "mxfp8", "mxfp8", "f32"])
        unit = 256 if dtype == "mxfp8" else 64
        H = unit * _spread(rng, 1, (1024 if dtype == "f32" else 4096) // unit)
        I = unit * _spread(rng, 1, (512 if dtype == "f32" else 1536) // unit)
        E = rng.randint(4, 200)
        K = rng.randint(1, min(8, E))
        n = rng.randint(1, min(E, 128))
        e_begin = rng.randint(0, E - n)
        return {"op": "layer", "T": _spread(rng, 1, 32), "H": H, "E": E, "K": K, "I": I, "e_begin": e_begin,
                "e_end": e_begin + n, "dtype": dtype, "bias": rng.random() < 0.3}
    act = rng.choice(["none", "none", "silu", "gelu", "gelu_tanh", "relu", "swiglu", "swiglu"])
    N = _spread(rng, 32, 4096 if act != "swiglu" else 2048)
    if rng.random() < 0.7:
        N = (N + 63) // 64 * 64
    K = 8 * _spread(rng, 8, 512)
    pad = 8 * rng.randint(0, 4)
    if rng.random() < 0.15:       # rows that start off a 16-byte boundary
        K += rng.randint(1, 7)
        pad = rng.randint(0, 5)
    return {"op": "dense", "M": _spread(rng, 1, 6000), "N": N, "K": K, "act": act, "a": rng.choice(["bf16", "bf16", "f16"]),
            "c": rng.choice(["bf16", "f16", "f32"]), "bias": rng.random() < 0.5,
            "residual": rng.choice(["none", "none", "f32", "bf16", "f16"]), "pad": pad}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _experts(gen, n, rows, cols, dtype):
    """[n, rows, cols] weights, an expert at a time."""
    w = torch.empty((n, rows, cols), dtype=TYPES[dtype], device="cuda")
    for e in range(n):
        w[e] = _normal(gen, (rows, cols), STD_W, torch.float16 if dtype == "f32" else TYPES[dtype])
    return w


def _experts_mxfp8(gen, n, rows, cols):
    """(codes [n, rows, cols], scales [n, rows/32, cols]), both bytes: the value is E4M3(code) * 2^(scale - 127)."""
    codes = torch.empty((n, rows, cols), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n, rows // 32, cols), dtype=torch.uint8, device="cuda")
    for e in range(n):
        v = torch.randn((rows // 32, 32, cols), generator=gen, device="cuda") * STD_W
        shared = torch.floor(torch.log2(v.abs().amax(1))) - 8
        q = (v * torch.exp2(-shared)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        codes[e] = q.view(torch.uint8).view(rows, cols)
        scales[e] = (shared + 127).to(torch.uint8)
    return codes, scales


def _dequantised(codes, scales, dtype):
    """The values that MXFP8 codes [n, rows, cols] with their scales stand for."""
    n, rows, cols = codes.shape
    v = codes.view(torch.float8_e4m3fn).to(dtype).view(n, rows // 32, 32, cols)
    return (v * torch.exp2(scales.to(dtype) - 127)[:, :, None]).view(n, rows, cols)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    if c["op"] == "layer":
        mx = c["dtype"] == "mxfp8"
        t = TYPES["bf16" if mx else c["dtype"]]
        n = c["e_end"] - c["e_begin"]
        st = {"case": c, "x": _normal(gen, (c["T"], c["H"]), 1.0, t),
              "w_router": _normal(gen, (c["H"], c["E"]), STD_W, t),
              "bias": _normal(gen, (c["E"],), 0.5, torch.float32) if c["bias"] else None}
        sizes = {"gate": (c["H"], c["I"]), "up": (c["H"], c["I"]), "down": (c["I"], c["H"])}
        w = {k: _experts_mxfp8(gen, n, *v) if mx else _experts(gen, n, *v, c["dtype"]) for k, v in sizes.items()}
        if own:
            from moe_layer_03_amd import binding as B
            s = B.Shape(c["T"], c["H"], c["E"], c["K"], c["I"], c["e_begin"], c["e_end"])
            if mx:
                w = [_dequantised(*w[k], torch.float32).to(torch.bfloat16) for k in ("gate", "up", "down")]
                st["packed"] = B.moe_pack_weights_mxfp8(s, *w)
                need = B.moe_layer_few_tokens_workspace_bytes_mxfp8(s)
            else:
                st["packed"] = B.moe_pack_weights(s, w["gate"], w["up"], w["down"])
                need = B.moe_layer_few_tokens_workspace_bytes(s)
            st["shape"] = s
            st["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
            st["out"] = torch.empty((s.T, s.H), dtype=torch.float32, device="cuda")
            st["topk_idx"] = torch.empty((s.T, s.K), dtype=torch.int32, device="cuda")
            st["topk_w"] = torch.empty((s.T, s.K), dtype=torch.float32, device="cuda")
        else:
            st["w"] = w
        return st
    t = TYPES[c["a"]]
    st = {"case": c, "a": _normal(gen, (c["M"], c["K"] + c["pad"]), 1.0, t)[:, : c["K"]],
          "bias": _normal(gen, (2 if c["act"] == "swiglu" else 1, c["N"]), 0.1, torch.float32) if c["bias"] else None,
          "residual": None}
    if c["residual"] != "none":
        st["residual"] = _normal(gen, (c["M"], c["N"] + c["pad"]), 1.0, TYPES[c["residual"]])[:, : c["N"]]
    w = [_normal(gen, (c["K"], c["N"]), STD_W, t) for _ in range(2 if c["act"] == "swiglu" else 1)]
    if own:
        from moe_layer_03_amd import binding as B
        st["shape"] = B.DenseShape(c["M"], c["N"], c["K"], gated=c["act"] == "swiglu")
        st["packed"] = B.moe_pack_dense(st["shape"], *w)
        st["epilogue"] = {"none": B.MOE_EPI_NONE, "swiglu": B.MOE_EPI_SWIGLU, "silu": B.MOE_EPI_SILU,
                          "gelu": B.MOE_EPI_GELU, "gelu_tanh": B.MOE_EPI_GELU_TANH, "relu": B.MOE_EPI_RELU}[c["act"]]
        st["c"] = torch.empty((c["M"], c["N"]), dtype=TYPES[c["c"]], device="cuda")
    else:
        st["w"] = w
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _silu(v):
    return v / (1 + torch.exp(-v))


def _activation(v, act):
    if act == "silu":
        return _silu(v)
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return torch.clamp(v, min=0) if act == "relu" else v


def _plain_layer(st):
    c, x = st["case"], st["x"]
    logits = x.double() @ st["w_router"].double()
    if st["bias"] is not None:
        logits = logits + st["bias"].double()
    value, index = torch.sort(logits, dim=1, descending=True, stable=True)
    value, index = value[:, : c["K"]], index[:, : c["K"]]
    weight = torch.exp(value - value[:, :1])
    weight = (weight / weight.sum(1, keepdim=True)).float()
    n, pairs = c["e_end"] - c["e_begin"], c["T"] * c["K"]
    here = (index >= c["e_begin"]) & (index < c["e_end"])
    expert = (index - c["e_begin"]).clamp(0, n - 1)
    share = torch.where(here, weight, torch.zeros_like(weight))
    if n <= pairs:                # every expert held here on every token, each weight read once
        pick = slice(None)
        rows = x.float().expand(n, -1, -1)
        share = torch.zeros((c["T"], n), device=x.device).scatter_add_(1, expert, share).t()
    else:                         # the weights of every (token, slot) pair
        pick = expert.reshape(-1)
        rows = x.float().repeat_interleave(c["K"], 0)[:, None]

    def chosen(w):
        if c["dtype"] == "mxfp8":
            return _dequantised(w[0][pick], w[1][pick], torch.float32)
        return w[pick].float()

    h = _silu(torch.bmm(rows, chosen(st["w"]["gate"]))) * torch.bmm(rows, chosen(st["w"]["up"]))
    y = torch.bmm(h, chosen(st["w"]["down"]))
    out = (share[..., None] * y).sum(0) if n <= pairs else (share[..., None] * y.view(c["T"], c["K"], c["H"])).sum(1)
    return {"out": out, "topk_idx": index.int(), "topk_w": weight}


def _plain_dense(st):
    c = st["case"]
    a = st["a"].float()
    v = [a @ w.float() for w in st["w"]]
    if st["bias"] is not None:
        v = [p + b for p, b in zip(v, st["bias"])]
    v = _silu(v[0]) * v[1] if c["act"] == "swiglu" else _activation(v[0], c["act"])
    if st["residual"] is not None:
        v = v + st["residual"].float()
    return v.to(TYPES[c["c"]])


def run(st):
    c = st["case"]
    if not own:
        return _plain_layer(st) if c["op"] == "layer" else _plain_dense(st)
    from moe_layer_03_amd import binding as B
    if c["op"] == "dense":
        return B.moe_dense_gemm(st["shape"], st["a"], st["packed"], st["epilogue"], bias=st["bias"],
                                residual=st["residual"], c=st["c"])
    call = B.moe_layer_few_tokens_mxfp8 if c["dtype"] == "mxfp8" else B.moe_layer_few_tokens
    out = call(st["shape"], st["x"], st["w_router"], st["packed"], st["bias"], out=st["out"], ws=st["ws"],
               topk_idx=st["topk_idx"], topk_w=st["topk_w"])
    return {"out": out, "topk_idx": st["topk_idx"], "topk_w": st["topk_w"]}


def work(case):
    c = case
    if c["op"] == "layer":
        n = c["e_end"] - c["e_begin"]
        size = 4 if c["dtype"] == "f32" else 2
        # experts held here that at least one token chooses, in expectation
        active = n * (1 - (1 - c["K"] / c["E"]) ** c["T"])
        weight = {"bf16": 2, "f32": 2, "mxfp8": 1 + 1 / 32}[c["dtype"]]
        return {"bytes": c["T"] * c["H"] * (size + 4) + c["H"] * c["E"] * size + active * 3 * c["H"] * c["I"] * weight
                + c["T"] * c["K"] * 8,
                "flops": 2 * c["T"] * c["E"] * c["H"] + 6 * c["H"] * c["I"] * c["T"] * c["K"] * n / c["E"]}
    parts = 2 if c["act"] == "swiglu" else 1
    size = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}
    return {"bytes": 2 * c["M"] * c["K"] + 2 * parts * c["K"] * c["N"] + (4 * parts * c["N"] if c["bias"] else 0)
            + c["M"] * c["N"] * (size[c["c"]] + size[c["residual"]]),
            "flops": 2 * parts * c["M"] * c["N"] * c["K"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_layer(st):
    c, x = st["case"], st["x"].double()
    T, K, n = c["T"], c["K"], c["e_end"] - c["e_begin"]
    logits = (x[:, :, None] * st["w_router"].double()).sum(1)
    if st["bias"] is not None:
        logits += st["bias"]
    order = logits.cpu().tolist()
    index = [sorted(range(c["E"]), key=lambda e: (-row[e], e))[:K] for row in order]
    weight = [[math.exp(row[e] - row[pick[0]]) for e in pick] for row, pick in zip(order, index)]
    weight = [[v / math.fsum(row) for v in row] for row in weight]
    out = torch.zeros((T, c["H"]), dtype=torch.float64, device="cuda")
    for e in sorted({e - c["e_begin"] for pick in index for e in pick if 0 <= e - c["e_begin"] < n}):
        if c["dtype"] == "mxfp8":
            g, u, d = (_dequantised(*(p[e: e + 1] for p in st["w"][k]), torch.float64)[0] for k in ("gate", "up", "down"))
        else:
            g, u, d = (st["w"][k][e].double() for k in ("gate", "up", "down"))
        for t in range(T):
            if e + c["e_begin"] in index[t]:
                a = x[t] @ g
                y = (a * torch.sigmoid(a) * (x[t] @ u)) @ d
                out[t] += weight[t][index[t].index(e + c["e_begin"])] * y
    return {"out": out, "topk_idx": None, "topk_w": torch.tensor(weight, dtype=torch.float64)}


def _exact_dense(st):
    c, a = st["case"], st["a"].double()
    v = torch.stack([torch.mm(a, w.double()) for w in st["w"]])
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
    return _exact_layer(st) if case["op"] == "layer" else _exact_dense(st)
