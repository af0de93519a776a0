"""The operators of a decoder layer's feed-forward half in 8 bits, as measured cases: the residual's addition with
the RMS norm (and its quantization to e4m3), the product of e4m3 activations with e4m3 weights that carry one scale
for each block of 128, and the gated pair of such products with its activation.

`run` computes each operator in its plain form (elementary torch operations in 32 bits) or, where
`own` is true, through this repository's library.  `exact` is the operators' definition in 64 bits.

Activations in 8 bits are codes [tokens, K] in e4m3 and scales [K / 128, tokens] in 32 bits, value = code * scale, with
  scale = max(largest |x| of the token's block of 128, 2^-100) / 448,  code = e4m3(x / scale).
Weights are codes [rows, K] and scales [row blocks of 128, K / 128]; a gated pair holds the gate's rows, then the
other's, each with row blocks of its own.
"""
import math

import torch

own = False

F32, F64, E4M3 = torch.float32, torch.float64, torch.float8_e4m3fn
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BLOCK, EPS = 128, 1e-6


# ----------------------------------------------------------------------------- cases
def _norm(name, tokens, dim, dtype, out, residual=True):
    return dict(name=name, op="norm", tokens=tokens, dim=dim, dtype=dtype, out=out, residual=residual)


def _product(name, m, n, k, out, gate="none"):
    return dict(name=name, op="product", m=m, n=n, k=k, out=out, gate=gate)


def listed():
    return [
        # between two products of one decode step, 16 requests at width 4096: latency
        _norm("norm_step", 16, 4096, "f16", "e4m3"),
        # before a 16-bit product with 4-bit weights: the output stays in 16 bits, an odd number of tokens
        _norm("norm_wide", 2047, 4096, "f16", "f16"),
        # a whole prompt at width 5120, to 8 bits
        _norm("norm_prompt", 8192, 5120, "bf16", "e4m3"),
        # one token through a square projection: the weights' bytes
        _product("product_one", 1, 4096, 4096, "f16"),
        # a decode step of 16 requests, the projection back from the feed-forward width
        _product("product_step", 16, 4096, 11008, "bf16"),
        # a ragged batch between decode and prompt: neither the weights' bytes nor the products alone
        _product("product_batch", 200, 10240, 5120, "f16"),
        # a prompt of odd length, an output width that is no multiple of a tile, in 32 bits
        _product("product_odd", 4001, 3200, 5120, "f32"),
        # a whole prompt
        _product("product_prompt", 8192, 10240, 5120, "bf16"),
        # one token through both projections to the feed-forward width, output ready for the projection back
        _product("gated_one", 1, 11008, 4096, "e4m3", "silu"),
        # drafted tokens of a small batch
        _product("gated_step", 40, 11008, 4096, "e4m3", "silu"),
        # a ragged batch with the other activation, in 16 bits
        _product("gated_batch", 333, 11008, 4096, "bf16", "gelu"),
        # a whole prompt: the largest
        _product("gated_prompt", 8192, 11008, 4096, "e4m3", "silu"),
    ]


def _log(rng, low, high, step=1):
    """A multiple of `step` spread over the logarithm of [low, high]."""
    x = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(x / step)) * step))


def draw(rng):
    if rng.random() < 0.3:
        out = rng.choice(("e4m3", "e4m3", "16"))
        dtype = rng.choice(("f16", "bf16"))
        return dict(op="norm", tokens=_log(rng, 1, 8192), dim=_log(rng, 128, 8192, 128 if out == "e4m3" else 8), dtype=dtype,
                    out=dtype if out == "16" else out, residual=rng.random() < 0.8)
    gate = rng.choice(("none", "none", "silu", "gelu"))
    out = rng.choice(("f16", "bf16", "f32") if gate == "none" else ("e4m3", "e4m3", "f16", "bf16"))
    n, k = _log(rng, 256, 11008, 128 if out == "e4m3" else 16), _log(rng, 128, 11008, 128)
    most = (1 << 40) // (2 * n * k * (1 if gate == "none" else 2))
    return dict(op="product", m=_log(rng, 1, max(1, min(8192, most))), n=n, k=k, out=out, gate=gate)


# ----------------------------------------------------------------------------- inputs
def _quantise(x):
    """x [tokens, K] in 32 bits -> (codes e4m3 [tokens, K], scales [K / 128, tokens])."""
    y = x.unflatten(-1, (-1, BLOCK))
    scale = y.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100) / 448
    return (y / scale).clamp(-448, 448).to(E4M3).flatten(-2), scale[..., 0].t().contiguous()


def _activations(tokens, dim, gen):
    """A trained model's kind: each dim with its own spread, a few dims far out, tokens of different size."""
    spread = torch.rand(dim, generator=gen, device="cuda") + 0.5
    spread = spread * (1 + 9 * (torch.rand(dim, generator=gen, device="cuda") < 0.01))
    size = torch.exp(0.5 * torch.randn((tokens, 1), generator=gen, device="cuda"))
    return torch.randn((tokens, dim), generator=gen, device="cuda") * spread * size


def _weights(rows, k, gen):
    """rows x k weights in e4m3 with a scale for each block of 128 x 128 (the last row block may be shorter)."""
    blocks = -(-rows // BLOCK)
    w = torch.randn((blocks * BLOCK, k), generator=gen, device="cuda")
    w[rows:] = 0
    w = w.view(blocks, BLOCK, k // BLOCK, BLOCK)
    size = 0.02 * torch.exp(0.3 * torch.randn((blocks, 1, k // BLOCK, 1), generator=gen, device="cuda"))
    largest = w.abs().amax((1, 3), keepdim=True)
    codes = (w * (448 / largest)).clamp(-448, 448).to(E4M3).reshape(blocks * BLOCK, k)[:rows]
    return codes, (largest * size / 448)[:, 0, :, 0]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "norm":
        t, d, t16 = case["tokens"], case["dim"], TYPES[case["dtype"]]
        state = dict(x=_activations(t, d, gen).to(t16), residual=(4 * _activations(t, d, gen)).to(t16) if case["residual"] else None,
                     weight=(1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(t16))
    else:
        m, n, k = case["m"], case["n"], case["k"]
        codes, scales = _quantise(_activations(m, k, gen))
        parts = [_weights(n, k, gen) for _ in range(1 if case["gate"] == "none" else 2)]
        state = dict(a=codes, a_scales=scales, w=torch.cat([p[0].view(torch.uint8) for p in parts]).view(E4M3),
                     w_scales=torch.cat([p[1] for p in parts]).contiguous())
    state["case"] = dict(case)
    if own:
        _keep(state)
    return state


# ----------------------------------------------------------------------------- the library's calls
def _keep(state):
    """What a program of the library keeps between calls: descriptors, output buffers, the workspace."""
    import weight_only_quantized_qgemm_amd as q
    case = state["case"]
    kinds = {"f16": q.DT_F16, "bf16": q.DT_BF16, "f32": q.DT_F32, "e4m3": q.DT_FP8_E4M3}
    state["lib"] = q
    if case["op"] == "norm":
        t, d = case["tokens"], case["dim"]
        state["p"] = q.add_norm_problem(t, d, kinds[case["dtype"]], kinds[case["out"]], eps=EPS)
        state["sum"] = torch.empty_like(state["x"]) if case["residual"] else None
    else:
        t, d = case["m"], case["n"]
        gate = {"none": q.GATE_NONE, "silu": q.GATE_SILU, "gelu": q.GATE_GELU_TANH}[case["gate"]]
        state["p"] = q.w8a8_problem(t, d, case["k"], kinds[case["out"]], gate=gate)
        state["ws"] = q.alloc_w8a8_workspace(state["p"])
    state["y"] = torch.empty((t, d), dtype=TYPES[case["out"]], device="cuda")
    state["y_scales"] = torch.empty((d // BLOCK, t), dtype=F32, device="cuda") if case["out"] == "e4m3" else None


def _run_own(state):
    q, case = state["lib"], state["case"]
    if case["op"] == "norm":
        q.add_norm(state["p"], state["x"], state["residual"], state["weight"], state["sum"], state["y"], state["y_scales"])
        return {"sum": state["sum"], "y": state["y"], "scales": state["y_scales"]}
    q.w8a8_run(state["p"], state["a"], state["a_scales"], state["w"], state["w_scales"], state["y"], state["y_scales"], state["ws"])
    return {"y": state["y"], "scales": state["y_scales"]}


# ----------------------------------------------------------------------------- the plain forms
def _plain_norm(state):
    case = state["case"]
    h = state["x"].to(F32)
    if case["residual"]:
        h = h + state["residual"].to(F32)
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * state["weight"].to(F32)
    y, scales = _quantise(y) if case["out"] == "e4m3" else (y.to(TYPES[case["out"]]), None)
    return {"sum": h.to(state["x"].dtype) if case["residual"] else None, "y": y, "scales": scales}


def _plain_product(state):
    case, n = state["case"], state["case"]["n"]
    a = (state["a"].to(F32).unflatten(-1, (-1, BLOCK)) * state["a_scales"].t()[..., None]).flatten(-2)
    s = state["w_scales"].repeat_interleave(BLOCK, 0).view(1 if case["gate"] == "none" else 2, -1, case["k"] // BLOCK)[:, :n]
    w = (state["w"].to(F32).unflatten(-1, (-1, BLOCK)) * s.reshape(-1, case["k"] // BLOCK, 1)).flatten(-2)
    y = torch.matmul(a, w.t())
    if case["gate"] != "none":
        g, u = y[:, :n], y[:, n:]
        if case["gate"] == "silu":
            g = g / (1 + torch.exp(-g))
        else:
            g = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
        y = g * u
    y, scales = _quantise(y) if case["out"] == "e4m3" else (y.to(TYPES[case["out"]]), None)
    return {"y": y, "scales": scales}


def run(state):
    if own:
        return _run_own(state)
    return _plain_norm(state) if state["case"]["op"] == "norm" else _plain_product(state)


# ----------------------------------------------------------------------------- cost
def work(case):
    out = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1 + 4 / BLOCK}[case["out"]]
    if case["op"] == "norm":
        n = case["tokens"] * case["dim"]
        return {"bytes": n * ((6 if case["residual"] else 2) + out) + 2 * case["dim"], "flops": 8 * n}
    m, n, k = case["m"], case["n"], case["k"]
    rows = n if case["gate"] == "none" else 2 * n
    return {"bytes": (m * (1 + 4 / BLOCK) + rows * (1 + 4 / BLOCK ** 2)) * k + m * n * out, "flops": 2 * m * rows * k}


# ----------------------------------------------------------------------------- the definition in 64 bits
def _codes64(y):
    """y [tokens, dim] in 64 bits -> the values of its e4m3 codes and their scales."""
    scale = torch.stack([b.abs().max(1).values for b in y.split(BLOCK, 1)]).clamp(min=2.0 ** -100) / 448
    t = y / scale.t().repeat_interleave(BLOCK, 1)
    power = torch.frexp(t.abs())[1].clamp(min=-5).to(F64) - 4              # 3 bits after the leading one, none below 2^-9
    step = torch.exp2(power)
    return torch.round(t / step) * step, scale


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "norm":
        h = state["x"].double() + (state["residual"].double() if case["residual"] else 0)
        length = torch.sqrt(h.square().sum(1) / case["dim"] + EPS)
        y = torch.einsum("td,d,t->td", h, state["weight"].double(), 1 / length)
        y, scales = _codes64(y) if case["out"] == "e4m3" else (y, None)
        return {"sum": h if case["residual"] else None, "y": y, "scales": scales}
    m, n, k = case["m"], case["n"], case["k"]
    sides = []
    for part in range(1 if case["gate"] == "none" else 2):
        w = state["w"][part * n:(part + 1) * n].double()
        scales = state["w_scales"].double()[part * -(-n // BLOCK):(part + 1) * -(-n // BLOCK)]
        y = torch.zeros((m, n), dtype=F64, device="cuda")
        for b in range(k // BLOCK):
            at = slice(b * BLOCK, (b + 1) * BLOCK)
            y += (state["a"][:, at].double() @ w[:, at].t()) * state["a_scales"][b].double()[:, None] * scales[
                :, b].repeat_interleave(BLOCK)[:n]
        sides.append(y)
    y = sides[0]
    if case["gate"] == "silu":
        y = y * torch.sigmoid(y) * sides[1]
    elif case["gate"] == "gelu":
        y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)) * sides[1]
    y, scales = _codes64(y) if case["out"] == "e4m3" else (y, None)
    return {"y": y, "scales": scales}
