"""The attention operators next to the weight-only GEMMs, as measured cases: the norm and rotation
of query and key heads, the 4-bit paged cache (written and read back) and attention over it.

`run` computes each operator in its plain form (elementary torch operations in 32 bits) or, where
`own` is true, through this repository's library.  `exact` is the operators' definition in 64 bits.

Cache layout, per page and kv head one block of bytes [K codes | V codes | K params | V params] with
D = head_dim, P = page_size, NG = D / group_size, u = D / 32:
  K codes  row t of D/2 bytes; dword u*g + i (g < 4, i < u) holds dims 8 (4 i + g) .. + 7, low nibble first
  V codes  byte ((t / 4) * 16 + r) * 4 u + (t % 4) * u + i / 2, nibble i % 2: dim 16 i + r (r < 16)
  params   [NG][P][2] 16-bit values (scale, zero) of token t and group: value = code * scale + zero
"""
import math

import torch

own = False

F32, F64 = torch.float32, torch.float64
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ----------------------------------------------------------------------------- cases
def _rope(name, dtype, tokens, q_heads, kv_heads, dim, rot, interleaved):
    return dict(name=name, op="rope", dtype=dtype, tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, dim=dim, rot=rot,
                interleaved=interleaved)


def _cache(name, dtype, tokens, kv_heads, dim, group, page, scattered):
    return dict(name=name, op="cache", dtype=dtype, tokens=tokens, kv_heads=kv_heads, dim=dim, group=group, page=page,
                scattered=scattered)


def _attn(name, dtype, batch, q_heads, kv_heads, dim, group, page, q_low, q_high, past_low, past_high, causal=True, window=0):
    return dict(name=name, op="attention", dtype=dtype, batch=batch, q_heads=q_heads, kv_heads=kv_heads, dim=dim, group=group,
                page=page, q_low=q_low, q_high=q_high, past_low=past_low, past_high=past_high, causal=causal, window=window)


def listed():
    return [
        # the heads of one decode step of a 16-request batch at model width 4096: latency
        _rope("rope_step", "f16", 16, 32, 8, 128, 128, False),
        # the heads of one 8192-token prompt pass at width 5120; only half of each head is rotated, in adjacent pairs
        _rope("rope_prompt", "bf16", 8192, 40, 8, 128, 64, True),
        # one decode step of 64 requests: a token each, anywhere in the cache
        _cache("cache_step", "bf16", 64, 8, 128, 128, 64, True),
        # a prompt of odd length entering the cache page by page, in the finest groups
        _cache("cache_prompt", "f16", 16383, 8, 128, 32, 16, False),
        # one request, one token, a short context: the smallest call, latency
        _attn("decode_one", "f16", 1, 32, 8, 128, 128, 16, 1, 1, 776, 776),
        # a serving batch: 64 requests of very different context, a token each, at width 8192
        _attn("decode_batch", "bf16", 64, 64, 8, 128, 128, 64, 1, 1, 0, 8191),
        # few requests over a very long cache, five query heads to a kv head (width 5120)
        _attn("decode_long", "f16", 4, 40, 8, 128, 64, 256, 1, 1, 100001, 131071),
        # drafted tokens checked at once (1 to 5 a request), one kv head for every query head, heads of 64
        _attn("draft_check", "bf16", 12, 32, 32, 64, 64, 48, 1, 5, 500, 4095),
        # pieces of prompts with earlier context in the cache, sliding window, requests without new tokens among them
        _attn("chunk_window", "bf16", 6, 64, 8, 128, 32, 32, 0, 700, 0, 6000, True, 4096),
        # one whole prompt at width 4096, causal: the largest
        _attn("prompt", "f16", 1, 32, 8, 128, 128, 64, 8192, 8192, 0, 0),
    ]


def _log(rng, low, high):
    """A whole number spread over the logarithm of [low, high]."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _heads(rng, dim):
    while True:
        kv, ratio = rng.choice((1, 2, 3, 4, 8, 16)), rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 16))
        if kv * ratio * dim <= 8192 and kv * ratio * dim != 3072 and kv * dim != 3072:
            return kv * ratio, kv


def _not_3072(n):
    return n + 1 if n == 3072 else n


def draw(rng):
    dtype, dim = rng.choice(("f16", "bf16")), rng.choice((64, 128, 128, 256))
    q_heads, kv_heads = _heads(rng, dim)
    group, page = dim // rng.choice((1, 2, 4) if dim > 64 else (1, 2)), rng.choice((16, 32, 48, 64, 128, 256))
    kind = rng.choice(("rope", "cache", "decode", "decode", "draft", "chunk", "prompt"))
    if kind == "rope":
        return dict(op="rope", dtype=dtype, tokens=_not_3072(_log(rng, 1, 8192)), q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice((dim, dim // 2, dim // 4)), interleaved=rng.random() < 0.4)
    if kind == "cache":
        return dict(op="cache", dtype=dtype, tokens=_not_3072(_log(rng, 1, 16384)), kv_heads=min(kv_heads, 8), dim=dim, group=group,
                    page=page, scattered=rng.random() < 0.5)
    case = dict(op="attention", dtype=dtype, q_heads=q_heads, kv_heads=kv_heads, dim=dim, group=group, page=page,
                causal=True, window=0)
    if kind in ("decode", "draft"):
        batch, q_high = _log(rng, 1, 128), 1 if kind == "decode" else rng.randint(2, 8)
        room = max(2, min(131072, 1 << 28 >> max(0, (batch * kv_heads * dim - 1).bit_length())))
        past = _not_3072(_log(rng, 1, room))
        return dict(case, batch=batch, q_low=1, q_high=q_high, past_low=rng.choice((0, past // 2, past)), past_high=past,
                    window=rng.choice((0, 0, 0, 1000)))
    batch = 1 if kind == "prompt" else rng.randint(1, 8)
    most = max(64, min(8192, int(math.sqrt((1 << 31) / (batch * q_heads) * min(1, 128 / dim)))))
    q_high = _not_3072(_log(rng, 16, most // (1 if kind == "prompt" else 2)))
    past = 0 if kind == "prompt" else rng.randint(0, max(1, min(16384, (1 << 37) // (batch * q_heads * q_high * max(dim, 128)))))
    return dict(case, batch=batch, q_low=q_high if kind == "prompt" else q_high // 3, q_high=q_high, past_low=past // 4, past_high=past,
                causal=kind == "prompt" or rng.random() < 0.8, window=rng.choice((0, 0, 512)) if kind == "prompt" else 0)


def _lengths(case):
    """Query and context lengths of each request: spread over the case's ranges, both ends among them."""
    b, qs, ks = case["batch"], [], []
    for i in range(b):
        x = (i * 0.6180339887 + 0.5) % 1.0 if i > 1 else float(1 - i)        # the longest first, then the shortest
        y = (i * 0.7548776662 + 0.5) % 1.0 if i > 1 else float(1 - i)
        n = case["q_low"] + int(round(y * (case["q_high"] - case["q_low"])))
        qs.append(n)
        ks.append(_not_3072(n + case["past_low"] + int(round(x * (case["past_high"] - case["past_low"])))))
    return qs, ks


# ----------------------------------------------------------------------------- inputs
def _block_bytes(case):
    return case["page"] * (case["dim"] + 8 * (case["dim"] // case["group"]))


def _quantise(x, group):
    """x [..., D] in 16 bits -> (codes uint8 [..., D], scale and zero 16-bit [..., NG]), in 32 bits."""
    y = x.to(F32).unflatten(-1, (-1, group))
    low, high = y.amin(-1), y.amax(-1)
    span = high - low
    bad = ~torch.isfinite(span)
    scale = torch.where(bad, torch.full_like(span, float("nan")), span / 15).to(x.dtype)
    zero = torch.where(bad, torch.full_like(span, float("nan")), low).to(x.dtype)
    s, z = scale.to(F32)[..., None], zero.to(F32)[..., None]
    codes = torch.where(s > 0, torch.round((y - z) / s).clamp(0, 15), torch.zeros_like(y))
    return codes.to(torch.uint8).flatten(-2), scale, zero


def _to_blocks(k, v, group):
    """k, v [..., P, D] of whole pages -> the bytes of their blocks [..., block_bytes]."""
    lead, (p, d) = k.shape[:-2], k.shape[-2:]
    u = d // 32
    kc, ks, kz = _quantise(k, group)
    vc, vs, vz = _quantise(v, group)
    kc = kc.reshape(*lead, p, u, 4, 8).transpose(-3, -2)                        # (g, i, nibble)
    kb = (kc[..., 0::2] | kc[..., 1::2] << 4).reshape(*lead, p * d // 2)
    vc = vc.reshape(*lead, p // 4, 4, d // 16, 16).movedim(-1, -3)              # (t / 4, r, t % 4, i)
    vb = (vc[..., 0::2] | vc[..., 1::2] << 4).reshape(*lead, p * d // 2)
    par = [torch.stack((s, z), -1).transpose(-2, -3).contiguous().view(torch.uint8).reshape(*lead, -1)
           for s, z in ((ks, kz), (vs, vz))]
    return torch.cat((kb, vb, *par), -1)


def _values(shape, dtype, gen, outliers):
    """Activations of a trained model's kind: each dim with its own mean and spread, a few dims far out."""
    d = shape[-1]
    mean = torch.randn(shape[-2:], generator=gen, device="cuda") * 0.5
    spread = torch.rand(shape[-2:], generator=gen, device="cuda") + 0.5
    if outliers:
        mean = mean + 6.0 * (torch.rand((shape[-2], d), generator=gen, device="cuda") < 0.02)
    return (torch.randn(shape, generator=gen, device="cuda") * spread + mean).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, d = TYPES[case["dtype"]], case["dim"]
    if case["op"] == "rope":
        t, hq, hk, rot = case["tokens"], case["q_heads"], case["kv_heads"], case["rot"]
        positions = torch.randint(0, 32768, (t,), generator=gen, device="cuda", dtype=torch.int32)
        angle = torch.arange(32768, device="cuda", dtype=F64)[:, None] * 10000.0 ** (
            -2.0 * torch.arange(rot // 2, device="cuda", dtype=F64) / rot)
        state = dict(qkv=_values((t, hq + 2 * hk, d), dtype, gen, True), positions=positions,
                     table=torch.cat((angle.cos(), angle.sin()), -1).to(F32),
                     q_weight=(1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dtype),
                     k_weight=(1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dtype))
    elif case["op"] == "cache":
        t, hk, p = case["tokens"], case["kv_heads"], case["page"]
        pages = -(-t // p) + 3
        if case["scattered"]:
            pages = max(pages, -(-4 * t // p))
            slots = torch.randperm(pages * p, generator=gen, device="cuda")[:t]
        else:
            table = torch.randperm(pages, generator=gen, device="cuda")
            i = torch.arange(t, device="cuda")
            slots = table[i // p] * p + i % p
        qkv = _values((t, 2 * hk, d), dtype, gen, True)
        state = dict(k=qkv[:, :hk], v=qkv[:, hk:], slots=slots,
                     data=torch.zeros(pages * hk * _block_bytes(case), dtype=torch.uint8, device="cuda"), pages=pages)
    else:
        b, hq, hk, p = case["batch"], case["q_heads"], case["kv_heads"], case["page"]
        qs, ks = _lengths(case)
        columns = -(-max(ks) // p) + 1
        need = [-(-n // p) for n in ks]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        row = torch.arange(columns, device="cuda")[None, :]
        count = torch.tensor(need, device="cuda")[:, None]
        first = count.cumsum(0) - count
        table = torch.where(row < count, order[(first + row).clamp(max=pages - 1)], torch.zeros_like(order[:1])).to(torch.int32)
        # pages that nothing fills, and the slots past each request's end, hold what was there: any bits
        data = torch.randint(0, 256, (pages, hk * _block_bytes(case)), generator=gen, device="cuda", dtype=torch.uint8)
        step = max(1, (1 << 27) // (hk * p * d))
        for at in range(0, pages, step):
            n = min(step, pages - at)
            k, v = (_values((n * p, hk, d), dtype, gen, o).unflatten(0, (n, p)).transpose(1, 2) for o in (True, False))
            data[at:at + n] = _to_blocks(k, v, case["group"]).reshape(n, -1)
        ends = torch.tensor(ks, device="cuda")
        used = torch.arange(columns * p, device="cuda")[None, :] < ends[:, None]
        tail = (~used).unflatten(1, (columns, p)) & (row < count)[..., None]
        which, place = table[:, :, None].expand(-1, -1, p)[tail].long(), torch.arange(p, device="cuda").expand(b, columns, p)[tail]
        params = data.reshape(pages, hk, -1)[:, :, p * d:].reshape(pages, hk, 2 * (d // case["group"]), p, 4)
        params[which, :, :, place] = 255                                          # NaN where no token is
        data = torch.cat((data.reshape(pages, hk, -1)[:, :, :p * d], params.reshape(pages, hk, -1)), -1).reshape(-1)
        starts = [0]
        for n in qs:
            starts.append(starts[-1] + n)
        state = dict(q=_values((starts[-1], hq, d), dtype, gen, False) * (2.0 if case["q_high"] < 64 else 1.0), data=data, pages=pages, table=table,
                     lens=ends.to(torch.int32), starts=torch.tensor(starts, device="cuda", dtype=torch.int32),
                     # where each query row lies in the batch, for the plain form
                     row_b=torch.tensor([i for i, n in enumerate(qs) for _ in range(n)], device="cuda", dtype=torch.int64),
                     row_i=torch.tensor([j for n in qs for j in range(n)], device="cuda", dtype=torch.int64),
                     max_q=max(qs))
    state["case"] = dict(case)
    if own:
        _keep(state)
    return state


# ----------------------------------------------------------------------------- the library's calls
def _keep(state):
    """What a program of the library keeps between calls: descriptors, output buffers, the workspace."""
    import weight_only_quantized_qgemm_amd as q
    case = state["case"]
    dtype = {"f16": q.DT_F16, "bf16": q.DT_BF16}[case["dtype"]]
    t16, d = TYPES[case["dtype"]], case["dim"]
    state["lib"] = q
    if case["op"] == "rope":
        hq, hk, t = case["q_heads"], case["kv_heads"], case["tokens"]
        state["p"] = q.norm_rope_problem(t, hq, hk, d, dtype, rot_dim=case["rot"], max_pos=32768, interleaved=case["interleaved"],
                                         eps=1e-6)
        state["q_out"] = torch.empty((t, hq, d), dtype=t16, device="cuda")
        state["k_out"] = torch.empty((t, hk, d), dtype=t16, device="cuda")
        return
    state["cache"] = q.cache(state["pages"], case["page"], case["kv_heads"], d, dtype, group_size=case["group"])
    if case["op"] == "cache":
        for name in ("k_out", "v_out"):
            state[name] = torch.empty((case["tokens"], case["kv_heads"], d), dtype=t16, device="cuda")
    else:
        state["p"] = q.attention_problem(state["cache"], case["batch"], state["q"].shape[0], case["q_heads"], state["max_q"],
                                         state["table"].shape[1], causal=case["causal"], window=case["window"])
        state["ws"] = q.alloc_attention_workspace(state["p"])
        state["out"] = torch.empty(state["q"].shape, dtype=t16, device="cuda")


def _run_own(state):
    q, case = state["lib"], state["case"]
    if case["op"] == "rope":
        hq, hk = case["q_heads"], case["kv_heads"]
        q.qk_norm_rope(state["p"], state["qkv"][:, :hq], state["qkv"][:, hq:hq + hk], state["q_weight"], state["k_weight"],
                       state["positions"], state["table"], state["q_out"], state["k_out"])
        return {"q": state["q_out"], "k": state["k_out"]}
    if case["op"] == "cache":
        q.cache_write(state["cache"], state["data"], state["k"], state["v"], state["slots"])
        q.cache_read(state["cache"], state["data"], state["slots"], state["k_out"], state["v_out"])
        return {"k": state["k_out"], "v": state["v_out"]}
    q.attention(state["p"], state["q"], state["data"], state["table"], state["lens"], state["starts"], state["out"], state["ws"])
    return {"out": state["out"]}


# ----------------------------------------------------------------------------- the plain forms
def _plain_rope(state):
    case, dtype = state["case"], TYPES[state["case"]["dtype"]]
    hq, hk, rot = case["q_heads"], case["kv_heads"], case["rot"]
    x = state["qkv"][:, :hq + hk].to(F32)
    w = torch.cat((state["q_weight"].to(F32).expand(hq, -1), state["k_weight"].to(F32).expand(hk, -1)))
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    rows = state["table"][state["positions"].long()][:, None]
    c, s = rows[..., :rot // 2], rows[..., rot // 2:]
    head = y[..., :rot]
    a, b = (head[..., 0::2], head[..., 1::2]) if case["interleaved"] else (head[..., :rot // 2], head[..., rot // 2:])
    a, b = a * c - b * s, b * c + a * s
    head = torch.stack((a, b), -1).flatten(-2) if case["interleaved"] else torch.cat((a, b), -1)
    y = torch.cat((head, y[..., rot:]), -1).to(dtype)
    return {"q": y[:, :hq].contiguous(), "k": y[:, hq:].contiguous()}


def _nibbles(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _from_blocks(blocks, case):
    """Bytes of blocks [..., block_bytes] -> k, v [..., P, D] in 32 bits."""
    lead, p, d, ng, u = blocks.shape[:-1], case["page"], case["dim"], case["dim"] // case["group"], case["dim"] // 32
    n, m = p * d // 2, p * ng * 4
    kc = _nibbles(blocks[..., :n].reshape(*lead, p, 4, u, 4)).transpose(-2, -3).reshape(*lead, p, ng, -1).to(F32)
    vc = _nibbles(blocks[..., n:2 * n].reshape(*lead, p // 4, 16, 4, u))             # (t / 4, r, t % 4, i)
    vc = vc.transpose(-2, -3).transpose(-1, -2).reshape(*lead, p, ng, -1).to(F32)
    kp, vp = (blocks[..., 2 * n + i * m:2 * n + (i + 1) * m].contiguous().view(TYPES[case["dtype"]]).reshape(*lead, ng, p, 2)
              .transpose(-2, -3).to(F32) for i in (0, 1))
    return [(c * q[..., :1] + q[..., 1:]).flatten(-2) for c, q in ((kc, kp), (vc, vp))]


def _plain_cache(state):
    """Written to the blocks of its slots as codes and parameters, then read back from there."""
    case, dtype = state["case"], TYPES[state["case"]["dtype"]]
    p, d, hk, ng, u = case["page"], case["dim"], case["kv_heads"], case["dim"] // case["group"], case["dim"] // 32
    blocks = state["data"].reshape(-1, hk, _block_bytes(case))
    page, t, n = state["slots"] // p, state["slots"] % p, p * d // 2
    kc, ks, kz = _quantise(state["k"], case["group"])
    vc, vs, vz = _quantise(state["v"], case["group"])
    kc = kc.reshape(-1, hk, u, 4, 8).transpose(2, 3)
    kb = (kc[..., 0::2] | kc[..., 1::2] << 4).reshape(-1, hk, d // 2)
    vc = vc.reshape(-1, hk, d // 16, 16).transpose(2, 3)
    vb = vc[..., 0::2] | vc[..., 1::2] << 4
    heads = torch.arange(hk, device="cuda")
    blocks[..., :n].unflatten(-1, (p, d // 2))[page, :, t] = kb
    blocks[..., n:2 * n].unflatten(-1, (p // 4, 16, 4, u))[page[:, None], heads, t[:, None] // 4, :, t[:, None] % 4] = vb
    par = blocks[..., 2 * n:].unflatten(-1, (2 * ng, p, 4))
    both = torch.cat((torch.stack((ks, kz), -1), torch.stack((vs, vz), -1)), 2).contiguous().view(torch.uint8)
    par[page[:, None], heads, :, t[:, None]] = both
    kb = blocks[..., :n].unflatten(-1, (p, d // 2))[page, :, t]
    vb = blocks[..., n:2 * n].unflatten(-1, (p // 4, 16, 4, u))[page[:, None], heads, t[:, None] // 4, :, t[:, None] % 4]
    got = par[page[:, None], heads, :, t[:, None]].contiguous().view(dtype).to(F32)   # [n, hk, 2 ng, 2]
    kc = _nibbles(kb.reshape(-1, hk, 4, u, 4)).transpose(-2, -3).reshape(-1, hk, ng, case["group"]).to(F32)
    vc = _nibbles(vb).transpose(-1, -2).reshape(-1, hk, ng, case["group"]).to(F32)
    k, v = ((c * q[..., :1] + q[..., 1:]).flatten(-2).to(dtype) for c, q in ((kc, got[:, :, :ng]), (vc, got[:, :, ng:])))
    return {"k": k, "v": v}


def _plain_attention(state):
    case = state["case"]
    b, hq, hk, d, p = case["batch"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    columns, max_q = state["table"].shape[1], state["max_q"]
    k, v = _from_blocks(state["data"].reshape(-1, hk, _block_bytes(case))[state["table"].long()], case)
    k, v = (x.transpose(1, 2).reshape(b, hk, 1, columns * p, d) for x in (k, v))
    lens, starts = state["lens"].long(), state["starts"].long()
    n = starts[1:] - starts[:-1]
    i = torch.arange(max_q, device="cuda")
    rows = (starts[:-1, None] + i).clamp(max=state["q"].shape[0] - 1)
    q = state["q"].to(F32)[rows].transpose(1, 2).reshape(b, hk, hq // hk, max_q, d)
    t = torch.arange(columns * p, device="cuda")
    seen = t < lens[:, None, None]
    if case["causal"]:
        at = (lens - n)[:, None, None] + i[:, None]
        seen = seen & (t <= at)
        if case["window"]:
            seen = seen & (t > at - case["window"])
    v = torch.where((t < lens[:, None])[:, None, None, :, None], v, torch.zeros_like(v))
    s = torch.matmul(q.reshape(b, hk, -1, d), k[:, :, 0].transpose(-1, -2)).reshape(b, hk, hq // hk, max_q, -1)
    s = torch.where(seen.reshape(b, 1, 1, -1, columns * p), s * (1 / math.sqrt(d)), torch.full_like(s[:1, :1, :1, :1, :1], -math.inf))
    w = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.reshape(b, hk, -1, columns * p), v[:, :, 0]).reshape(b, hk, hq // hk, max_q, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).reshape(b, hq, max_q, d)
    return {"out": o[state["row_b"], :, state["row_i"]].to(TYPES[case["dtype"]])}


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "cache": _plain_cache, "attention": _plain_attention}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------- cost
def work(case):
    d = case["dim"]
    if case["op"] == "rope":
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * d
        return {"bytes": 4 * n + case["tokens"] * (case["rot"] + 1) * 4 + 4 * d, "flops": 8 * n}
    token = d + 8 * (d // case["group"])                                       # cache bytes of a token and kv head
    if case["op"] == "cache":
        n = case["tokens"] * case["kv_heads"]
        return {"bytes": n * (4 * d + token) + n * (token + 4 * d) + 16 * case["tokens"], "flops": 10 * n * d}
    pairs = seen = 0
    qs, ks = _lengths(case)
    for n, k in zip(qs, ks):
        if not n:
            continue
        if not case["causal"]:
            pairs, seen = pairs + n * k, seen + k
            continue
        w = case["window"] or k
        pairs += sum(min(w, k - n + i + 1) for i in range(n))
        seen += min(k, w + n - 1)
    return {"bytes": seen * case["kv_heads"] * token + 4 * sum(qs) * case["q_heads"] * d + 4 * sum(-(-k // case["page"]) for k in ks),
            "flops": 4 * pairs * case["q_heads"] * d}


# ----------------------------------------------------------------------------- the definition in 64 bits
def _cell(case, t, kind):
    """Byte offset in a block and shift of each dim's code, and offsets of the (scale, zero) 16-bit words; t: slots in the page."""
    d, p, g = case["dim"], case["page"], case["group"]
    u, dim = d // 32, torch.arange(d, device="cuda")
    if kind == "k":
        block = dim // 8
        code = t[:, None] * (d // 2) + (u * (block % 4) + block // 4) * 4 + dim % 8 // 2
        shift = dim % 2 * 4
    else:
        i, r = dim // 16, dim % 16
        code = p * d // 2 + ((t[:, None] // 4) * 16 + r) * 4 * u + t[:, None] % 4 * u + i // 2
        shift = i % 2 * 4
    par = p * d + (0 if kind == "k" else p * (d // g) * 4) + (dim // g * p + t[:, None]) * 4
    return code, shift, par


def _value64(case, blocks, page, t, head, kind):
    """Values [len(t), D] in 64 bits of the cache's slots."""
    code, shift, par = _cell(case, t, kind)
    one = blocks[:, head]
    c = (one[page[:, None], code].long() >> shift & 15).to(F64)
    word = [one[page[:, None], par + j].int() | one[page[:, None], par + j + 1].int() << 8 for j in (0, 2)]
    s, z = (x.to(torch.int16).view(TYPES[case["dtype"]]).to(F64) for x in word)
    return c * s + z


def exact(case, seed):
    state = prepare(case, seed)
    d = case["dim"]
    if case["op"] == "rope":
        hq, hk, rot = case["q_heads"], case["kv_heads"], case["rot"]
        out = []
        for x, w in ((state["qkv"][:, :hq], state["q_weight"]), (state["qkv"][:, hq:hq + hk], state["k_weight"])):
            x = x.to(F64)
            y = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + 1e-6) * w.to(F64)
            row = state["table"].to(F64)[state["positions"].long()]
            pair = torch.arange(rot // 2, device="cuda")
            first, second = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + rot // 2)
            z = torch.complex(y[..., first], y[..., second]) * torch.complex(row[:, :rot // 2], row[:, rot // 2:])[:, None]
            y = y.clone()
            y[..., first], y[..., second] = z.real, z.imag
            out.append(y)
        return {"q": out[0], "k": out[1]}
    if case["op"] == "cache":
        out = []
        for x in (state["k"], state["v"]):
            y = x.to(F64).reshape(case["tokens"], case["kv_heads"], -1, case["group"])
            z = y.min(-1, keepdim=True).values
            s = ((y.max(-1, keepdim=True).values - z) / 15).to(F32).to(x.dtype).to(F64)
            c = torch.where(s > 0, torch.clamp(torch.round((y - z) / s), 0, 15), torch.zeros_like(y))
            out.append((c * s + z).reshape(x.shape))
        return {"k": out[0], "v": out[1]}
    hq, hk, p = case["q_heads"], case["kv_heads"], case["page"]
    blocks = state["data"].reshape(state["pages"], hk, -1)
    qs, ks = _lengths(case)
    out, at = torch.zeros(state["q"].shape, dtype=F64, device="cuda"), 0
    for b, (n, length) in enumerate(zip(qs, ks)):
        for h in range(hk if n else 0):
            t = torch.arange(length, device="cuda")
            page = state["table"][b].long()[t // p]
            k, v = (_value64(case, blocks, page, t % p, h, kind) for kind in "kv")
            for first in range(0, n, 2048):
                rows = torch.arange(first, min(n, first + 2048), device="cuda")
                q = state["q"][at + rows][:, h * (hq // hk):(h + 1) * (hq // hk)].to(F64)
                s = (q.reshape(-1, d) @ k.T).reshape(len(rows), -1, length) / math.sqrt(d)
                if case["causal"]:
                    place = (length - n + rows)[:, None, None]
                    hidden = (t > place) | ((t <= place - case["window"]) if case["window"] else torch.zeros_like(t, dtype=torch.bool))
                    s = s.masked_fill(hidden, -math.inf)
                w = torch.softmax(s, -1)
                out[at + rows, h * (hq // hk):(h + 1) * (hq // hk)] = (w.reshape(-1, length) @ v).reshape(len(rows), -1, d)
        at += n
    return {"out": out}
