"""Launches of qgemm_attention that ordinary small cases do not reach, against the 64-bit oracle:
few queries over a context split between many workgroups (numbers of parts that are not powers of
two among them), hundreds of requests, wavefronts that work on their own, shared pages, NaN groups,
graph replays of a split launch, side streams of the head and cache operators."""
import numpy as np
import pytest

from gpu_cases import say
from oracle import attention as oa
from test_gpu_attention import T16, _check, _run, _sequences, dt, same_bits, up

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_qgemm_amd as lib
    return lib


def scale_of(dim):
    return np.float64(np.float32(dim ** -0.5))


# kind, query lengths, context lengths, q_heads, kv_heads, dim, group, page, causal, window, parts
SPLIT = [
    ("f16", [64], [1300], 2, 1, 64, 64, 16, True, 0, 4),
    ("f16", [70], [2100], 1, 1, 128, 128, 16, True, 0, 7),
    ("bf16", [40, 3], [3000, 900], 4, 2, 128, 32, 48, True, 0, 12),
    ("f16", [33, 20], [1500, 20], 2, 2, 256, 64, 64, True, 0, 5),
    ("bf16", [100], [900], 1, 1, 256, 128, 16, True, 70, 3),
    ("bf16", [30, 30, 0], [700, 30, 500], 2, 1, 64, 32, 32, False, 0, 3),
    ("f16", [50], [2100], 3, 1, 128, 64, 16, True, 1000, 7),              # parts outside the window
]


@pytest.mark.parametrize("case", range(len(SPLIT)))
def test_split_context(q, case):
    kind, qlens, klens, hq, hk, dim, group, page, causal, window, parts = SPLIT[case]
    say(f"case attention split {SPLIT[case]}")
    s = _sequences(q, kind, qlens, klens, hq, hk, dim, group, page, 100 + case, spread=1.5)
    p = q.attention_problem(s["c"], len(klens), sum(qlens), hq, max(qlens), s["max_pages"], causal=causal, window=window,
                            kernel_hint=q.ATTENTION_TILES)
    assert q.attention_describe(p).endswith(f"splits={parts}")
    out = _run(q, s, kind, hq, causal, window, hint=q.ATTENTION_TILES, extra=8)
    _check(s, out, kind, hq, causal, window, scale_of(dim))


@pytest.mark.parametrize("kind,heads,dim,group,hint", [
    ("f16", (16, 8), 64, 64, 0), ("bf16", (8, 8), 128, 32, 0), ("bf16", (16, 8), 64, 32, 2), ("f16", (8, 8), 256, 64, 1)])
def test_hundreds_of_requests(q, kind, heads, dim, group, hint):
    # 210 requests of every length from 0 on, a query each except every seventh
    say(f"case attention 210 requests {kind} {heads} D={dim} hint={hint}")
    klens = [(i * 37) % 131 for i in range(210)]
    qlens = [0 if i % 7 == 3 else 1 for i in range(210)]
    s = _sequences(q, kind, qlens, klens, *heads, dim, group, 16, 200)
    p = q.attention_problem(s["c"], 210, sum(qlens), heads[0], 1, s["max_pages"], kernel_hint=hint)
    assert hint == 2 or "waves=1" in q.attention_describe(p)
    out = _run(q, s, kind, heads[0], hint=hint)
    _check(s, out, kind, heads[0], True, 0, scale_of(dim))


def test_many_prompts(q):
    say("case attention 90 prompts")
    qlens = [(i * 29) % 41 for i in range(90)]
    klens = [n + (i * 53) % 67 for i, n in enumerate(qlens)]
    s = _sequences(q, "bf16", qlens, klens, 4, 1, 64, 64, 16, 201)
    for hint in (0, 1, 2):
        _check(s, _run(q, s, "bf16", 4, hint=hint, max_q=41), "bf16", 4, True, 0, scale_of(64))


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("group", [64, 256])
def test_six_rows_of_the_widest_heads(q, kind, group):
    say(f"case attention D=256 six rows {kind} group={group}")
    s = _sequences(q, kind, [3, 2], [190, 333], 4, 2, 256, group, 16, 202)
    _check(s, _run(q, s, kind, 4, hint=q.ATTENTION_ROWS), kind, 4, True, 0, scale_of(256))


@pytest.mark.parametrize("hint", [1, 2])
def test_requests_that_share_pages(q, hint):
    # three requests over one context's pages: the same rows give the same bits
    say(f"case attention shared pages hint={hint}")
    s = _sequences(q, "f16", [2], [95], 8, 2, 128, 64, 32, 203)
    alone = _run(q, s, "f16", 8, hint=hint)
    _check(s, alone, "f16", 8, True, 0, scale_of(128))
    three = dict(s, table=s["table"].repeat(3, 1), lens=s["lens"].repeat(3), q=np.concatenate([s["q"]] * 3), qlens=[2] * 3,
                 klens=[95] * 3, seqs=s["seqs"] * 3, starts=torch.tensor([0, 2, 4, 6], dtype=torch.int32, device="cuda"))
    out = _run(q, three, "f16", 8, hint=hint)
    assert torch.equal(out[:2], out[2:4]) and torch.equal(out[:2], out[4:])
    _check(three, out, "f16", 8, True, 0, scale_of(128))


@pytest.mark.parametrize("hint", [1, 2])
@pytest.mark.parametrize("kind,dim,group", [("bf16", 128, 32), ("bf16", 256, 64), ("f16", 64, 32), ("bf16", 64, 64)])
def test_one_group_that_is_not_finite(q, kind, dim, group, hint):
    # NaN in one group of one token's value: the dims of that group are NaN for the queries that see the
    # token, the others (and every earlier query) keep their bits
    say(f"case attention NaN group {kind} D={dim} G={group} hint={hint}")
    s = _sequences(q, kind, [60], [60], 2, 1, dim, group, 16, 204)
    clean = _run(q, s, kind, 2, hint=hint)
    k, v = (torch.empty(1, 1, dim, dtype=T16[kind], device="cuda") for _ in "kv")
    at = torch.tensor([int(s["table"][0, 2]) * 16 + 5], device="cuda")               # token 37
    q.cache_read(s["c"], s["data"], at, k, v)
    rewritten = v.clone()
    rewritten[..., dim - group:] = float("nan")
    q.cache_write(s["c"], s["data"], k, v, at)                                        # requantized, finite
    base = _run(q, s, kind, 2, hint=hint)
    assert same_bits(base[:37], clean[:37])
    q.cache_write(s["c"], s["data"], k, rewritten, at)
    dirty = _run(q, s, kind, 2, hint=hint)
    assert same_bits(dirty[:37], clean[:37])
    assert torch.isnan(dirty[37:, :, dim - group:]).all()
    if group < dim:
        assert torch.isfinite(dirty[37:, :, :dim - group]).all()


def test_graph_replays_of_a_split_launch(q):
    # the parts' tickets and partial results are ready again after every replay
    say("case attention graph of a split launch")
    s = _sequences(q, "bf16", [40], [1500], 4, 2, 128, 64, 16, 205)
    p = q.attention_problem(s["c"], 1, 40, 4, 40, s["max_pages"], kernel_hint=q.ATTENTION_TILES)
    assert "splits=1" not in q.attention_describe(p).split()
    ws, out, qx = q.alloc_attention_workspace(p), torch.zeros(40, 4, 128, dtype=torch.bfloat16, device="cuda"), up(s["q"], "bf16")
    table = s["table"].clamp(min=0)
    args = (p, qx, s["data"], table, s["lens"], s["starts"])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        q.attention(*args, out, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.attention(*args, out, ws)
    for length in (1500, 40, 777, 39, 0, 1499):
        s["lens"].fill_(length)
        out.fill_(9.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        eager = torch.zeros_like(out)
        q.attention(*args, eager, q.alloc_attention_workspace(p))
        torch.cuda.synchronize()
        assert torch.equal(out, eager), length


def test_head_and_cache_operators_on_side_streams(q):
    say("case norm_rope and cache on a side stream")
    x = torch.randn(5, 3, 128, device="cuda").half()
    pos, table = torch.arange(5, dtype=torch.int32, device="cuda"), torch.randn(8, 128, device="cuda")
    p = q.norm_rope_problem(5, 2, 1, 128, rot_dim=128, max_pos=8)
    c = q.cache(2, 16, 1, 128, q.DT_F16)
    slots = torch.tensor([3, 30, 7, 0, 19], device="cuda")

    def steps(src, data, stream=None):
        o, kv = torch.empty_like(src), [torch.empty(5, 1, 128, dtype=torch.float16, device="cuda") for _ in "kv"]
        q.qk_norm_rope(p, src[:, :2], src[:, 2:], None, None, pos, table, o[:, :2], o[:, 2:], stream=stream)
        q.cache_write(c, data, o[:, 2:], src[:, 2:], slots, stream=stream)
        q.cache_read(c, data, slots, *kv, stream=stream)
        return o, *kv

    want = steps(x, q.alloc_cache(c))
    side = torch.cuda.Stream()
    late, data = torch.zeros_like(x), q.alloc_cache(c)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(x)
        got = steps(late, data)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    late.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(x)
    got = steps(late, data, stream=side)                     # named, from another current stream
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_one_workspace_for_every_problem(q):
    # a zero-filled workspace of the largest size, in stream order: whatever ran before, the same bits
    say("case attention one workspace")
    made = [("f16", [1] * 5, [300, 1, 900, 64, 2000], 8, 2, 128, 64, 1), ("f16", [70], [2100], 1, 1, 128, 128, 2),
            ("bf16", [1], [1800], 32, 2, 256, 256, 1), ("bf16", [33, 20], [1500, 20], 2, 2, 256, 64, 2),
            ("f16", [1] * 40, [90] * 40, 64, 64, 64, 32, 1)]
    calls = []
    for i, (kind, qlens, klens, hq, hk, dim, group, hint) in enumerate(made):
        s = _sequences(q, kind, qlens, klens, hq, hk, dim, group, 16, 300 + i)
        p = q.attention_problem(s["c"], len(klens), sum(qlens), hq, max(qlens), s["max_pages"], kernel_hint=hint)
        calls.append((p, up(s["q"], kind), s["data"], s["table"], s["lens"], s["starts"]))
    want = []
    for args in calls:
        out = torch.zeros_like(args[1])
        q.attention(*args, out, q.alloc_attention_workspace(args[0]))
        want.append(out)
    ws = torch.zeros(max(q.attention_workspace_bytes(a[0]) for a in calls), dtype=torch.uint8, device="cuda")
    for i in (0, 1, 2, 3, 4, 1, 0, 3, 3, 4, 2, 0, 1):
        out = torch.zeros_like(want[i])
        q.attention(*calls[i], out, ws)
        assert torch.equal(out, want[i]), i


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_cache_codes_for_every_scale(q, kind):
    # every significand a scale can have, at sizes from the smallest subnormal to the largest, elements at
    # and next to the ties between codes: codes and parameters are the definition's
    say(f"case cache every scale {kind}")
    g = np.random.default_rng([30, len(kind)])
    bits = 10 if kind == "f16" else 7
    sizes = [2.0 ** -24, 2.0 ** -20, 2.0 ** -15, 2.0 ** -14, 2.0 ** -13, 1.0, 2.0 ** 10] if kind == "f16" else \
        [2.0 ** -133, 2.0 ** -126, 2.0 ** -100, 2.0 ** -61, 2.0 ** -60, 2.0 ** -59, 1.0, 2.0 ** 60, 2.0 ** 120]
    heads, dim = 2, 128
    for size in sizes:
        scale = (1 + np.arange(2 ** bits) / 2 ** bits) * size
        n = len(scale)
        c = g.integers(0, 15, (n, heads, dim)) + 0.5 + g.choice([0, 0, 1e-3, -1e-3, 3e-2, -3e-2, 0.4], (n, heads, dim))
        x = oa.round16(c * scale[:, None, None], kind)
        x[:, :, 0], x[:, :, 1] = 0.0, oa.round16(15 * scale, kind)[:, None]
        x = oa.round16(x - oa.round16(g.integers(0, 3, (n, 1, 1)) * 5 * scale[:, None, None], kind), kind)
        assert np.isfinite(x).all()
        c = q.cache(-(-n // 16), 16, heads, dim, dt(q, kind), group_size=64)
        data = q.alloc_cache(c)
        slots = torch.arange(n, device="cuda")
        q.cache_write(c, data, up(x, kind), up(x[:, ::-1], kind), slots)
        parts = [oa.quantize(a, 64, kind) for a in (x, x[:, ::-1])]
        got, at = data.cpu().numpy().reshape(-1, heads, oa.block_bytes(16, dim, 64)), 0
        for page in range(-(-n // 16)):
            m = min(16, n - at)
            for h in range(heads):
                full = []
                for codes, s, z in parts:
                    cc, ss, zz = np.zeros((16, dim), np.uint8), np.zeros((16, 2)), np.zeros((16, 2))
                    cc[:m], ss[:m], zz[:m] = codes[at:at + m, h], s[at:at + m, h], z[at:at + m, h]
                    full += [cc, ss, zz]
                want = oa.pack_block(*full, kind)
                par = 16 * dim                                        # zeros of either sign are one value
                assert np.array_equal(got[page, h, :par], want[:par]), (size, page, h)
                assert np.array_equal(*(oa.from_bits16(b[par:].copy().view(np.uint16), kind) for b in (got[page, h], want)))
            at += m


@pytest.mark.parametrize("hint", [1, 2])
@pytest.mark.parametrize("kind,dim,group,apart", [("bf16", 128, 32, 7), ("bf16", 256, 64, 6), ("bf16", 64, 32, 20), ("f16", 128, 32, 3)])
def test_key_groups_of_different_size(q, kind, dim, group, apart, hint):
    # each group of keys 2^apart smaller than the one before, the queries as much larger there: every
    # group weighs the same in the scores
    say(f"case attention key groups apart {kind} D={dim} G={group} by 2^{apart} hint={hint}")
    s = _sequences(q, kind, [40, 1], [150, 70], 4, 2, dim, group, 16, 206)
    ng = dim // group
    step = 2.0 ** (-apart * np.arange(ng))
    for b, k in enumerate(s["klens"]):
        (kc, ks, kz), v = s["seqs"][b]
        s["seqs"][b] = [(kc, ks * step, kz * step), v]                # powers of two: values of the type
        assert np.array_equal(oa.round16(ks * step, kind), ks * step) or kind == "f16"
    # the same in the cache: the parameters' exponents
    page, hk = 16, 2
    u8 = s["data"].cpu().numpy().reshape(-1, hk, oa.block_bytes(page, dim, group))
    par = u8[:, :, page * dim:page * dim + page * ng * 4].copy().view(np.uint16).reshape(-1, hk, ng, page, 2)
    value = oa.from_bits16(par, kind) * step[:, None, None]
    bits = np.where(np.isnan(value), par, oa.bits16(np.nan_to_num(value), kind))
    u8[:, :, page * dim:page * dim + page * ng * 4] = bits.astype(np.uint16).reshape(*u8.shape[:2], -1).view(np.uint8)
    if kind == "f16":                                                 # fp16 rounds the smallest of them
        for b in range(2):
            (kc, ks, kz), v = s["seqs"][b]
            s["seqs"][b] = [(kc, oa.round16(ks, kind), oa.round16(kz, kind)), v]
    s["data"] = torch.from_numpy(u8.reshape(-1)).cuda()
    s["q"] = oa.round16(s["q"] * np.repeat(1 / step, group) * step[-1], kind)
    scale = float(np.float32(dim ** -0.5 / step[-1]))
    _check(s, _run(q, s, kind, 4, scale=scale, hint=hint), kind, 4, True, 0, scale)
