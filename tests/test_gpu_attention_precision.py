"""Attention where numbers of very different size meet, against the 64-bit oracle and a bound that allows
the formats' own rounding only: a dominating token over a long context, value groups and query heads of different
magnitude, a huge scale of negligible weight, scores and values at the end of the type's range."""
import numpy as np
import pytest

from gpu_cases import say
from oracle import attention as oa
from test_gpu_attention import T16, _run, down, dt, up

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# what is kept of a weight far below the largest of its group: fp16's 2^-25 against a largest that stands at 2^6 at
# least, and in the tiles kernel, where the groups of a row share a reference, two bits less
FLOOR = {1: 2.0 ** -31, 2: 2.0 ** -29}


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_qgemm_amd as lib
    return lib


def store(q, kind, k, v, qx, group, page=64):
    """One sequence: k, v [kv_heads, tokens, D] and queries [n, q_heads, D], values of the type."""
    hk, n, dim = k.shape
    pages = -(-n // page)
    c = q.cache(pages, page, hk, dim, dt(q, kind), group_size=group)
    data = q.alloc_cache(c)
    q.cache_write(c, data, up(k.swapaxes(0, 1), kind), up(v.swapaxes(0, 1), kind), torch.arange(n, device="cuda"))
    return dict(c=c, data=data, table=torch.arange(pages, dtype=torch.int32, device="cuda")[None], q=qx,
                parts=[oa.quantize(x, group, kind) for x in (k, v)], group=group, max_pages=pages, qlens=[len(qx)], klens=[n],
                lens=torch.tensor([n], dtype=torch.int32, device="cuda"),
                starts=torch.tensor([0, len(qx)], dtype=torch.int32, device="cuda"))


def check(s, out, kind, hint, scale):
    got, group, worst = down(out), s["group"], 0.0
    ratio = s["q"].shape[1] // s["c"].kv_heads
    for h in range(s["q"].shape[1]):
        (kc, ks, kz), (vc, vs, vz) = [[a[h // ratio] for a in part] for part in s["parts"]]
        val = oa.dequantize(vc, vs, vz, group)
        want, w = oa.attention(s["q"][:, h], oa.dequantize(kc, ks, kz, group), val, s["klens"][0], True, 0, scale)
        bound = oa.attention_weight_bound(s["q"][:, h], w, val, want, ks, kz, vs, vz, group, scale, kind, FLOOR[hint],
                                          hint == 2 and kind == "bf16")
        off = np.abs(got[:, h] - want)
        assert np.isfinite(want).all() and np.isfinite(off).all()
        worst = max(worst, float(np.max(off / np.maximum(bound, 1e-300))))
        say(f"  head {h}: largest error / bound {float(np.max(off / np.maximum(bound, 1e-300))):.3f}")
    assert worst <= 1, worst


KINDS = pytest.mark.parametrize("kind", ["f16", "bf16"])
KERNELS = pytest.mark.parametrize("hint", [1, 2])


@KERNELS
@KINDS
@pytest.mark.parametrize("below,sink", [(17.5, 1.0), (16.0, 0.0), (17.5, 0.0)])
def test_a_dominating_token_over_a_long_context(q, kind, below, sink, hint):
    # 131072 tokens, all but one e^-below of the largest: together they still count
    say(f"case attention dominating token {kind} hint={hint} e^-{below} value {sink}")
    g = np.random.default_rng([60, hint])
    n, dim, rows = 131072, 64, 1 if hint == 1 else 33
    k, v = np.zeros((1, n, dim)), np.empty((1, n, dim))
    k[0] = oa.round16(0.002 * g.standard_normal((n, 1)), kind)
    v[0] = np.linspace(-1, 1, dim) + 0.2 * g.standard_normal((n, dim)) - 0.3
    k[0, 100], v[0, 100] = 2.0, sink * v[0, 100]
    qx = np.full((rows, 1, dim), 1.0)
    s = store(q, kind, k, oa.round16(v, kind), qx, dim, 256)
    scale = float(np.float32(below / (2 * dim)))
    check(s, _run(q, s, kind, 1, scale=scale, hint=hint), kind, hint, scale)


@KERNELS
@KINDS
@pytest.mark.parametrize("dim,group", [(64, 64), (128, 32), (256, 128)])
@pytest.mark.parametrize("at", [0, 20, 59])
def test_a_dominating_token_without_a_value(q, kind, dim, group, at, hint):
    # the largest score by far belongs to a token whose value is 0: the others make the result
    say(f"case attention dominating zero value {kind} D={dim} G={group} at {at} hint={hint}")
    g = np.random.default_rng([66, dim, group])
    n = 60
    k, v = oa.round16(0.1 * g.standard_normal((1, n, dim)), kind), 1000 * g.standard_normal((1, n, dim))
    k[0, at], v[0, at] = 20.0 / dim, 0.0
    s = store(q, kind, oa.round16(k, kind), oa.round16(v, kind), np.full((1, 2, dim), 1.0), group, 16)
    check(s, _run(q, s, kind, 2, scale=1.0, hint=hint), kind, hint, 1.0)


@KERNELS
@KINDS
@pytest.mark.parametrize("below", [16.0, 17.5])
def test_a_dominating_token_in_one_part(q, kind, below, hint):
    # requests so many that a workgroup walks a whole context (they share its pages): one token is e^below times each
    # of the 131071 others, whose sum stands in the dims where its value is 0
    say(f"case attention dominating token, one part {kind} hint={hint} e^-{below}")
    g = np.random.default_rng([67])
    n, dim, batch = 131072, 64, 5000
    odd = np.arange(dim) % 2
    k, v = np.zeros((1, n, dim)), odd + 0.05 * g.standard_normal((1, n, dim))
    k[0, 5], v[0, 5] = 2.0, 1.0 - odd
    s = store(q, kind, k, oa.round16(v, kind), np.full((1, 1, dim), 1.0), dim, 256)
    many = dict(s, q=np.full((batch, 1, dim), 1.0), table=s["table"].repeat(batch, 1), lens=s["lens"].repeat(batch), qlens=[1] * batch,
                klens=[n] * batch, starts=torch.arange(batch + 1, dtype=torch.int32, device="cuda"))
    p = q.attention_problem(s["c"], batch, batch, 1, 1, s["max_pages"], kernel_hint=hint)
    assert hint == 1 or q.attention_describe(p).endswith("splits=1")
    scale = float(np.float32(below / (2 * dim)))
    out = _run(q, many, kind, 1, scale=scale, hint=hint)
    assert hint == 1 or torch.equal(out, out[:1].expand_as(out))
    for i in (0, 1234, batch - 1):
        check(s, out[i:i + 1], kind, hint, scale)


def sizes(kind, ng, order):
    """A size for each group, 2^20 (fp16) or 2^30 (bf16) between the first and the last."""
    top, far = (11.0, 20.0) if kind == "f16" else (0.0, 30.0)
    e = top - np.round(far * np.arange(ng) / (ng - 1))
    return 2.0 ** (e if order == "falling" else e[::-1])


@KERNELS
@KINDS
@pytest.mark.parametrize("dim,group", [(64, 32), (128, 64), (128, 32), (256, 128), (256, 64)])
@pytest.mark.parametrize("order", ["falling", "rising"])
def test_value_groups_far_apart(q, kind, dim, group, order, hint):
    say(f"case attention value groups apart {kind} D={dim} G={group} {order} hint={hint}")
    g = np.random.default_rng([61, dim, group])
    n, rows = 400, 40
    k = oa.round16(g.standard_normal((2, n, dim)), kind)
    v = (g.standard_normal((2, n, dim)) + g.standard_normal(dim)) * np.repeat(sizes(kind, dim // group, order), group)
    s = store(q, kind, k, oa.round16(v, kind), oa.round16(g.standard_normal((rows, 4, dim)), kind), group, 48)
    scale = float(np.float32(dim ** -0.5))
    check(s, _run(q, s, kind, 4, scale=scale, hint=hint), kind, hint, scale)


@KERNELS
@KINDS
@pytest.mark.parametrize("dim,group", [(64, 64), (64, 32), (128, 32), (256, 64)])
@pytest.mark.parametrize("at", [0, 70, 399])
@pytest.mark.parametrize("groups", ["all", "one"])
def test_a_huge_scale_of_negligible_weight(q, kind, dim, group, at, groups, hint):
    # one token's values are 2^16 (fp16) or 2^40 (bf16) times the others', its weight e^-60 of theirs
    say(f"case attention huge value, no weight {kind} D={dim} G={group} at {at} {groups} hint={hint}")
    g = np.random.default_rng([62, dim, group])
    n, rows = 400, 40
    k = oa.round16(0.3 * g.standard_normal((1, n, dim)), kind)
    v = g.standard_normal((1, n, dim))
    qx = oa.round16(0.1 * g.standard_normal((rows, 2, dim)) + 1, kind)
    k[0, at] = -60.0 / dim
    k = oa.round16(k, kind)
    v *= 0.125
    v[0, at, :group if groups == "one" else dim] *= 2.0 ** (16 if kind == "f16" else 40)
    s = store(q, kind, k, oa.round16(v, kind), qx, group, 16)
    check(s, _run(q, s, kind, 2, scale=1.0, hint=hint), kind, hint, 1.0)


@KERNELS
@KINDS
@pytest.mark.parametrize("dim,group", [(64, 64), (128, 32), (256, 128)])
def test_what_lies_before_the_window_is_not_read(q, kind, dim, group, hint):
    # slots of the window's first page that no query sees hold anything: the same bits
    say(f"case attention before the window {kind} D={dim} G={group} hint={hint}")
    g = np.random.default_rng([68, dim, group])
    n, rows, window = 150, 9, 100                                     # the first query sees tokens from 42 on
    k, v = (oa.round16(g.standard_normal((1, n, dim)), kind) for _ in "kv")
    outs = []
    for size in (1.0, 2.0 ** 12, np.nan):
        k2, v2 = k.copy(), v.copy()
        k2[:, :42] *= size
        v2[:, :42, :group] *= size
        s = store(q, kind, k2, v2, oa.round16(g.standard_normal((rows, 2, dim)), kind) if not outs else s["q"], group, 16)
        outs.append(_run(q, s, kind, 2, True, window, hint=hint))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@KERNELS
@pytest.mark.parametrize("kind,step", [("f16", 8), ("bf16", 25)])
@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("dim,group", [(64, 64), (128, 32), (256, 128)])
def test_query_heads_far_apart(q, kind, step, order, dim, group, hint):
    # four heads, each 2^step times the one before; the smallest head's scores are of ordinary size.  The same for
    # the tokens' queries in a second call
    for along in ("heads", "queries"):
        say(f"case attention query {along} apart {kind} by 2^{step} order {order} D={dim} G={group} hint={hint}")
        g = np.random.default_rng([63, dim, group])
        n, rows = 300, 4 if along == "queries" else 20
        base = 2.0 ** (-13 if kind == "f16" else -40)
        size = (base * 2.0 ** (step * np.arange(4)))[::order]
        qx = g.standard_normal((rows, 4, dim)) * (size[None, :, None] if along == "heads" else size[:, None, None])
        k, v = (oa.round16(g.standard_normal((1, n, dim)), kind) for _ in "kv")
        s = store(q, kind, k, v, oa.round16(qx, kind), group, 16)
        scale = float(np.float32(dim ** -0.5 / base))
        check(s, _run(q, s, kind, 4, scale=scale, hint=hint), kind, hint, scale)


@KERNELS
@pytest.mark.parametrize("dim,group", [(64, 64), (128, 32)])
def test_a_row_does_not_change_with_its_neighbours(q, dim, group, hint):
    # the first head alone, beside ordinary heads and beside one 2^40 times as large: the same bits
    say(f"case attention neighbours D={dim} G={group} hint={hint}")
    g = np.random.default_rng([64, dim])
    k, v = (oa.round16(g.standard_normal((1, 500, dim)), "bf16") for _ in "kv")
    qx = oa.round16(g.standard_normal((20, 4, dim)), "bf16")
    outs = []
    for other in (1.0, 2.0 ** 40, 2.0 ** -40):
        mixed = qx.copy()
        mixed[:, 1:] *= other
        mixed[::2, 1:] *= other
        s = store(q, "bf16", k, v, mixed, group, 16)
        outs.append(_run(q, s, "bf16", 4, scale=0.1, hint=hint)[:, 0])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@KERNELS
@pytest.mark.parametrize("size", [-1e28, -1e33, -1e37, 1e37])
def test_scores_at_the_end_of_the_range(q, size, hint):
    # scores far beyond 2^100 in magnitude: whatever 32 bits leave of their differences, a mean of the values with
    # weights that sum to 1, so between the smallest and the largest
    say(f"case attention scores of {size} hint={hint}")
    g = np.random.default_rng([65])
    n, dim = 90, 64
    v = oa.round16(3 + 0.3 * g.standard_normal((1, n, dim)), "bf16")
    qx = oa.round16(np.full((20, 2, dim), 2.0 ** 40), "bf16")
    k = oa.round16(np.full((1, n, dim), size / 2.0 ** 46), "bf16")
    s = store(q, "bf16", k, v, qx, dim, 16)
    got = down(_run(q, s, "bf16", 2, scale=1.0, hint=hint))
    val = oa.dequantize(*(a[0] for a in s["parts"][1]), dim)
    assert np.all(got >= val.min(0) * (1 - 2.0 ** -7)) and np.all(got <= val.max(0) * (1 + 2.0 ** -7))


@KERNELS
@pytest.mark.parametrize("dim,group", [(64, 64), (128, 32), (256, 64)])
def test_values_at_the_end_of_the_range(q, dim, group, hint):
    # one visible token: its value, up to the largest that bf16 holds
    say(f"case attention largest values D={dim} G={group} hint={hint}")
    for size in (1e38, 1.8e38, 3.3e38, -2.5e38):
        v = oa.round16(np.full((1, 1, dim), size), "bf16")
        s = store(q, "bf16", np.ones((1, 1, dim)), v, np.ones((1, 2, dim)), group, 16)
        got = down(_run(q, s, "bf16", 2, hint=hint))
        assert np.all(np.abs(got / v[0, 0] - 1) <= 2.0 ** -8), size
