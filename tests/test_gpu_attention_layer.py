"""The attention operators together, between two INT4 products: example_attention.py's layer for
prompts and decode steps, each operator against the 64-bit oracle on what the one before it gave,
and the captured decode step against the same calls one by one."""
import numpy as np
import pytest

from gpu_cases import say
from oracle import attention as oa
from oracle import quant, reference

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import example_attention
    return example_attention


def f64(t):
    return t.double().cpu().numpy()


def product_check(x, w, got):
    """fp16 result of an fp32 sum over K products of exact factors: one rounding, and K additions
    over the sum of magnitudes."""
    codes, sbits = quant.quantize_int4(w, 128)
    wdq = reference.dequant_int4(codes, sbits, 128).astype(np.float64)
    want, mag = x @ wdq.T, np.abs(x) @ np.abs(wdq).T
    off = np.abs(got - want)
    # the dequantized weight is rounded to fp16 as an operand: 2^-11 of each product
    assert np.all(off <= oa.UNIT["f16"] * np.abs(want) + 2.0 ** -25 + (2.0 ** -11 + x.shape[1] * 2.0 ** -24) * mag), off.max()


LAYERS = [  # width, q_heads, kv_heads, dim, group, page, rot, window
    (512, 4, 2, 64, 32, 16, 64, 0), (256, 8, 1, 128, 128, 48, 64, 0), (384, 3, 3, 128, 32, 32, 128, 20),
    (512, 4, 2, 256, 64, 16, 128, 0)]


def build(ex, shape, pages, seed):
    width, hq, hk, dim, group, page, rot, window = shape
    g = np.random.default_rng(seed)
    w = [(g.standard_normal(s, dtype=np.float32) * s[1] ** -0.5) for s in
         (((hq + 2 * hk) * dim, width), (width, hq * dim))]
    norm = [oa.round16(1 + 0.2 * g.standard_normal(dim), "f16") for _ in "qk"]
    layer = ex.AttentionLayer(*w, *(torch.from_numpy(n.astype(np.float16)).cuda() for n in norm), ex.rotation_table(rot, 200),
                              hq, hk, dim, pages, page, group, window)
    return layer, w, norm


@pytest.mark.parametrize("shape", LAYERS)
def test_layer_stage_by_stage(ex, shape):
    width, hq, hk, dim, group, page, rot, window = shape
    say(f"case attention layer {shape}")
    prompts, steps = [37, 1, 64, 5], 3
    each = -(-(max(prompts) + steps) // page)
    layer, w, norm = build(ex, shape, each * 4 + 1, [21, dim, group])
    g = np.random.default_rng([22, dim, group])
    table = torch.from_numpy(g.permutation(each * 4).astype(np.int32).reshape(4, each)).cuda()
    context = [[[], []] for _ in prompts]                     # the keys and values each request has stored
    lens = list(prompts)
    for step in range(1 + steps):
        q_lens = prompts if step == 0 else [1] * 4
        if step:
            lens = [n + 1 for n in lens]
        if step < 2:
            t = ex.Tokens(table, q_lens, prompts, page)
        if step:
            t.advance()
        assert t.lens.tolist() == lens
        x = torch.from_numpy(g.standard_normal((t.total, width)).astype(np.float16)).cuda()
        b = layer.plan(t)
        layer.project(b, x)
        product_check(f64(x), w[0], f64(b["qkv"]).reshape(t.total, -1))
        before = f64(b["qkv"])
        layer.rotate(b, t)
        after = f64(b["qkv"])
        assert np.array_equal(before[:, hq + hk:], after[:, hq + hk:])
        pos, rows = t.positions.cpu().numpy(), f64(layer.table)
        for part, weight in ((np.s_[:, :hq], norm[0]), (np.s_[:, hq:hq + hk], norm[1])):
            want, mag = oa.norm_rope(before[part], weight, pos, rows, rot, False)
            assert np.all(np.abs(after[part] - want) <= oa.norm_rope_bound(want, mag, dim, "f16"))
        layer.store(b, t)
        at = 0
        for seq, n in zip(context, q_lens):
            for side, first in ((0, hq), (1, hq + hk)):
                seq[side].append(after[at:at + n, first:first + hk])
            at += n
        layer.attend(b, t)
        heads, at = f64(b["heads"]), 0
        for i, (seq, n) in enumerate(zip(context, q_lens)):
            k, v = (oa.quantize(np.concatenate(s).transpose(1, 0, 2), group, "f16") for s in seq)
            for h in range(hq):
                (kc, ks, kz), (vc, vs, vz) = [[a[h * hk // hq] for a in s] for s in (k, v)]
                kv, vv = oa.dequantize(kc, ks, kz, group), oa.dequantize(vc, vs, vz, group)
                qx = after[at:at + n, h]
                want, wt = oa.attention(qx, kv, vv, lens[i], True, window, np.float64(np.float32(dim ** -0.5)))
                bound = oa.attention_bound(qx, wt, want, ks, kz, vs, vz, lens[i], group, dim ** -0.5, "f16")
                assert np.all(np.abs(heads[at:at + n, h] - want) <= bound), (step, i, h)
            at += n
        out = layer.output(b)
        product_check(heads.reshape(t.total, -1), w[1], f64(out))


@pytest.mark.parametrize("shape", LAYERS[:2])
def test_captured_decode_steps_equal_separate_calls(ex, shape):
    width, _, _, dim, group, page, _, _ = shape
    say(f"case attention layer graph {shape}")
    prompts = [20, 3, 47]
    each = 120 // page + 1
    layer, _, _ = build(ex, shape, each * 3, [23, dim])
    table = torch.arange(each * 3, dtype=torch.int32, device="cuda").view(3, each)
    torch.manual_seed(5)
    layer(torch.randn(sum(prompts), width, device="cuda").half(), ex.Tokens(table, prompts, prompts, page))
    start = layer.data.clone()
    inputs = torch.randn(6, 3, width, device="cuda").half()
    t = ex.Tokens(table, [1] * 3, prompts, page)
    want = []
    for x in inputs:
        t.advance()
        want.append(layer(x, t).clone())
    end, lens = layer.data.clone(), t.lens.clone()
    layer.data.copy_(start)
    t = ex.Tokens(table, [1] * 3, prompts, page)
    x = inputs[0].clone()
    graph, out = ex.capture(layer, x, t)
    for i in range(6):
        x.copy_(inputs[i])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), i
        assert torch.isfinite(out.float().sum())              # eager work between the replays
    assert torch.equal(layer.data, end) and torch.equal(t.lens, lens)
