"""The attention operators at the ends of their arguments' ranges, against the 64-bit oracle."""
import numpy as np
import pytest

from gpu_cases import say
from test_gpu_attention import _check, _run, _sequences, up
from test_gpu_attention_plans import scale_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_qgemm_amd as lib
    return lib


# kind, query lengths, context lengths, q_heads, kv_heads, dim, group, page
WIDE = [("f16", [700], [700], 4, 1, 64, 64, 16), ("bf16", [70, 3], [2100, 40], 1, 1, 128, 32, 48),
        ("f16", [200, 30], [100, 0], 2, 1, 128, 64, 16), ("bf16", [1, 5, 2], [900, 2, 64], 8, 2, 64, 32, 16)]


@pytest.mark.parametrize("hint", [0, 1, 2])
@pytest.mark.parametrize("case", range(len(WIDE)))
def test_windows_wider_than_any_context(q, case, hint):
    # windows up to the type's largest hide nothing, also where a sequence has more queries than tokens
    kind, qlens, klens, hq, hk, dim, group, page = WIDE[case]
    say(f"case attention wide windows {WIDE[case]} hint={hint}")
    s = _sequences(q, kind, qlens, klens, hq, hk, dim, group, page, 400 + case)
    outs = [_run(q, s, kind, hq, True, w, hint=hint) for w in (2 ** 31 - 1, 2 ** 31 - 200, 2 ** 30)]
    _check(s, outs[0], kind, hq, True, 0, scale_of(dim))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("hint,total,ratio", [(1, 300, 4), (2, 300, 4), (1, 3, 2), (0, 1000, 4)])
def test_starts_that_claim_more_rows_than_there_are_write_nothing(q, hint, total, ratio):
    # no output, no byte behind the workspace, and the workspace is ready for the next call; starts that decrease
    # without that own no rows there
    say(f"case attention starts that claim too much hint={hint} total={total}")
    s = _sequences(q, "f16", [total, 0, 0, 0], [1200, 0, 0, 0], 2 * ratio, 2, 64, 64, 16, 410)
    s["table"] = s["table"][:1].repeat(4, 1)
    s["lens"].fill_(1200)
    p = q.attention_problem(s["c"], 4, total, 2 * ratio, total, s["max_pages"], kernel_hint=hint)
    n = q.attention_workspace_bytes(p)
    if total > 3 and hint == 2:
        assert "splits=1" not in q.attention_describe(p).split()
    guarded = torch.zeros(n + 4096, dtype=torch.uint8, device="cuda")
    guarded[n:] = 0x5A
    qx = up(s["q"], "f16")

    def call(starts, ws):
        out = torch.full_like(qx, 7.0)
        q.attention(p, qx, s["data"], s["table"], s["lens"], torch.tensor(starts, dtype=torch.int32, device="cuda"), out, ws)
        torch.cuda.synchronize()
        assert (guarded[n:] == 0x5A).all(), starts
        return out

    good = call([0, total, total, total, total], q.alloc_attention_workspace(p))
    for starts in ([0, total, 0, total, 0], [0, total, 0, total, total], [0, total, 1, total, total]):
        assert (call(starts, guarded[:n]) == 7).all(), starts
        assert torch.equal(call([0, total, total, total, total], guarded[:n]), good), starts
    part = call([0, 2, 2, 2, 2], guarded[:n])
    for starts, want in (([0, total, 0, 0, 0], good), ([total, 0, total, total, total], good), ([0, 2, 1, 1, 0], part), ([0, 2, 0, 0, -5], part)):
        assert torch.equal(call(starts, guarded[:n]), want), starts
    assert (part[2:] == 7).all() and not (part[:2] == 7).all(-1).any()


def test_short_contexts_in_very_wide_tables(q):
    # one token each over tables of 4 million slots: more units than the rows kernel numbers, so the tiles kernel,
    # against the rows kernel over a narrow table
    say("case attention 1024 requests, tables of 2^22 slots")
    batch, hk, dim, page, wide = 1024, 32, 64, 16, 1 << 18
    g = torch.Generator(device="cuda").manual_seed(70)
    c = q.cache(4, page, hk, dim, q.DT_BF16)
    data = q.alloc_cache(c)
    k, v = (torch.randn(64, hk, dim, generator=g, device="cuda").bfloat16() for _ in "kv")
    q.cache_write(c, data, k, v, torch.arange(64, device="cuda"))
    qx = torch.randn(batch, hk, dim, generator=g, device="cuda").bfloat16()
    lens = (torch.arange(batch, device="cuda") * 7 % 65).int()
    starts = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    outs = []
    for columns, kind in ((wide, "tiles"), (4, "rows")):
        p = q.attention_problem(c, batch, batch, hk, 1, columns)
        assert q.attention_describe(p).startswith(kind)
        table = torch.zeros(batch, columns, dtype=torch.int32, device="cuda")
        table[:, :4] = torch.arange(4, dtype=torch.int32, device="cuda")
        out = torch.full_like(qx, 7.0)
        q.attention(p, qx, data, table, lens, starts, out, q.alloc_attention_workspace(p))
        outs.append(out.float())
        del table
    assert not outs[0][lens == 0].any() and not outs[1][lens == 0].any()
    # each within a rounding to bf16 and to fp16 weights of the values' mean
    assert (outs[0] - outs[1]).abs().max() <= 2.0 ** -8 * 2 * outs[1].abs().max() + 2.0 ** -10 * v.float().abs().max()


def test_pinned_lengths(q):
    # small arrays in pinned memory are read by the kernels where they lie
    say("case attention pinned lengths and starts")
    s = _sequences(q, "f16", [1, 3], [100, 70], 4, 2, 128, 128, 16, 420)
    want = _run(q, s, "f16", 4)
    held = dict(s, lens=s["lens"].cpu().pin_memory(), starts=s["starts"].cpu().pin_memory())
    assert torch.equal(_run(q, held, "f16", 4), want)
    with pytest.raises(ValueError, match="seq_lens must be on the GPU"):
        _run(q, dict(s, lens=s["lens"].cpu()), "f16", 4)
