"""The 8-bit operators at the ends of their ranges: buffers whose offsets pass 32 bits, the longest K, the most rows."""
import numpy as np
import pytest

from gpu_cases import say
from test_gpu_w8a8 import F8, STEP, T16, U24, dt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_qgemm_amd as q
    yield q
    torch.cuda.empty_cache()


def codes(rows, k, seed):
    """Finite e4m3 codes of either sign and any size up to 15."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 256, (rows, k), generator=g, device="cuda", dtype=torch.uint8)
    return (c & 0x80 | (c & 0x7f) % 0x58).view(F8)


def scales(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(shape, generator=g, device="cuda") + 0.5


def check(q, m, n, k, gate, out, ins, y, tokens, columns):
    """Outputs at `tokens` x `columns` against 64 bits (rounded sums: as product_want in test_gpu_w8a8)."""
    a, sa, w, sw = ins
    def part(first, first_scale):
        rows = first + columns
        wv = w.view(torch.uint8)[rows].view(F8).double().unflatten(1, (-1, 128)) * sw[first_scale + columns // 128].double()[..., None]
        av = a.view(torch.uint8)[tokens].view(F8).double().unflatten(1, (-1, 128)) * sa[:, tokens].t().double()[..., None]
        wv, av = wv.flatten(1), av.flatten(1)
        return av @ wv.t().contiguous(), (176 + k // 64) * 2.0 ** -23 * (av.abs() @ wv.abs().t().contiguous())
    want, tol = part(0, 0)
    if gate:
        other, other_tol = part(n, -(-n // 128))
        act = want * torch.sigmoid(want)
        slope = 1.13 * tol + act.abs() * (12 * want.abs() + 8) * U24
        want, tol = act * other, slope * (other.abs() + other_tol) + act.abs() * other_tol + 2 * U24 * (act * other).abs()
    off = (y[tokens][:, columns].double() - want).abs()
    assert bool((off <= tol + STEP[out] * (want.abs() + tol)).all()), float((off - tol - STEP[out] * want.abs()).max())


@pytest.mark.parametrize("m,n,k,gate,out,hints", [
    (3, 266256, 16384, 0, "bf16", {}), (20, 133200, 16384, 1, "f32", dict(kernel_hint=1)), (70, 266256, 16384, 0, "f32", {}),
    (70, 133200, 16384, 1, "bf16", dict(split_hint=2)), (262213, 256, 16384, 0, "bf16", {}), (262213, 4112, 256, 0, "f32", {})])
def test_offsets_past_32_bits(q, m, n, k, gate, out, hints):
    """Weights, activations or outputs of more than 4 GiB; the first and last tokens and columns."""
    say(f"case large {m} {n} {k} {gate} {out} {hints}")
    parts = 2 if gate else 1
    ins = (codes(m, k, 1), scales(k // 128, m, seed=2), codes(parts * n, k, 3), scales(parts * -(-n // 128), k // 128, seed=4) * k ** -0.5 / 30)
    p = q.w8a8_problem(m, n, k, dt(q, out), gate=gate, **hints)
    assert max(m * k, parts * n * k, m * n * (4 if out == "f32" else 2)) > 2 ** 32
    y = torch.full((m, n), float("nan"), dtype=torch.float32 if out == "f32" else T16[out], device="cuda")
    q.w8a8_run(p, *ins, y, None, q.alloc_w8a8_workspace(p))
    torch.cuda.synchronize()
    pick = lambda n: torch.unique(torch.cat((torch.arange(min(n, 20)), n - 1 - torch.arange(min(n, 20)), torch.arange(0, n, max(1, n // 37))))).cuda()
    check(q, m, n, k, gate, out, ins, y, pick(m), pick(n))
    assert bool(torch.isfinite(y).all())


@pytest.mark.parametrize("hint", [0, 2])
@pytest.mark.parametrize("gate", [0, 1])
def test_longest_k(q, gate, hint):
    """Operands +-1 with scales of 1 and 2, and a common 2^-12: whole numbers up to 2^24 times it, so the sums are exact in any order."""
    m, n, k = 5, 32, 1 << 22
    say(f"case longest k {gate} {hint}")
    parts, g = 2 if gate else 1, torch.Generator(device="cuda").manual_seed(k + gate)
    two = lambda *s: torch.randint(0, 2, s, generator=g, device="cuda").float()
    a, w = 2 * two(m, k) - 1, 2 * two(parts * n, k) - 1
    sa, sw = 1 + two(k // 128, m), (1 + two(parts, k // 128)) * 2.0 ** -12
    p = q.w8a8_problem(m, n, k, q.DT_F32, gate=gate, kernel_hint=hint)
    y = torch.empty((m, n), device="cuda")
    q.w8a8_run(p, a.to(F8), sa, w.to(F8), sw, y, None, q.alloc_w8a8_workspace(p))
    torch.cuda.synchronize()
    blocks = torch.bmm(a.unflatten(1, (-1, 128)).transpose(0, 1).contiguous(), w.unflatten(1, (-1, 128)).permute(1, 2, 0).contiguous())
    sums = (blocks.double() * sa.double()[..., None] * sw.double().t().repeat_interleave(n, 1)[:, None]).sum(0)
    if not gate:
        assert torch.equal(y.double(), sums)
        return
    x, u = sums[:, :n], sums[:, n:]
    want = x * torch.sigmoid(x) * u
    assert bool(((y.double() - want).abs() <= (12 * x.abs() + 12) * U24 * want.abs()).all())


@pytest.mark.parametrize("tokens,dim,out", [(1 << 24, 8, "f16"), ((1 << 24) - 3, 128, "e4m3"), (70001, 32768, "f16")])
def test_add_norm_most_rows(q, tokens, dim, out):
    """2^24 rows fit one launch as long as a row is a wavefront's."""
    say(f"case add_norm {tokens} {dim} {out}")
    g = torch.Generator(device="cuda").manual_seed(dim)
    x = torch.randint(-32768, 32768, (tokens, dim), generator=g, device="cuda", dtype=torch.int16)
    x = (x.view(torch.uint8) & 0xbf).view(torch.float16)                       # finite, below 2
    y = torch.empty((tokens, dim), dtype=F8 if out == "e4m3" else torch.float16, device="cuda")
    s = torch.empty((dim // 128, tokens), device="cuda") if out == "e4m3" else None
    q.add_norm(q.add_norm_problem(tokens, dim, q.DT_F16, q.DT_FP8_E4M3 if s is not None else None, eps=1e-3), x, None, None, None, y, s)
    torch.cuda.synchronize()
    for at in (0, tokens // 2, tokens - 64):
        rows = x[at:at + 64].double()
        want = rows / torch.sqrt((rows * rows).mean(1, keepdim=True) + 1e-3)
        if s is None:
            # as norm_check in test_gpu_w8a8: the roundings of the sum and the root, then the output's (and that of a subnormal)
            tol = 32 * U24 * want.abs()
            assert bool(((y[at:at + 64].double() - want).abs() <= tol + 2.0 ** -11 * (want.abs() + tol) + 2.0 ** -25).all()), at
        else:
            scale = s[:, at:at + 64].double().t()
            assert bool(((scale * 448 / want.abs().unflatten(1, (-1, 128)).amax(-1) - 1).abs() <= 40 * U24).all()), at
            held = (y[at:at + 64].double().unflatten(1, (-1, 128)) * scale[..., None]).flatten(1)
            half = torch.maximum(want.abs() * 2.0 ** -4, scale.repeat_interleave(128, 1) * 2.0 ** -10)
            assert bool(((held - want).abs() <= half * (1 + 64 * U24) + 40 * U24 * want.abs()).all()), at
