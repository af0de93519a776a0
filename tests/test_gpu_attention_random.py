"""Seeded random attention problems through both kernels, every element against the 64-bit oracle: lengths, head
counts, groups, pages, masks and magnitudes drawn together."""
import numpy as np
import pytest

from gpu_cases import say
from oracle import attention as oa
from test_gpu_attention import _run, down, dt, up

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FLOOR = {1: 2.0 ** -31, 2: 2.0 ** -29}


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_qgemm_amd as lib
    return lib


def problem(g):
    dim = int(g.choice([64, 128, 128, 256]))
    ng = int(g.choice([1, 2] if dim == 64 else [1, 2, 4]))
    hk, ratio, page = int(g.choice([1, 2, 3])), int(g.choice([1, 1, 2, 3, 4, 7, 16])), 16 * int(g.choice([1, 1, 2, 3, 5, 16]))
    batch = int(g.integers(1, 6))
    longest = int(g.choice([1, 1, 5, 40, 130]))
    qlens = [int(g.integers(0, longest + 1)) for _ in range(batch)]
    qlens[int(g.integers(batch))] = longest
    klens = [max(0, n + int(g.choice([-20, 0, 0, 1, 60, 700, 2000]))) for n in qlens]
    causal = bool(g.random() < 0.8)
    window = int(g.choice([0, 0, 0, 1, 17, 300, 2 ** 31 - 1])) if causal else 0
    return dict(kind=str(g.choice(["f16", "bf16"])), dim=dim, group=dim // ng, hk=hk, hq=hk * ratio, page=page, qlens=qlens, klens=klens,
                causal=causal, window=window, spread=float(g.choice([0.3, 1.0, 4.0])), apart=int(g.choice([0, 0, 3])))


def build(q, c, g):
    kind, dim, page, hk, ng = c["kind"], c["dim"], c["page"], c["hk"], c["dim"] // c["group"]
    need = [-(-k // page) for k in c["klens"]]
    pages = sum(need) + 2
    order, columns = g.permutation(pages).astype(np.int32), max(max(need), 1) + 1
    table = np.full((len(need), columns), 1 << 30, np.int32)
    cache = q.cache(pages, page, hk, dim, dt(q, kind), group_size=c["group"])
    # NaN parameters wherever nothing is written
    data = torch.full((q.cache_bytes(cache),), 255, dtype=torch.uint8, device="cuda")
    at, parts = 0, []
    for b, k in enumerate(c["klens"]):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        x = [g.standard_normal((hk, k, dim)) * (0.5 + g.random(dim)) + g.standard_normal(dim) for _ in "kv"]
        x[1] = x[1] * np.repeat(2.0 ** (c["apart"] * g.permutation(ng)), c["group"]) * np.exp(0.5 * g.standard_normal((1, k, 1)))
        x = [oa.round16(a, kind) for a in x]
        if k:
            t = np.arange(k)
            slots = table[b, t // page].astype(np.int64) * page + t % page
            q.cache_write(cache, data, *(up(a.swapaxes(0, 1), kind) for a in x), torch.from_numpy(slots).cuda())
        parts.append([oa.quantize(a, c["group"], kind) for a in x])
    starts = np.concatenate(([0], np.cumsum(c["qlens"]))).astype(np.int32)
    qx = oa.round16(g.standard_normal((starts[-1], c["hq"], dim)) * c["spread"] * 2.0 ** g.integers(-3, 4, (1, c["hq"], 1)), kind)
    return dict(c=cache, data=data, table=torch.from_numpy(table).cuda(), q=qx, parts=parts, max_pages=columns, qlens=c["qlens"],
                klens=c["klens"], lens=torch.tensor(c["klens"], dtype=torch.int32, device="cuda"), starts=torch.from_numpy(starts).cuda())


@pytest.mark.parametrize("seed", range(60))
def test_random_problems(q, seed):
    g = np.random.default_rng([80, seed])
    c = problem(g)
    s, kind, group, scale = build(q, c, g), c["kind"], c["group"], np.float64(np.float32(c["dim"] ** -0.5))
    for hint in (1, 2):
        say(f"case attention random {seed} hint={hint} {c}")
        got, at, worst = down(_run(q, s, kind, c["hq"], c["causal"], c["window"], hint=hint, extra=8 * (seed % 2))), 0, 0.0
        for b, (n, k) in enumerate(zip(c["qlens"], c["klens"])):
            for h in range(c["hq"] if n else 0):
                (kc, ks, kz), (vc, vs, vz) = [[a[h * c["hk"] // c["hq"]] for a in part] for part in s["parts"][b]]
                val, qx = oa.dequantize(vc, vs, vz, group), s["q"][at:at + n, h]
                want, w = oa.attention(qx, oa.dequantize(kc, ks, kz, group), val, k, c["causal"], c["window"], scale)
                off = np.abs(got[at:at + n, h] - want)
                if not k:
                    assert not got[at:at + n, h].any()
                    continue
                bound = oa.attention_weight_bound(qx, w, val, want, ks, kz, vs, vz, group, scale, kind, FLOOR[hint],
                                                  hint == 2 and kind == "bf16")
                worst = max(worst, float(np.max(off / np.maximum(bound, 1e-300))))
                assert np.all(off <= bound), (hint, b, h, float(np.max(off / np.maximum(bound, 1e-300))))
            at += n
        say(f"  largest error / bound {worst:.3f}")
