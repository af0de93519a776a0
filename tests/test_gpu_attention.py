"""The attention operators on the GPU, every element against the 64-bit oracle.

Head norm and rotation and attention are held to error bounds derived from their number formats
(oracle/attention.py); the cache's codes and parameters must be the oracle's bytes exactly.  The
cases sit where such kernels go wrong: one token, lengths around the tile and page sizes, sequences
of length 0 and without queries, queries before the first token, windows, NaN and infinities in
slots that no query sees, odd head ratios, token strides, indices out of range, buffers past 4 GiB,
other streams, graph replays."""
import numpy as np
import pytest

from gpu_cases import say
from oracle import attention as oa

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

T16 = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_qgemm_amd as lib
    return lib


def dt(q, kind):
    return q.DT_F16 if kind == "f16" else q.DT_BF16


def up(x, kind):
    """float64 values of the type -> a device tensor."""
    return torch.from_numpy(np.ascontiguousarray(oa.bits16(x, kind).view(np.int16))).view(T16[kind]).cuda()


def down(t):
    return t.float().cpu().numpy().astype(np.float64)


def same_bits(a, b):
    """Equal bit for bit, NaN included."""
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def strided(x, kind, extra):
    """The rows of x [T, H, D] inside a wider buffer (extra elements a token), NaN around them."""
    t, h, d = x.shape
    wide = torch.full((t, h * d + extra), float("nan"), dtype=T16[kind], device="cuda")
    wide[:, :h * d] = up(x, kind).reshape(t, h * d)
    return wide[:, :h * d].unflatten(1, (h, d))


# ============================================================================= norm and rotation
ROPE = [  # kind, tokens, q_heads, kv_heads, dim, rot, interleaved, norm, weights, extra
    ("f16", 1, 1, 1, 64, 64, False, True, True, 0), ("bf16", 3, 5, 1, 64, 32, True, True, True, 8),
    ("f16", 7, 32, 8, 128, 128, False, True, True, 0), ("bf16", 130, 40, 8, 128, 64, True, True, True, 1024),
    ("bf16", 2, 3, 2, 256, 256, False, True, False, 16), ("f16", 5, 2, 7, 256, 128, True, True, True, 0),
    ("f16", 9, 4, 0, 128, 8, False, True, True, 0), ("bf16", 9, 0, 4, 128, 120, False, True, True, 24),
    ("f16", 65, 6, 2, 64, 24, True, True, True, 8), ("bf16", 33, 12, 4, 128, 128, False, False, False, 0),
    ("f16", 4, 9, 3, 128, 0, False, True, True, 0), ("f16", 700, 17, 3, 128, 96, False, True, True, 0)]


@pytest.mark.parametrize("kind,tokens,hq,hk,dim,rot,inter,norm,weights,extra", ROPE)
def test_norm_rope(q, kind, tokens, hq, hk, dim, rot, inter, norm, weights, extra):
    say(f"case norm_rope {kind} T={tokens} heads={hq}/{hk} D={dim} rot={rot} inter={inter} norm={norm}")
    g = np.random.default_rng([1, tokens, hq, dim, rot])
    max_pos = 50
    x = [oa.round16(g.standard_normal((tokens, h, dim)) * 10.0 ** g.integers(-2, 3, (tokens, h, 1)), kind) for h in (hq, hk)]
    x[0][:1] = 0.0                                                    # a head of zeros
    w = [oa.round16(1 + 0.3 * g.standard_normal(dim), kind) if weights else None for _ in x]
    pos = g.integers(0, max_pos, tokens).astype(np.int32)
    pos[:2] = (-7, max_pos + 5)[:min(2, tokens)]                      # nearest row
    table = g.standard_normal((max_pos, max(rot, 1))).astype(np.float32)
    ins = [strided(a, kind, extra) if a.shape[1] else None for a in x]
    outs = [strided(np.full(a.shape, 7.0), kind, 2 * extra) if a.shape[1] else None for a in x]
    p = q.norm_rope_problem(tokens, hq, hk, dim, dt(q, kind), rot_dim=rot, max_pos=max_pos, interleaved=inter, norm=norm, eps=1e-5)
    args = [None if a is None else up(a, kind) for a in w] + [torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda()]
    q.qk_norm_rope(p, *ins, *args, *outs)
    q.qk_norm_rope(p, *ins, *args, *ins)                              # in place: the same bits
    for a, b, i, o in zip(x, w, ins, outs):
        if o is None:
            continue
        want, mag = oa.norm_rope(a, b, pos, table, rot, inter, norm, 1e-5)
        off = np.abs(down(o) - want)
        assert np.all(off <= oa.norm_rope_bound(want, mag, dim, kind)), off.max()
        assert torch.equal(i, o)
        if extra:                                                     # what lies between the tokens stays
            assert torch.isnan(o.as_strided((tokens, 2 * extra), (o.stride(0), 1), o.shape[1] * dim)).all()


def test_norm_rope_keeps_non_finite_rows_apart(q):
    say("case norm_rope non-finite rows")
    x = np.ones((3, 4, 128))
    x[1, 2, 5], x[2, 0, 0] = np.nan, np.inf
    t = up(x, "f16")
    out, k = torch.empty_like(t), torch.empty(3, 0, 128, dtype=torch.float16)
    p = q.norm_rope_problem(3, 4, 0, 128, rot_dim=0)
    q.qk_norm_rope(p, t, None, None, None, None, None, out, None)
    bad = ~torch.isfinite(out).all(-1).cpu()
    assert bad.nonzero().tolist() == [[1, 2], [2, 0]] and k.numel() == 0


# ============================================================================= the cache
CACHE = [  # kind, tokens, kv_heads, dim, group, page, pages, extra
    ("f16", 1, 1, 64, 64, 16, 1, 0), ("bf16", 7, 3, 64, 32, 48, 4, 8), ("f16", 64, 8, 128, 128, 64, 3, 0),
    ("bf16", 65, 2, 128, 64, 16, 9, 256), ("f16", 130, 5, 128, 32, 32, 6, 64), ("bf16", 33, 1, 256, 256, 16, 4, 0),
    ("f16", 18, 2, 256, 128, 80, 2, 16), ("bf16", 5, 4, 256, 64, 128, 1, 0)]


def _host_cache(g, pages, heads, page, dim, group, kind):
    """Values, codes and the buffer's bytes of a whole cache."""
    x = [oa.round16(g.standard_normal((pages, heads, page, dim)) * 2 + g.standard_normal(dim), kind) for _ in "kv"]
    parts = [oa.quantize(a, group, kind) for a in x]
    data = np.stack([oa.pack_block(*(a[i, h] for a in parts[0]), *(a[i, h] for a in parts[1]), kind)
                     for i in range(pages) for h in range(heads)]).reshape(-1)
    return x, parts, data


@pytest.mark.parametrize("kind,tokens,heads,dim,group,page,pages,extra", CACHE)
@pytest.mark.parametrize("order", ["scattered", "in order"])
def test_cache_write_and_read(q, kind, tokens, heads, dim, group, page, pages, extra, order):
    say(f"case cache {kind} T={tokens} H={heads} D={dim} G={group} P={page} {order}")
    g = np.random.default_rng([2, tokens, dim, group, page])
    slots = g.permutation(pages * page)[:tokens] if order == "scattered" else np.arange(tokens) + (pages * page - tokens) // 2
    tokens = len(slots)
    x = [oa.round16(g.standard_normal((tokens, heads, dim)) * 10.0 ** g.integers(-4, 4, (tokens, heads, 1)), kind) for _ in "kv"]
    x[0][0, 0, :] = 1.5                                                # a constant head
    x[1][-1, -1, :group] = np.arange(group) % 16                       # exact codes
    x[0][-1, 0, 0] = np.nan
    x[1][0, 0, dim - 1] = np.inf
    c = q.cache(pages, page, heads, dim, dt(q, kind), group_size=group)
    before = g.integers(0, 256, q.cache_bytes(c)).astype(np.uint8)
    data = torch.from_numpy(before).cuda()
    st = torch.from_numpy(slots.astype(np.int64)).cuda()
    q.cache_write(c, data, strided(x[0], kind, extra), strided(x[1], kind, 2 * extra), st)
    parts = [oa.quantize(a, group, kind) for a in x]
    # expected bytes: the written tokens' nibbles and parameters, everything else as it was
    got = data.cpu().numpy().reshape(pages, heads, -1)
    want = before.reshape(pages, heads, -1).copy()
    ones = np.full((page, dim), 15, np.uint8)
    par = np.zeros((page, dim // group))
    for n, s in enumerate(slots):
        pg, t = divmod(int(s), page)
        only = np.zeros((page, dim), np.uint8)
        only[t] = 15
        mask = oa.pack_block(only, par, par, only, par, par, kind)
        for side in (0, 1):
            at = page * dim + side * page * 4 * (dim // group)
            m = mask[at:at + page * 4 * (dim // group)].reshape(-1, page, 4)
            m[:, t] = 255
        for h in range(heads):
            full = []
            for codes, sc, z in parts:
                cc, ss, zz = np.zeros((page, dim), np.uint8), par.copy(), par.copy()
                cc[t], ss[t], zz[t] = codes[n, h], sc[n, h], z[n, h]
                full += [cc, ss, zz]
            new = oa.pack_block(*full, kind)
            want[pg, h] = want[pg, h] & ~mask | new & mask
    # NaN parameters: any NaN will do; compare them as NaN
    gp, wp = (v[:, :, page * dim:].copy().view(np.uint16) for v in (got, want))
    both_nan = np.isnan(oa.from_bits16(gp, kind)) & np.isnan(oa.from_bits16(wp, kind))
    assert np.array_equal(got[:, :, :page * dim], want[:, :, :page * dim])
    assert np.array_equal(np.where(both_nan, 0, gp), np.where(both_nan, 0, wp))
    assert ones.any()
    # read back: the values, rounded once; -1 and slots past the end read as zeros
    ask = np.concatenate((slots, [-1, pages * page, -(1 << 40), 1 << 40])).astype(np.int64)
    outs = [torch.full((len(ask), heads, dim), 3.0, dtype=T16[kind], device="cuda") for _ in "kv"]
    q.cache_read(c, data, torch.from_numpy(ask).cuda(), *outs)
    for o, (codes, sc, z) in zip(outs, parts):
        v = oa.dequantize(codes, sc, z, group)
        near = np.abs(down(o[:tokens]) - v)
        tiny = 2.0 ** -25 if kind == "f16" else 0.0
        bound = oa.UNIT[kind] * np.abs(v) + 2.0 ** -23 * np.abs(v) + tiny
        assert np.array_equal(np.isnan(down(o[:tokens])), np.isnan(v))
        assert np.all((near <= bound) | np.isnan(v))
        assert not o[tokens:].any()


def test_cache_write_skips_slots_outside(q):
    say("case cache write with padding slots")
    c = q.cache(2, 16, 2, 128, q.DT_BF16, group_size=64)
    data = q.alloc_cache(c).fill_(0xAB)
    x = torch.randn(6, 2, 128, device="cuda").bfloat16()
    q.cache_write(c, data, x, x, torch.tensor([-1, 32, 1 << 50, -(1 << 50), 33, -2], device="cuda"))
    assert (data == 0xAB).all()
    q.cache_write(c, data, x, x, torch.tensor([-1, 31, 32, -1, 0, -1], device="cuda"))
    out = [torch.empty(2, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    q.cache_read(c, data, torch.tensor([31, 0], device="cuda"), *out)
    assert torch.allclose(out[0].float(), x[[1, 4]].float(), atol=0.25) and torch.equal(out[0], out[1])
    assert (data == 0xAB).any()


# ============================================================================= attention
def _sequences(q, kind, qlens, klens, hq, hk, dim, group, page, seed, spread=1.0, spare=3):
    """Random cache content for the sequences, pages in random order, NaN parameters and random codes
    wherever no token is."""
    g = np.random.default_rng([3, seed, dim, group, page, len(klens)])
    need = [-(-k // page) for k in klens]
    pages = sum(need) + spare
    order = g.permutation(pages).astype(np.int32)
    max_pages = max(max(need), 1) + 1
    table = np.full((len(klens), max_pages), -12345, np.int32)        # entries past the length are not read
    u8 = g.integers(0, 256, (pages, hk, oa.block_bytes(page, dim, group))).astype(np.uint8)
    nan = 0x7E00 if kind == "f16" else 0x7FC0
    u8[:, :, page * dim:] = np.full(u8[:, :, page * dim:].shape[-1] // 2, nan, np.uint16).view(np.uint8)
    seqs, at = [], 0
    for b, k in enumerate(klens):
        x = [oa.round16(g.standard_normal((hk, k, dim)) * (0.5 + g.random(dim)) + g.standard_normal(dim), kind) for _ in "kv"]
        parts = [oa.quantize(a, group, kind) for a in x]
        for j in range(need[b]):
            pg = order[at]
            at += 1
            table[b, j] = pg
            n = min(page, k - j * page)
            for h in range(hk):
                full = []
                for side, (codes, sc, z) in enumerate(parts):
                    cc = g.integers(0, 16, (page, dim)).astype(np.uint8)
                    ss, zz = np.full((page, dim // group), np.nan), np.full((page, dim // group), np.nan)
                    cc[:n], ss[:n], zz[:n] = (a[h, j * page:j * page + n] for a in (codes, sc, z))
                    full += [cc, ss, zz]
                u8[pg, h] = oa.pack_block(*full, kind)
        seqs.append(parts)
    starts = np.concatenate(([0], np.cumsum(qlens))).astype(np.int32)
    qx = oa.round16(g.standard_normal((starts[-1], hq, dim)) * spread, kind)
    c = q.cache(pages, page, hk, dim, dt(q, kind), group_size=group)
    return dict(c=c, data=torch.from_numpy(u8.reshape(-1)).cuda(), table=torch.from_numpy(table).cuda(), q=qx, seqs=seqs,
                lens=torch.tensor(klens, dtype=torch.int32, device="cuda"), starts=torch.from_numpy(starts).cuda(),
                qlens=qlens, klens=klens, max_pages=max_pages, group=group)


def _run(q, s, kind, hq, causal=True, window=0, scale=None, hint=0, extra=0, out_extra=0, max_q=None, stream=None):
    total = s["q"].shape[0]
    p = q.attention_problem(s["c"], len(s["klens"]), total, hq, max_q or max(s["qlens"]), s["max_pages"], causal=causal,
                            window=window, scale=scale, kernel_hint=hint)
    ws = q.alloc_attention_workspace(p)
    if ws is not None:                                                # guard bytes behind the workspace
        n = ws.numel()
        ws = torch.cat((ws, torch.full((256,), 0x5A, dtype=torch.uint8, device="cuda")))
    out = strided(np.full(s["q"].shape, 7.0), kind, out_extra)
    qx = strided(s["q"], kind, extra)
    use = None if ws is None else ws[:n]
    for _ in range(2):                                                # the second call meets the first's workspace
        first = out.clone()
        q.attention(p, qx, s["data"], s["table"], s["lens"], s["starts"], out, use, stream=stream)
        torch.cuda.synchronize()
    assert same_bits(first, out), "two calls differ"
    if ws is not None:
        assert (ws[n:] == 0x5A).all()
    return out


def _check(s, out, kind, hq, causal, window, scale):
    got, at = down(out), 0
    ratio = hq // s["c"].kv_heads
    worst = 0.0
    for b, (n, k) in enumerate(zip(s["qlens"], s["klens"])):
        for h in range(hq if n else 0):
            (kc, ks, kz), (vc, vs, vz) = [[a[h // ratio] for a in part] for part in s["seqs"][b]]
            kv, vv = oa.dequantize(kc, ks, kz, s["group"]), oa.dequantize(vc, vs, vz, s["group"])
            qx = s["q"][at:at + n, h]
            want, w = oa.attention(qx, kv, vv, k, causal, window, scale)
            bound = oa.attention_bound(qx, w, want, ks, kz, vs, vz, k, s["group"], scale, kind) if k else np.zeros((n, 1))
            off = np.abs(got[at:at + n, h] - want)
            bad = np.isnan(want)                                       # a query that sees a NaN token
            assert np.array_equal(np.isnan(got[at:at + n, h]), bad)
            off, bound = np.where(bad, 0, off), np.where(bad, 0, bound)
            assert np.all(off <= bound), (b, h, float(np.max(off - bound)))
            empty = ~w.any(1)
            assert not got[at:at + n, h][empty].any()
            worst = max(worst, float(np.max(off / np.maximum(bound, 1e-30), initial=0)))
        at += n
    say(f"  largest error / bound {worst:.3f}")


# kind, query lengths, context lengths, q_heads, kv_heads, dim, group, page, causal, window
ATTN = [
    ("f16", [1], [1], 1, 1, 64, 64, 16, True, 0),
    ("bf16", [1], [1], 8, 1, 128, 128, 16, True, 0),
    ("f16", [1, 1, 1, 1, 1], [15, 16, 17, 31, 33], 4, 1, 128, 128, 16, True, 0),
    ("bf16", [1, 1, 1, 1], [63, 64, 65, 129], 5, 1, 128, 32, 48, True, 0),
    ("f16", [1, 1, 1], [0, 1, 300], 8, 2, 128, 64, 32, True, 0),              # nothing to see: zeros
    ("f16", [1, 0, 1, 0], [257, 40, 0, 0], 6, 3, 64, 32, 16, True, 0),        # no queries, no tokens
    ("bf16", [1] * 9, [700, 1, 64, 513, 1000, 2, 90, 255, 256], 16, 2, 128, 128, 64, True, 0),
    ("f16", [1, 1], [1999, 1024], 7, 1, 256, 64, 16, True, 0),
    ("bf16", [1, 1], [511, 800], 2, 2, 256, 256, 32, True, 0),
    ("f16", [1, 1], [128, 130], 64, 4, 64, 64, 16, True, 0),                  # 16 rows
    ("bf16", [1], [100], 96, 4, 64, 32, 16, True, 0),                         # 24 rows
    ("f16", [1], [333], 35, 1, 128, 128, 16, True, 0),                        # 35 rows
    ("bf16", [1], [210], 71, 1, 64, 64, 80, True, 0),                         # 71 rows of one token
    ("f16", [5, 3, 1], [500, 3, 64], 8, 2, 128, 128, 16, True, 0),            # drafts
    ("bf16", [8, 2], [77, 2], 4, 4, 64, 32, 16, True, 0),
    ("f16", [4, 9, 2], [2, 0, 5], 4, 2, 128, 64, 16, True, 0),                # queries before the first token
    ("f16", [3, 1], [400, 90], 4, 1, 128, 32, 16, True, 1),                   # windows
    ("bf16", [2, 2], [700, 30], 8, 1, 128, 128, 64, True, 100),
    ("f16", [1, 1], [650, 64], 8, 2, 64, 64, 32, True, 64),
    ("f16", [2, 5], [40, 300], 4, 2, 128, 128, 16, False, 0),                 # every query sees everything
    ("bf16", [40, 1, 17], [40, 200, 90], 8, 2, 128, 128, 16, True, 0),        # prompts and chunks
    ("f16", [129], [129], 4, 4, 64, 64, 16, True, 0),
    ("bf16", [100, 60], [333, 60], 6, 1, 128, 32, 48, True, 0),
    ("f16", [70, 33], [90, 500], 3, 1, 256, 128, 16, True, 0),
    ("bf16", [65, 20], [130, 64], 4, 2, 256, 64, 32, True, 50),
    ("f16", [90, 3], [60, 3], 4, 2, 128, 64, 64, True, 0),                    # rows without a token among others
    ("f16", [66], [290], 5, 1, 128, 128, 16, False, 0),
    ("bf16", [260], [260], 2, 1, 64, 32, 16, True, 37),
]


@pytest.mark.parametrize("hint", [0, 1, 2])
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention(q, case, hint):
    kind, qlens, klens, hq, hk, dim, group, page, causal, window = ATTN[case]
    say(f"case attention {case} hint={hint} {ATTN[case]}")
    s = _sequences(q, kind, qlens, klens, hq, hk, dim, group, page, case)
    out = _run(q, s, kind, hq, causal, window, hint=hint, extra=8 * (case % 3), out_extra=16 * (case % 2))
    _check(s, out, kind, hq, causal, window, np.float64(np.float32(dim ** -0.5)))


@pytest.mark.parametrize("hint", [1, 2])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_attention_scores_far_apart(q, kind, hint):
    # scores of hundreds, rising and falling along the context: the running maximum moves often; a
    # negative and a zero scale; value groups whose spread differs by orders of magnitude
    for scale, qlens, klens in ((1.0, [2, 40], [700, 300]), (-3.0, [1, 20], [500, 130]), (0.0, [3], [90])):
        say(f"case attention far-apart {kind} hint={hint} scale={scale}")
        s = _sequences(q, kind, qlens, klens, 8, 2, 128, 64, 16, 77, spread=3.0)
        out = _run(q, s, kind, 8, scale=scale, hint=hint)
        _check(s, out, kind, 8, True, 0, scale)


@pytest.mark.parametrize("hint", [1, 2])
@pytest.mark.parametrize("kind,low,high", [("f16", 1e-4, 3e4), ("bf16", 1e-30, 1e30), ("f16", 1e-7, 1e-5), ("bf16", 1e-38, 1e-36)])
def test_attention_value_magnitudes(q, kind, low, high, hint):
    # value scales over the whole range of the type, tiny and huge tokens side by side
    say(f"case attention magnitudes {kind} {low} {high} hint={hint}")
    g = np.random.default_rng([4, hint])
    n, dim, page = 200, 128, 32
    pages = -(-n // page)
    mag = np.exp(g.uniform(np.log(low), np.log(high), (pages, 1, page, 1)))
    mag = np.sort(mag.reshape(-1))[::1 if hint == 1 else -1].reshape(mag.shape)
    k = oa.round16(g.standard_normal((pages, 1, page, dim)), kind)
    v = oa.round16(g.standard_normal((pages, 1, page, dim)) * mag, kind)
    parts = [oa.quantize(x, dim, kind) for x in (k, v)]
    data = np.stack([oa.pack_block(*(a[i, 0] for a in parts[0]), *(a[i, 0] for a in parts[1]), kind) for i in range(pages)])
    c = q.cache(pages, page, 1, dim, dt(q, kind))
    qx = oa.round16(g.standard_normal((40, 2, dim)) * 0.5, kind)
    flat = [[a.reshape(1, pages * page, -1)[:, :n] for a in part] for part in parts]
    s = dict(c=c, data=torch.from_numpy(data.reshape(-1)).cuda(), table=torch.arange(pages, dtype=torch.int32, device="cuda"),
             q=qx, seqs=[flat], lens=torch.tensor([n], dtype=torch.int32, device="cuda"),
             starts=torch.tensor([0, 40], dtype=torch.int32, device="cuda"), qlens=[40], klens=[n], max_pages=pages, group=dim)
    out = _run(q, s, kind, 2, hint=hint)
    _check(s, out, kind, 2, True, 0, np.float64(np.float32(dim ** -0.5)))


@pytest.mark.parametrize("hint", [1, 2])
def test_attention_query_magnitudes(q, hint):
    # heads of very different size next to each other, up to the type's largest, with scores in range
    for kind, top in (("f16", 6e4), ("bf16", 1e30)):
        say(f"case attention query magnitudes {kind} hint={hint}")
        s = _sequences(q, kind, [6], [150], 8, 1, 128, 128, 16, 5)
        s["q"] = oa.round16(s["q"] * (top / 4), kind)
        scale = float(np.float32(0.1 / top))
        out = _run(q, s, kind, 8, scale=scale, hint=hint)
        _check(s, out, kind, 8, True, 0, scale)


@pytest.mark.parametrize("hint", [1, 2])
def test_attention_nan_and_infinity_stay_where_they_are_seen(q, hint):
    # a NaN token late in the context: queries before it are clean, later ones are NaN; a NaN query
    # row spoils itself only, and so does an infinite one
    say(f"case attention NaN hint={hint}")
    s = _sequences(q, "f16", [50, 2], [50, 20], 4, 2, 128, 128, 16, 6)
    clean = _run(q, s, "f16", 4, hint=hint)
    kv = up(np.full((1, 2, 128), np.nan), "f16")
    page = int(s["table"][0, 2])                                      # token 40 of sequence 0
    q.cache_write(s["c"], s["data"], kv, kv, torch.tensor([page * 16 + 8], device="cuda"))
    dirty = _run(q, s, "f16", 4, hint=hint)
    assert torch.equal(dirty[:40], clean[:40]) and torch.equal(dirty[50:], clean[50:])
    assert torch.isnan(dirty[40:50]).all()
    s["q"] = s["q"].copy()
    s["q"][7, 1, 3], s["q"][9, 2, 0] = np.nan, np.inf
    spoilt = _run(q, s, "f16", 4, hint=hint)
    keep = torch.ones(40, 4, dtype=torch.bool, device="cuda")
    keep[7, 1] = keep[9, 2] = False
    assert torch.equal(spoilt[:40][keep], clean[:40][keep]) and torch.isnan(spoilt[7, 1]).all()


@pytest.mark.parametrize("hint", [1, 2])
def test_attention_indices_out_of_range_stay_in_bounds(q, hint):
    # wrong lengths, starts and pages give some result, never an access outside the buffers; the
    # sequences that are well described are not touched by it
    say(f"case attention bounds hint={hint}")
    s = _sequences(q, "f16", [3, 3, 3], [60, 70, 40], 4, 2, 128, 128, 16, 8)
    good = _run(q, s, "f16", 4, hint=hint)
    s["table"][1, 0], s["table"][1, 1] = 1 << 30, -5
    s["lens"][2] = 1 << 30
    bad = _run(q, s, "f16", 4, hint=hint)
    assert torch.equal(bad[:3], good[:3])
    s["lens"][2] = -4
    none = _run(q, s, "f16", 4, hint=hint)
    assert not none[6:].any() and torch.equal(none[:3], good[:3])
    s["starts"][3], s["starts"][2] = 1 << 30, 6
    far = _run(q, s, "f16", 4, hint=hint)
    assert torch.equal(far[:3], good[:3])


@pytest.mark.parametrize("hint", [1, 2])
def test_attention_rows_of_no_sequence_keep_their_output(q, hint):
    say(f"case attention uncovered rows hint={hint}")
    s = _sequences(q, "bf16", [2, 3], [20, 30], 4, 2, 64, 64, 16, 9)
    s["starts"] = torch.tensor([1, 3, 4], dtype=torch.int32, device="cuda")
    out = _run(q, s, "bf16", 4, hint=hint)
    assert (out[0] == 7).all() and (out[4] == 7).all() and not (out[1:4] == 7).all(-1).any()


@pytest.mark.parametrize("hint", [1, 2])
def test_attention_past_four_gib(q, hint):
    # pages beyond 4 GiB of the buffer, written, read back and attended to there
    say(f"case attention past 4 GiB hint={hint}")
    page, hk, dim = 256, 8, 128
    pages = 17000
    c = q.cache(pages, page, hk, dim, q.DT_F16)                        # 4.7 GB
    assert q.cache_bytes(c) > (1 << 32) + (1 << 28)
    small = _sequences(q, "f16", [2, 20], [300, 700], 8, hk, dim, dim, page, 10, spare=0)
    data = torch.zeros(q.cache_bytes(c), dtype=torch.uint8, device="cuda")
    n = small["data"].numel()
    data[-n:] = small["data"]
    want = _run(q, small, "f16", 8, hint=hint)
    first = pages - n // (q.cache_bytes(c) // pages)
    big = dict(small, c=c, data=data, table=small["table"].clamp(min=0) + first)
    assert torch.equal(_run(q, big, "f16", 8, hint=hint), want)
    x = torch.randn(5, hk, dim, device="cuda").half()
    at = torch.tensor([pages * page - 1, (pages - 1) * page, 0, 16000 * page + 7, 1000 * page], device="cuda")
    q.cache_write(c, data, x, x, at)
    out = [torch.empty_like(x) for _ in "kv"]
    q.cache_read(c, data, at, *out)
    tight, loose = (q.cache(1, 16, hk, dim, q.DT_F16) for _ in "ab")
    d2, o2 = q.alloc_cache(tight), [torch.empty_like(x) for _ in "kv"]
    q.cache_write(tight, d2, x, x, torch.arange(5, device="cuda"))
    q.cache_read(loose, d2, torch.arange(5, device="cuda"), *o2)
    assert torch.equal(out[0], o2[0]) and torch.equal(out[1], o2[1])


def test_other_streams(q):
    # the calls run on the stream they are given, in its order
    say("case attention operators on a side stream")
    s = _sequences(q, "f16", [1, 1], [100, 700], 8, 2, 128, 128, 16, 11)
    want = _run(q, s, "f16", 8)
    p = q.attention_problem(s["c"], 2, 2, 8, 1, s["max_pages"])
    ws, out = q.alloc_attention_workspace(p), torch.zeros(2, 8, 128, dtype=torch.float16, device="cuda")
    qx = up(s["q"], "f16")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = torch.zeros_like(s["data"])
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(s["data"])
        q.attention(p, qx, late, s["table"], s["lens"], s["starts"], out, ws)          # torch's current stream
    side.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    torch.cuda.synchronize()
    q.attention(p, qx, late, s["table"], s["lens"], s["starts"], out, ws, stream=side)  # named
    side.synchronize()
    assert torch.equal(out, want)


def test_graph_replays_follow_the_lengths_in_device_memory(q):
    # one captured step (write a token, attend) replayed while lengths, slots and the token change
    say("case attention operators in a graph")
    hq, hk, dim, page = 8, 2, 128, 16
    s = _sequences(q, "bf16", [1, 1], [40, 70], hq, hk, dim, 64, page, 12)
    c, table = s["c"], s["table"].clamp(min=0)
    table[:, 4:] = 0
    k = torch.zeros(2, hk, dim, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    qx, out = up(s["q"], "bf16"), torch.zeros(2, hq, dim, dtype=torch.bfloat16, device="cuda")
    p = q.attention_problem(c, 2, 2, hq, 1, s["max_pages"])
    ws = q.alloc_attention_workspace(p)

    def step(o, w, data):
        q.cache_write(c, data, k, k, slots)
        q.attention(p, qx, data, table, lens, s["starts"], o, w)

    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(out, ws, s["data"])
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(out, ws, s["data"])
    for i in range(4):
        lens.copy_(torch.tensor([41 + i, 3 + 13 * i], dtype=torch.int32))
        k.copy_(torch.randn(2, hk, dim))
        slots.copy_(torch.stack([table[b, (int(lens[b]) - 1) // page].long() * page + (int(lens[b]) - 1) % page for b in (0, 1)]))
        out.fill_(9.0)
        torch.cuda.synchronize()
        before = s["data"].clone()
        g.replay()
        torch.cuda.synchronize()
        eager, w2 = torch.zeros_like(out), q.alloc_attention_workspace(p)
        step(eager, w2, before)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(before, s["data"])
