"""The 8-bit operators on the GPU against their 64-bit definitions: the residual addition with RMS norm, products of
e4m3 activations and weights, gated pairs."""
import numpy as np
import pytest

from gpu_cases import say
from oracle import codecs, w8a8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U24, F8 = 2.0 ** -24, torch.float8_e4m3fn
T16 = {"f16": torch.float16, "bf16": torch.bfloat16}
STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}          # largest relative error of a rounding
TINY = {"f16": 2.0 ** -25, "bf16": 0.0, "f32": 0.0}                       # and of one to a subnormal


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_qgemm_amd as q
    return q


def dt(q, name):
    return {"f16": q.DT_F16, "bf16": q.DT_BF16, "f32": q.DT_F32, "e4m3": q.DT_FP8_E4M3}[name]


def f64(t):
    return t.double().cpu().numpy()


def guarded(shape, dtype):
    """A tensor in the middle of a larger buffer, and a check that nothing around it was written."""
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    pad = 4096
    buf = torch.full((n + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    t = buf[pad:pad + n].view(dtype).view(shape)

    def check():
        edge = torch.cat((buf[:pad], buf[pad + n:]))
        assert bool((edge == 0xA5).all()), "written outside the output"
    return t, check


def codes_match(values, want, tol, scale):
    """Held values against the exact ones: the value's own error and half a step of its code."""
    half = w8a8.half_step(np.abs(want) + tol, scale)
    assert np.all(np.abs(values - want) <= (tol + half) * (1 + 8 * U24)), np.nanmax(np.abs(values - want) - tol - half)


# ----------------------------------------------------------------------------- add_norm
def norm_inputs(tokens, dim, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((tokens, dim), generator=g) * torch.exp(torch.randn((tokens, 1), generator=g))
    x = x * (1 + 20 * (torch.rand(dim, generator=g) < 0.01))
    r = torch.randn((tokens, dim), generator=g) * 3
    return x.to(T16[dtype]), r.to(T16[dtype]), (1 + 0.3 * torch.randn(dim, generator=g)).to(T16[dtype])


def norm_check(x, r, w, norm, eps, dtype, out, got_sum, y, scales):
    s64 = x.double() if r is None else x.double() + r.double()
    s32 = x.float() if r is None else x.float() + r.float()
    if got_sum is not None:
        bad = torch.nonzero(got_sum.cpu() != s32.to(T16[dtype]))
        assert not len(bad), (len(bad), bad[:4], got_sum.cpu()[tuple(bad[0])], s32[tuple(bad[0])])
    _, want = w8a8.add_norm(s64.numpy(), None, None if w is None else w.double().numpy(), norm, eps)
    # the sum, its product with the root and with the weight, and the root itself: a rounding each; the sum of squares
    # adds 32 values one by one in a thread, then 6 steps in a wavefront, 16 wavefronts, a division and eps: half of that
    rel = (4 + (32 + 6 + 16 + 2) / 2) * U24 if norm else 2 * U24
    tol = rel * np.abs(want)
    if out != "e4m3":
        got = f64(y)
        assert np.all(np.abs(got - want) <= tol + STEP[out] * (np.abs(want) + tol) + TINY[out]), np.abs(got - want).max()
        return
    ws = w8a8.activation_scales(want)
    gs = f64(scales)
    assert np.all(np.abs(gs - ws) <= (rel + 3 * U24) * ws), np.abs(gs / ws - 1).max()
    codes = y.view(torch.uint8).cpu().numpy()
    codes_match(w8a8.activation_values(codes, scales.cpu().numpy()), want, tol + 4 * U24 * np.abs(want),
                np.repeat(gs.T, 128, axis=1))
    # the largest of a block is held as 448 itself
    top = np.abs(codecs.e4m3_decode(codes)).reshape(codes.shape[0], -1, 128).max(-1)
    assert np.all((top == 448) | (gs.T <= 2.0 ** -100))


NORMS = [(t, d, dtype, out) for dtype in ("f16", "bf16") for t, d, outs in (
    (1, 128, "eh"), (3, 8, "h"), (5, 24, "h"), (257, 512, "eh"), (2, 1000, "h"), (66, 1024, "eh"), (4, 1152, "eh"), (7, 2048, "eh"),
    (1, 2176, "eh"), (130, 4096, "eh"), (33, 5120, "eh"), (2, 8192, "eh"), (3, 8200, "h"), (2, 16384, "eh"), (3, 20096, "eh"),
    (1, 32768, "eh")) for out in [{"e": "e4m3", "h": dtype}[o] for o in outs]]


@pytest.mark.parametrize("tokens,dim,dtype,out", NORMS)
def test_add_norm(q, tokens, dim, dtype, out):
    say(f"case add_norm {tokens} {dim} {dtype} {out}")
    x, r, w = norm_inputs(tokens, dim, dtype, tokens * 7 + dim)
    for residual, weight, norm, keep in ((True, True, True, True), (False, True, True, False), (True, False, True, False),
                                         (True, True, False, True)):
        p = q.add_norm_problem(tokens, dim, dt(q, dtype), dt(q, out), norm=norm, eps=1e-5)
        y, y_ok = guarded((tokens, dim), F8 if out == "e4m3" else T16[out])
        scales, s_ok = guarded((dim // 128, tokens), torch.float32) if out == "e4m3" else (None, lambda: None)
        total, t_ok = guarded((tokens, dim), T16[dtype])
        q.add_norm(p, x.cuda(), r.cuda() if residual else None, w.cuda() if weight else None, total if keep else None, y, scales)
        torch.cuda.synchronize()
        norm_check(x, r if residual else None, w if weight else None, norm, 1e-5, dtype, out, total if keep else None, y, scales)
        y_ok(), s_ok(), t_ok()


@pytest.mark.parametrize("out", ["e4m3", "bf16"])
@pytest.mark.parametrize("dim", [128, 2048, 4224])
def test_add_norm_strides_and_in_place(q, dim, out):
    say(f"case add_norm strides {dim} {out}")
    t = 37
    x, r, w = norm_inputs(t, dim, "bf16", dim)
    wide = torch.full((t, dim + 72), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + dim] = x.cuda()
    res = torch.full((2 * t, dim), 5.0, dtype=torch.bfloat16, device="cuda")
    res[::2] = r.cuda()
    y = torch.empty((t, dim), dtype=F8 if out == "e4m3" else torch.bfloat16, device="cuda")
    scales = torch.empty((dim // 128, t), device="cuda") if out == "e4m3" else None
    p = q.add_norm_problem(t, dim, q.DT_BF16, dt(q, out))
    q.add_norm(p, wide[:, 8:8 + dim], res[::2], w.cuda(), res[::2], y, scales)           # the residual stream, in place
    torch.cuda.synchronize()
    norm_check(x, r, w, True, 1e-6, "bf16", out, res[::2], y, scales)
    assert bool((res[1::2] == 5).all()) and bool((wide[:, :8] == 7).all()) and bool((wide[:, 8 + dim:] == 7).all())
    wide[:, 8:8 + dim] = x.cuda()
    q.add_norm(p, wide[:, 8:8 + dim], r.cuda(), w.cuda(), wide[:, 8:8 + dim], y, scales)
    torch.cuda.synchronize()
    norm_check(x, r, w, True, 1e-6, "bf16", out, wide[:, 8:8 + dim], y, scales)
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, 8 + dim:] == 7).all())


def test_add_norm_edges(q):
    """Zero rows, rows below the least scale, values that are not finite."""
    say("case add_norm edges")
    t, dim = 6, 384
    g = torch.Generator().manual_seed(5)
    x = torch.randn((t, dim), generator=g)
    x[0] = 0
    x[1, :128] = 0
    x[2] *= 2.0 ** -30
    x[3] *= 2.0 ** 50
    x[4, 130] = float("inf")
    x[5, 7] = float("nan")
    x = x.bfloat16()
    y, scales = torch.empty((t, dim), dtype=F8, device="cuda"), torch.empty((3, t), device="cuda")
    q.add_norm(q.add_norm_problem(t, dim, q.DT_BF16, q.DT_FP8_E4M3, eps=0.5), x.cuda(), None, None, None, y, scales)
    torch.cuda.synchronize()
    norm_check(x[:4], None, None, True, 0.5, "bf16", "e4m3", None, y[:4], scales[:, :4].contiguous())
    assert bool((y[0].float() == 0).all()) and bool((scales[:, 0] == np.float32(2.0 ** -100 / 448)).all())
    # a NaN anywhere makes the whole row NaN; an infinite sum of squares makes the finite values of the row zero
    assert bool(torch.isnan(scales[:, 5]).all()) and bool(torch.isnan(y[5].float()).all())
    assert bool(torch.isnan(scales[1, 4])) and bool(torch.isnan(y[4, 128:256].float()).all())
    assert bool((y[4, :128].float() == 0).all())
    # without the norm: only the block itself
    x[5, :128] *= 2.0 ** -110
    x[5, 7] = 2.0 ** -102
    q.add_norm(q.add_norm_problem(t, dim, q.DT_BF16, q.DT_FP8_E4M3, norm=False), x.cuda(), None, None, None, y, scales)
    torch.cuda.synchronize()
    assert bool(torch.isnan(scales[1, 4])) and bool(torch.isfinite(scales[[0, 2], 4]).all())
    norm_check(x[:4], None, None, False, 0, "bf16", "e4m3", None, y[:4], scales[:, :4].contiguous())
    norm_check(x[5:], None, None, False, 0, "bf16", "e4m3", None, y[5:], scales[:, 5:].contiguous())


def test_add_norm_fp32_sum_feeds_the_norm(q):
    """y is made from the sum in fp32, not from the rounded one that is stored."""
    say("case add_norm unrounded")
    x = torch.full((1, 8), 256.0).bfloat16()
    r = torch.tensor([[0.75, 0.5, 0.25, 0.125, 0, 0, 0, 0]]).bfloat16()
    y, total = torch.empty((1, 8), dtype=torch.bfloat16, device="cuda"), torch.empty((1, 8), dtype=torch.bfloat16, device="cuda")
    w = (torch.arange(8) + 100.0).bfloat16()
    q.add_norm(q.add_norm_problem(1, 8, q.DT_BF16, eps=0.0), x.cuda(), r.cuda(), w.cuda(), total, y)
    torch.cuda.synchronize()
    norm_check(x, r, w, True, 0.0, "bf16", "bf16", total, y, None)


# ----------------------------------------------------------------------------- products
def product_inputs(m, n, k, parts, seed):
    g = np.random.default_rng(seed)
    blocks = parts * -(-n // 128)
    a = codecs.e4m3_encode(np.clip(g.standard_normal((m, k)) * 60, -448, 448))
    w = codecs.e4m3_encode(np.clip(g.standard_normal((parts * n, k)) * 100, -448, 448))
    sa = (np.exp(0.7 * g.standard_normal((k // 128, m))) / 60).astype(np.float32)
    sw = (np.exp(0.5 * g.standard_normal((blocks, k // 128))) * k ** -0.5 / 50).astype(np.float32)
    return a, sa, w, sw


def on_gpu(a, sa, w, sw):
    return (torch.from_numpy(a).cuda().view(F8), torch.from_numpy(sa).cuda(), torch.from_numpy(w).cuda().view(F8),
            torch.from_numpy(sw).cuda())


def product_want(a, sa, w, sw, gate, parts):
    """(exact outputs, largest error of an fp32 evaluation before the output's rounding).  A sum of a block adds 128
    products in some order, then the blocks (the scales' product and its FMA, a rounding each), then wavefronts and
    splits; no addition is off by more than 2^-23 of the sum of magnitudes.

    The e4m3 matrix instruction behind 16-bit outputs also cuts the products of each eight k at 2^-13 of the largest one's
    power of two.  Its worst case (test_products_of_eight) is more than this bound; here the cuts have random signs: of K
    products 7 K / 8 are cut, each by at most 2^-13 of a largest product of about three mean ones (E), so they add up to
    sqrt(7 K / 8) / sqrt(3) * 3 * 2^-13 E = 0.002 sqrt(K / 112) E in the mean square.  The bound has (176 + K / 64) 2^-23 K E:
    0.003 E at K = 128 and 0.03 E at 1152, to which a rounding of the output adds 2^-11 sqrt(K) E at least, 0.006 E at K = 128."""
    av, wv = w8a8.activation_values(a, sa), w8a8.weight_values(w, sw, parts)
    p, mag = av @ wv.T, np.abs(av) @ np.abs(wv).T
    tol = (128 + 2 * a.shape[1] // 128 + 48) * 2.0 ** -23 * mag
    if gate == "none":
        return p, tol
    n = p.shape[1] // 2
    g, u, tg, tu = p[:, :n], p[:, n:], tol[:, :n], tol[:, n:]
    y = w8a8.act(g, gate)
    # |act'| <= 1.13; the exponential's argument is off by 4 roundings of itself, the rest by 8 of the result
    slope = 1.13 * tg + np.abs(y) * (4 * 3 * np.abs(g) * U24 + 8 * U24)
    if gate == "gelu":
        slope += np.abs(y) * 4 * U24 * np.abs(g) ** 3
    return y * u, slope * (np.abs(u) + tu) + np.abs(y) * tu + 2 * U24 * np.abs(y * u)


def run_product(q, ins, n, gate, out, **hints):
    a, sa, w, sw = ins
    m, k = a.shape
    gates = {"none": q.GATE_NONE, "silu": q.GATE_SILU, "gelu": q.GATE_GELU_TANH}
    p = q.w8a8_problem(m, n, k, dt(q, out), gate=gates[gate], **hints)
    say(f"case product {m} {n} {k} {gate} {out} {q.w8a8_describe(p)}")
    y, y_ok = guarded((m, n), F8 if out == "e4m3" else torch.float32 if out == "f32" else T16[out])
    scales, s_ok = guarded((n // 128, m), torch.float32) if out == "e4m3" else (None, lambda: None)
    ws = q.alloc_w8a8_workspace(p)
    q.w8a8_run(p, a, sa, w, sw, y, scales, ws)
    torch.cuda.synchronize()
    y_ok(), s_ok()
    return y, scales, p, ws


def product_check(y, scales, want, tol, out):
    if out != "e4m3":
        off = np.abs(f64(y) - want)
        assert np.all(off <= tol + STEP[out] * (np.abs(want) + tol) + TINY[out]), (off - tol - STEP[out] * np.abs(want)).max()
        return
    gs, m, n = f64(scales), want.shape[0], want.shape[1]
    ws = w8a8.activation_scales(want)
    most = tol.reshape(m, -1, 128).max(-1).T / 448
    assert np.all(np.abs(gs - ws) <= most + 3 * U24 * (ws + most)), np.abs(gs / ws - 1).max()
    codes = y.view(torch.uint8).cpu().numpy()
    codes_match(w8a8.activation_values(codes, scales.cpu().numpy()), want, tol + 4 * U24 * np.abs(want), np.repeat(gs.T, 128, axis=1))
    top = np.abs(codecs.e4m3_decode(codes)).reshape(m, -1, 128).max(-1)
    assert np.all((top == 448) | (gs.T <= 2.0 ** -100))


SIZES = [(1, 16, 128), (1, 272, 1152), (3, 256, 5120), (9, 128, 1920), (2, 128, 256), (5, 640, 4096), (16, 256, 2048), (17, 400, 384), (33, 144, 1024),
         (48, 512, 640), (64, 1040, 512), (65, 256, 128), (66, 272, 384), (129, 640, 256), (255, 528, 640), (300, 1296, 512),
         (520, 256, 1280)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("gate", ["none", "silu", "gelu"])
def test_products(q, m, n, k, gate):
    parts = 1 if gate == "none" else 2
    host = product_inputs(m, n, k, parts, m * 31 + n + k)
    want, tol = product_want(*host, gate, parts)
    ins = on_gpu(*host)
    outs = ["f16", "bf16", "f32"] + (["e4m3"] if gate != "none" and n % 128 == 0 else [])
    for out in outs:
        y, scales, _, _ = run_product(q, ins, n, gate, out)
        product_check(y, scales, want, tol, out)


@pytest.mark.parametrize("m,n,k,gate,out", [(7, 256, 1792, "none", "f32"), (1, 144, 5120, "none", "f16"),
                                            (13, 384, 2688, "silu", "e4m3"), (16, 256, 4992, "gelu", "bf16"), (40, 256, 1792, "silu", "e4m3"), (64, 144, 1280, "gelu", "f16"),
                                            (20, 384, 640, "gelu", "e4m3"), (48, 128, 2304, "silu", "e4m3"), (37, 272, 2304, "none", "f32"), (130, 528, 1152, "none", "bf16"),
                                            (270, 384, 1152, "silu", "e4m3"), (61, 272, 1024, "silu", "f32")])
def test_kernels_splits_and_tiles(q, m, n, k, gate, out):
    """Every kernel, tile and number of splits gives results within the same bound, and the same call the same bits."""
    parts = 1 if gate == "none" else 2
    host = product_inputs(m, n, k, parts, m + n + k)
    want, tol = product_want(*host, gate, parts)
    ins = on_gpu(*host)
    hints = [dict(kernel_hint=q.W8A8_TILES, tile_hint=t, split_hint=s) for t in (64, 128, 256) for s in (1, 2, 5, 32)]
    if m <= 64:
        hints += [dict(kernel_hint=q.W8A8_ROWS, split_hint=s) for s in (1, 2, 3, 32)]
    for h in hints:
        y, scales, p, ws = run_product(q, ins, n, gate, out, **h)
        product_check(y, scales, want, tol, out)
        first = y.view(torch.uint8).clone()
        for _ in range(3):
            y.view(torch.uint8).zero_()
            q.w8a8_run(p, *ins, y, scales, ws)
            torch.cuda.synchronize()
            assert torch.equal(y.view(torch.uint8), first), h
        if ws is not None:
            assert bool((ws[:4 << 17] == 0).all()), "tickets"


def test_products_of_eight(q):
    """One large product among eight, all large ones cancelling: exact but for the documented cut of 16-bit outputs."""
    m, n, k = 80, 256, 128
    a = np.zeros((m, k), np.float32)
    a[:, :] = 2.0 ** -6
    a[:, ::16], a[:, 8::16] = 448, -448
    codes = torch.from_numpy(a).to(F8).cuda()
    w = torch.ones((n, k)).to(F8).cuda()
    ones = lambda *s: torch.ones(s, device="cuda")
    want, largest = 7 * 16 * 2.0 ** -6, 16 * 448.0
    for out in ("f16", "bf16", "f32"):
        for rows in (m, 16):
            ins = (codes[:rows].contiguous(), ones(1, rows), w, ones(2, 1))
            for h in [dict(kernel_hint=q.W8A8_TILES, tile_hint=t) for t in (64, 128, 256)] + [{}]:
                y, _, p, _ = run_product(q, ins, n, "none", out, **h)
                exact = out == "f32" or q.w8a8_describe(p).startswith("rows")
                assert float((y.double() - want).abs().max()) <= (0 if exact else 7 * 2.0 ** -13 * largest), (out, rows, h)


def test_last_round_split_along_k(q):
    """More tiles than compute units: whole ones first, those of the last round shared."""
    m, n, k = 130, 22000, 2560
    host = product_inputs(m, n, k, 1, 17)
    want, tol = product_want(*host, "none", 1)
    ins = on_gpu(*host)
    for tile in (64, 128):
        y, _, p, ws = run_product(q, ins, n, "none", "bf16", tile_hint=tile)
        product_check(y, None, want, tol, "bf16")
        first = y.clone()
        for _ in range(3):
            q.w8a8_run(p, *ins, y, None, ws)
            torch.cuda.synchronize()
            assert torch.equal(y, first)
    assert any("whole=256" in d and "splits=1" not in d for d in (q.w8a8_describe(q.w8a8_problem(m, n, k, tile_hint=t)) for t in (64, 128)))


def test_nan_codes_stay_in_their_rows_and_columns(q):
    for m, gate, out in ((3, "none", "f16"), (3, "silu", "e4m3"), (150, "none", "bf16"), (150, "silu", "e4m3")):
        n, k, parts = 256, 512, 1 if gate == "none" else 2
        a, sa, w, sw = product_inputs(m, n, k, parts, 9)
        a[1, 300] = 0x7f
        if gate == "none":
            w[17, 5] = 0xff
        sa[2, 2] = np.inf                                                     # a scale that is not finite, too
        y, scales, _, _ = run_product(q, on_gpu(a, sa, w, sw), n, gate, out)
        v = y.float().cpu().numpy()
        assert np.isnan(v[1]).all()
        assert not np.isfinite(v[2]).any()
        keep = np.ones(v.shape, bool)
        keep[1:3] = False
        if gate == "none":
            assert np.isnan(v[:, 17]).all()
            keep[:, 17] = False
        else:
            assert np.isnan(scales.cpu().numpy()[:, 1:3]).all()
        assert np.isfinite(v[keep]).all()


def test_zero_scales_and_zero_codes(q):
    a, sa, w, sw = product_inputs(20, 256, 256, 2, 3)
    a[4] = 0
    sw[0] = 0                                                                 # a gate's block of 128 rows
    y, scales, _, _ = run_product(q, on_gpu(a, sa, w, sw), 256, "silu", "e4m3")
    v, s = y.float().cpu().numpy(), scales.cpu().numpy()
    assert (v[4] == 0).all() and (v[:, :128] == 0).all() and (s[0] == np.float32(2.0 ** -100 / 448)).all()
    want, tol = product_want(a, sa, w, sw, "silu", 2)
    product_check(y, scales, want, tol, "e4m3")


def test_large_gate_arguments(q):
    """Gates far from zero: the exponential over- and underflows, the output does not."""
    for m in (4, 100):
        for gate in ("silu", "gelu"):
            a, sa, w, sw = product_inputs(m, 128, 256, 2, 4)
            sw[0] = np.float32(3.0)
            want, tol = product_want(a, sa, w, sw, gate, 2)
            for out in ("f32", "bf16"):
                y, scales, _, _ = run_product(q, on_gpu(a, sa, w, sw), 128, gate, out)
                # results below the smallest normal number are flushed
                product_check(y, scales, want, tol + 2.0 ** -120, out)


def test_one_workspace_for_all(q):
    """Calls of different plans share one workspace, one after the other."""
    cases = [(7, 256, 1792, "none", "f32", {}), (40, 256, 1792, "silu", "e4m3", dict(split_hint=3)),
             (130, 528, 1152, "none", "bf16", dict(split_hint=4)), (1, 16, 4096, "none", "f16", dict(split_hint=32))]
    plans = []
    for m, n, k, gate, out, h in cases:
        host = product_inputs(m, n, k, 1 if gate == "none" else 2, m + 1)
        y, scales, p, _ = run_product(q, on_gpu(*host), n, gate, out, **h)
        plans.append((p, on_gpu(*host), y.view(torch.uint8).clone(), torch.empty_like(y), None if scales is None else torch.empty_like(scales)))
    ws = torch.zeros(max(q.w8a8_workspace_bytes(p[0]) for p in plans), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for p, ins, _, y, scales in plans:
            q.w8a8_run(p, *ins, y, scales, ws)
        torch.cuda.synchronize()
        for _, _, want, y, _ in plans:
            assert torch.equal(y.view(torch.uint8), want)
            y.view(torch.uint8).zero_()


def test_empty(q):
    p = q.w8a8_problem(0, 128, 128, q.DT_F16)
    e = lambda *s: torch.empty(s, device="cuda")
    q.w8a8_run(p, e(0, 128).to(F8), e(1, 0), e(128, 128).to(F8), e(1, 1), e(0, 128).half())
    q.add_norm(q.add_norm_problem(0, 128), e(0, 128).half(), None, None, None, e(0, 128).half())
    torch.cuda.synchronize()
