"""The attention operators on the CPU: descriptors, sizes and refusals of the C ABI (nothing is
launched), and pins of the oracle that the GPU tests hold the kernels to."""
import ctypes

import numpy as np
import pytest

import weight_only_quantized_qgemm_amd as q
from oracle import attention as oa

INV, UNS, MIS, SMALL = q.ERR_INVALID_ARGUMENT, q.ERR_UNSUPPORTED, q.ERR_MISALIGNED, q.ERR_WORKSPACE_TOO_SMALL


# ----------------------------------------------------------------------------- refusals
def _cache(**kw):
    a = dict(num_pages=8, page_size=16, kv_heads=2, head_dim=128, group_size=128, dtype=q.DT_F16, reserved=0)
    a.update(kw)
    return q.Cache(**a)


BAD_CACHES = [(dict(num_pages=0), INV, "num_pages"), (dict(num_pages=1 << 31), INV, "num_pages"),
              (dict(page_size=8), INV, "page_size"), (dict(page_size=24), INV, "page_size"),
              (dict(page_size=4112), INV, "page_size"), (dict(kv_heads=0), INV, "kv_heads"),
              (dict(kv_heads=1025), INV, "kv_heads"), (dict(head_dim=96), UNS, "head_dim"),
              (dict(group_size=16), UNS, "group_size"), (dict(group_size=0), UNS, "group_size"),
              (dict(head_dim=64, group_size=16), UNS, "group_size"), (dict(dtype=q.DT_F32), UNS, "dtype"),
              (dict(dtype=77), INV, "dtype"), (dict(reserved=1), INV, "reserved")]


@pytest.mark.parametrize("kw,status,text", BAD_CACHES)
def test_cache_descriptor_refusals(kw, status, text):
    c, n = _cache(**kw), ctypes.c_size_t(7)
    assert q.lib.qgemm_cache_bytes(ctypes.byref(c), ctypes.byref(n)) == status and text in q.last_error()
    assert n.value == 7
    for st in (q.lib.qgemm_cache_write(ctypes.byref(c), 16, 16, 256, 16, 256, 16, 1, None),
               q.lib.qgemm_cache_read(ctypes.byref(c), 16, 16, 1, 16, 16, None)):
        assert st == status and text in q.last_error()
    a = q.Attention(c, 1, 1, 2, 1, 1, 1, 0, 1.0, 0, (0, 0))
    assert q.lib.qgemm_attention_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == status and text in q.last_error()


def test_null_descriptors_and_sizes():
    n = ctypes.c_size_t()
    assert q.lib.qgemm_cache_bytes(None, ctypes.byref(n)) == INV
    assert q.lib.qgemm_cache_bytes(ctypes.byref(_cache()), None) == INV
    assert q.lib.qgemm_attention_workspace_bytes(None, ctypes.byref(n)) == INV
    assert q.lib.qgemm_qk_norm_rope(None, 16, 1024, 16, 1024, None, None, 16, 16, 16, 1024, 16, 1024, None) == INV
    assert q.lib.qgemm_attention(None, 16, 256, 16, 16, 16, 16, 16, 256, None, 0, None) == INV


@pytest.mark.parametrize("dim,group", [(64, 64), (64, 32), (128, 128), (128, 32), (256, 64)])
def test_cache_bytes(dim, group):
    c = q.cache(5, 48, 3, dim, q.DT_BF16, group_size=group)
    assert q.cache_bytes(c) == 5 * 3 * oa.block_bytes(48, dim, group)
    big = q.cache(2 ** 31 - 1, 4096, 1024, dim, q.DT_F16, group_size=group)          # past 32 bits, not past 64
    assert q.cache_bytes(big) == (2 ** 31 - 1) * 1024 * oa.block_bytes(4096, dim, group)


def _write(c, **kw):
    a = dict(data=0x1000, k=0x2000, ks=256, v=0x3000, vs=256, slots=0x4000, n=3)
    a.update(kw)
    return q.lib.qgemm_cache_write(ctypes.byref(c), a["data"], a["k"], a["ks"], a["v"], a["vs"], a["slots"], a["n"], None)


def _read(c, **kw):
    a = dict(data=0x1000, slots=0x4000, n=3, k=0x2000, v=0x3000)
    a.update(kw)
    return q.lib.qgemm_cache_read(ctypes.byref(c), a["data"], a["slots"], a["n"], a["k"], a["v"], None)


def test_cache_call_refusals():
    c = _cache()
    for f in (_write, _read):
        for name in ("data", "k", "v", "slots"):
            assert f(c, **{name: None}) == INV and "NULL" in q.last_error()
        for name in ("data", "k", "v"):
            assert f(c, **{name: 0x1008}) == MIS and name in q.last_error()
        assert f(c, slots=0x4004) == MIS and "slots" in q.last_error()
        assert f(c, n=-1) == INV and f(c, n=(1 << 24) + 1) == INV and "tokens" in q.last_error()
        assert f(c, n=0, data=None, k=None, v=None, slots=None) == q.OK                   # nothing to do
    for name in ("ks", "vs"):
        for bad in (255, 252, 260, 0, -256, (1 << 31) + 8):
            assert _write(c, **{name: bad}) == INV and "stride" in q.last_error()


def _rope(**kw):
    a = dict(tokens=4, q_heads=4, kv_heads=2, head_dim=64, rot_dim=64, max_pos=32, dtype=q.DT_F16, interleaved=0, norm=1,
             eps=1e-6, reserved=0)
    call = dict(q=0x1000, qs=256, k=0x2000, ks=128, qw=None, kw=None, pos=0x3000, tab=0x4000, qo=0x5000, qos=256, ko=0x6000,
                kos=128)
    for n, v in kw.items():
        (a if n in a else call)[n] = v
    c = call
    return q.lib.qgemm_qk_norm_rope(ctypes.byref(q.NormRope(**a)), c["q"], c["qs"], c["k"], c["ks"], c["qw"], c["kw"],
                                    c["pos"], c["tab"], c["qo"], c["qos"], c["ko"], c["kos"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(tokens=-1), INV, "tokens"), (dict(tokens=(1 << 24) + 1), INV, "tokens"), (dict(q_heads=-1), INV, "heads"),
    (dict(q_heads=0, kv_heads=0), INV, "heads"), (dict(kv_heads=1025), INV, "heads"), (dict(head_dim=80), UNS, "head_dim"),
    (dict(rot_dim=4), INV, "rot_dim"), (dict(rot_dim=72), INV, "rot_dim"), (dict(rot_dim=-8), INV, "rot_dim"),
    (dict(max_pos=0), INV, "max_pos"), (dict(dtype=q.DT_F32), UNS, "dtype"), (dict(dtype=-1), INV, "dtype"),
    (dict(interleaved=2), INV, "interleaved"), (dict(norm=-1), INV, "norm"), (dict(eps=-1.0), INV, "eps"),
    (dict(eps=float("nan")), INV, "eps"), (dict(eps=float("inf")), INV, "eps"), (dict(reserved=3), INV, "reserved"),
    (dict(q=None), INV, "q"), (dict(ko=None), INV, "k_out"), (dict(pos=None), INV, "positions"), (dict(tab=None), INV, "cos_sin"),
    (dict(q=0x1002), MIS, "q"), (dict(ko=0x6008), MIS, "k_out"), (dict(pos=0x3002), MIS, "positions"),
    (dict(tab=0x4004), MIS, "cos_sin"), (dict(qw=0x7008), MIS, "weight"), (dict(kw=0x7008), MIS, "weight"),
    (dict(qs=248), INV, "stride"), (dict(ks=132), INV, "stride"), (dict(qos=0), INV, "stride"), (dict(kos=-128), INV, "stride"),
    (dict(qo=0x1000, qos=512), INV, "in place"), (dict(ko=0x2000, kos=136), INV, "in place")])
def test_norm_rope_refusals(kw, status, text):
    assert _rope(**kw) == status and text in q.last_error(), q.last_error()


def test_norm_rope_without_work_or_parts():
    assert _rope(tokens=0, q=None, k=None, qo=None, ko=None, pos=None, tab=None) == q.OK
    # a launch too large for one grid is refused, not cut
    assert _rope(tokens=1 << 24, q_heads=1024, kv_heads=1024, qs=65536, qos=65536, ks=65536, kos=65536) == UNS


def _attn(**kw):
    a = dict(total_q=4, batch=2, q_heads=4, max_q_len=2, max_pages=3, causal=1, window=0, scale=0.1, kernel_hint=0,
             reserved=(0, 0))
    call = dict(q=0x1000, qs=512, data=0x2000, table=0x3000, lens=0x4000, starts=0x5000, out=0x6000, os=512, ws=None, wsb=0)
    for n, v in kw.items():
        (a if n in a else call)[n] = v
    c = call
    p = q.Attention(cache=_cache(), **a)
    if c["ws"] == "enough":
        c["ws"], c["wsb"] = 0x10000, q.attention_workspace_bytes(p)
    return q.lib.qgemm_attention(ctypes.byref(p), c["q"], c["qs"], c["data"], c["table"], c["lens"], c["starts"], c["out"],
                                 c["os"], c["ws"], c["wsb"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(total_q=-1), INV, "total_q"), (dict(total_q=(1 << 24) + 1), INV, "total_q"), (dict(batch=0), INV, "batch"),
    (dict(batch=65536), INV, "batch"), (dict(q_heads=3), INV, "q_heads"), (dict(q_heads=0), INV, "q_heads"),
    (dict(q_heads=4098), INV, "q_heads"), (dict(max_q_len=0), INV, "max_q_len"), (dict(max_q_len=5), INV, "max_q_len"),
    (dict(max_pages=0), INV, "max_pages"), (dict(max_pages=(1 << 26) + 1), INV, "max_pages"), (dict(causal=2), INV, "causal"),
    (dict(window=-1), INV, "window"), (dict(window=4, causal=0), INV, "window"), (dict(scale=float("inf")), INV, "scale"),
    (dict(kernel_hint=3), INV, "kernel_hint"), (dict(reserved=(0, 1)), INV, "reserved"), (dict(q=None), INV, "q"),
    (dict(data=None), INV, "data"), (dict(out=None), INV, "out"), (dict(table=None), INV, "page_table"),
    (dict(lens=None), INV, "seq_lens"), (dict(starts=None), INV, "q_start"), (dict(q=0x1008), MIS, "16-byte"),
    (dict(data=0x2004), MIS, "16-byte"), (dict(out=0x6002), MIS, "16-byte"), (dict(table=0x3002), MIS, "4-byte"),
    (dict(lens=0x4001), MIS, "4-byte"), (dict(starts=0x5002), MIS, "4-byte"), (dict(qs=511), INV, "stride"),
    (dict(qs=500), INV, "stride"), (dict(os=516), INV, "stride"), (dict(os=0), INV, "stride")])
def test_attention_refusals(kw, status, text):
    assert _attn(**kw) == status and text in q.last_error(), q.last_error()


def test_attention_workspace_refusals():
    # whatever the plan asks for is checked before anything is enqueued
    need = 0
    for total, batch, hint in ((4, 2, 0), (1, 1, 0), (300, 1, 0), (300, 3, 1), (300, 3, 2)):
        p = q.Attention(_cache(), total, batch, 4, 1 if total < 5 else total // batch, 3, 1, 0, 0.1, hint, (0, 0))
        n = q.attention_workspace_bytes(p)
        assert n % 256 == 0
        assert q.attention_describe(p).split()[0] in ("rows", "tiles")
        if n:
            need += 1
            kw = dict(total_q=total, batch=batch, max_q_len=p.max_q_len, kernel_hint=hint)
            assert _attn(ws=0x10000, wsb=n - 1, **kw) == SMALL
            assert _attn(ws=None, wsb=n, **kw) == SMALL
            assert _attn(ws=0x10010, wsb=n, **kw) == MIS
    assert _attn(total_q=0, max_q_len=0, q=None, out=None) == q.OK
    empty = q.Attention(_cache(), 0, 1, 4, 0, 3, 1, 0, 0.1, 0, (0, 0))
    assert q.attention_describe(empty) == "empty" and q.attention_workspace_bytes(empty) == 0
    buf = ctypes.create_string_buffer(4)
    assert q.lib.qgemm_attention_describe(ctypes.byref(empty), buf, 4) == INV and buf.value == b"emp"
    assert q.lib.qgemm_attention_describe(ctypes.byref(empty), None, 4) == INV


def test_binding_refuses_tensors_that_do_not_fit():
    import torch
    c = q.cache(4, 16, 2, 64)
    ok = torch.zeros(3, 2, 64, dtype=torch.float16)
    data, slots = torch.zeros(q.cache_bytes(c), dtype=torch.uint8), torch.zeros(3, dtype=torch.int64)
    for bad in (ok[:2], ok.float(), ok.transpose(0, 1), torch.zeros(3, 2, 128, dtype=torch.float16)[..., ::2],
                torch.zeros(3, 4, 64, dtype=torch.float16)[:, ::2]):
        with pytest.raises(ValueError):
            q.cache_write(c, data, bad, ok, slots)
        with pytest.raises(ValueError):
            q.cache_write(c, data, ok, bad, slots)
    with pytest.raises(ValueError):
        q.cache_write(c, data[:-1], ok, ok, slots)
    with pytest.raises(ValueError):
        q.cache_write(c, data, ok, ok, slots.int())
    with pytest.raises(ValueError):
        q.cache_read(c, data, slots, ok[:2], ok)
    p = q.attention_problem(c, 1, 3, 4, 3, 2)
    x, i = torch.zeros(3, 4, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    for kw in (dict(q=x[:2]), dict(q=x.bfloat16()), dict(out=x[:, :2]), dict(page_table=i[:1]), dict(seq_lens=i.long()),
               dict(q_start=i[:1])):
        a = dict(q=x, data=data, page_table=i, seq_lens=i, q_start=i, out=x)
        a.update(kw)
        with pytest.raises(ValueError):
            q.attention(p, **a)
    r = q.norm_rope_problem(3, 4, 2, 64, max_pos=8)
    t, pos = torch.zeros(8, 64), torch.zeros(3, dtype=torch.int32)
    for kw in (dict(positions=pos[:2]), dict(positions=pos.long()), dict(cos_sin=t[:7]), dict(cos_sin=t.half()),
               dict(q_weight=torch.zeros(63, dtype=torch.float16)), dict(k_out=ok.bfloat16())):
        a = dict(q=x, k=ok, q_weight=None, k_weight=None, positions=pos, cos_sin=t, q_out=x, k_out=ok)
        a.update(kw)
        with pytest.raises(ValueError):
            q.qk_norm_rope(r, **a)


# ----------------------------------------------------------------------------- oracle pins
def test_oracle_round16():
    v = np.array([1.0, 1 + 2 ** -9, 1 + 2 ** -8, 1 + 3 * 2 ** -8, -3.0, 0.0, 1e-40, 3.4e38, np.inf, 65504.0, 2 ** -24, 2 ** -26])
    import torch
    t = torch.from_numpy(v)
    assert np.array_equal(oa.round16(v, "bf16"), t.to(torch.bfloat16).double().numpy())
    assert np.array_equal(oa.round16(v, "f16"), t.to(torch.float16).double().numpy())
    for kind in ("f16", "bf16"):
        x = oa.round16(np.array([0.5, -1.25, 0.0, 96.0, 3.0e-5]), kind)
        assert np.array_equal(oa.from_bits16(oa.bits16(x, kind), kind), x)


def test_oracle_quantize_by_hand():
    # 0, 1, .. 15 spaced by one: scale 1, zero the minimum, codes the steps
    x = np.arange(32.0).reshape(2, 16)[::-1] - 3.0
    c, s, z = oa.quantize(x, 16, "f16")
    assert np.array_equal(c, np.tile(np.arange(16), (2, 1))) and np.array_equal(s, [[1.0], [1.0]])
    assert np.array_equal(z, [[13.0], [-3.0]])
    # a constant group: scale 0, codes 0, the value itself
    c, s, z = oa.quantize(np.full((1, 32), 2.5), 32, "bf16")
    assert not c.any() and s[0, 0] == 0 and z[0, 0] == 2.5
    # halves go to the even code; a group with a NaN or an infinity is all NaN, its neighbour is not
    c, _, _ = oa.quantize(np.array([[0.0, 15.0, 0.5, 1.5, 2.5, 7.0, 8.0, 3.0]]), 8, "f16")
    assert c.tolist() == [[0, 15, 0, 2, 2, 7, 8, 3]]
    for badval in (np.nan, np.inf, -np.inf):
        x = np.arange(16.0).reshape(1, 16).copy()
        x[0, 3] = badval
        c, s, z = oa.quantize(x, 8, "f16")
        assert np.isnan(s[0, 0]) and np.isnan(z[0, 0]) and not c[0, :8].any() and s[0, 1] > 0 and z[0, 1] == 8


def test_oracle_values_are_within_half_a_step():
    g = np.random.default_rng(5)
    for kind, dim, group in (("f16", 128, 32), ("bf16", 64, 64), ("bf16", 256, 128)):
        x = oa.round16(g.standard_normal((50, dim)) * 3, kind)
        c, s, z = oa.quantize(x, group, kind)
        off = np.abs(oa.dequantize(c, s, z, group) - x)
        # half a step inside the grid; at its upper end the rounded scale leaves 15 roundings of it
        step = np.repeat(s, group, -1)
        assert np.all(off <= step * (0.5 + 15 * oa.UNIT[kind]) + 1e-6)


def test_oracle_block_layout_by_hand():
    # dims 0..7 in K dword 0, dims 32..39 in dword 1 (step 1 of lane group 0), dims 8..15 in dword u
    P, D = 16, 64
    kc, vc = np.zeros((P, D), np.uint8), np.zeros((P, D), np.uint8)
    kc[0, 0], kc[0, 33], kc[1, 8] = 5, 6, 7
    vc[0, 0], vc[5, 17], vc[2, 50] = 9, 10, 11
    one = np.ones((P, 1))
    b = oa.pack_block(kc, one, 2 * one, vc, 3 * one, 4 * one, "f16")
    assert b.size == oa.block_bytes(P, D, 64) == P * 72
    want = {0: 5, 4: 6 << 4, 32 + 8: 7}                            # u = 2: dword 2 g + i
    want[512 + 0] = 9                                              # t 0, r 0, i 0
    want[512 + ((1 * 16 + 1) * 8 + 1 * 2 + 0)] = 10 << 4           # t 5: quad 1, place 1; dim 17: r 1, i 1
    want[512 + (2 * 8 + 2 * 2 + 1)] = 11 << 4                      # t 2; dim 50: r 2, i 3
    assert {int(i): int(b[i]) for i in np.flatnonzero(b[:1024])} == want
    assert b[1024:].view(np.float16).reshape(2, P, 2).tolist() == [[[1.0, 2.0]] * P, [[3.0, 4.0]] * P]


def test_oracle_attention_by_hand():
    k = np.array([[1.0, 0.0], [0.0, 1.0], [1.0, 1.0]])
    v = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    # two queries at positions 1 and 2: the first sees two tokens, equal scores give the mean
    out, w = oa.attention(np.array([[0.0, 0.0], [np.log(2.0), 0.0]]), k, v, 3, True, 0, 1.0)
    assert np.allclose(out[0], [2.0, 3.0]) and np.allclose(w[1], [0.4, 0.2, 0.4])
    # a window of one is the value itself; queries before the first token see nothing
    assert np.allclose(oa.attention(np.ones((1, 2)), k, v, 3, True, 1, 1.0)[0], v[2:])
    out, w = oa.attention(np.ones((4, 2)), k, v, 3, True, 0, 1.0)
    assert not out[0].any() and not w[0].any() and np.allclose(out[1], v[0])
    assert np.allclose(oa.attention(np.zeros((1, 2)), k, v, 3, False, 0, 1.0)[0], v.mean(0))


def test_oracle_norm_rope_by_hand():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    y, _ = oa.norm_rope(x, None, None, None, 0, False, True, 0.0)
    assert np.allclose(y, x / 2.5)
    table = np.array([[0.0, 1.0, 1.0, 0.0]])                       # pair 0 by a quarter turn, pair 1 not at all
    y, _ = oa.norm_rope(x, None, np.array([5]), table, 4, False, False)
    assert np.allclose(y, [[[-0.0, 4.0, 3.0, 0.0]]])               # pairs (0, 2), (1, 3)
    y, _ = oa.norm_rope(x, None, np.array([-1]), table, 4, True, False)
    assert np.allclose(y, [[[-4.0, 3.0, 0.0, 0.0]]])               # pairs (0, 1), (2, 3)


# ----------------------------------------------------------------------------- the compiled calls
def test_calls_refuse_what_is_no_descriptor():
    import torch
    x = torch.zeros(2, 2, 128, dtype=torch.float16)
    s = torch.zeros(2, dtype=torch.int64)
    for bad in (q.norm_rope_problem(2, 2, 2, 128), None, 3):
        with pytest.raises(TypeError):
            q.cache_write(bad, x, x, x, s)
    with pytest.raises(TypeError, match="32 bytes"):
        q.cache_read(q.Problem(), x, s, x, x)
    with pytest.raises(TypeError):
        q._calls.attention(1, 2)
    with pytest.raises(AttributeError):
        q.cache_write(q.cache(1, 16, 2, 128), x, [1.0], x, s)


def test_calls_hold_no_references():
    # refused and passed checks alike leave the reference counts as they were
    import sys

    import torch
    x, flat = torch.zeros(2, 2, 128, dtype=torch.float16), torch.zeros(2, 256, dtype=torch.float16)
    c, s = q.cache(1, 16, 2, 128), torch.zeros(2, dtype=torch.int64)
    data, short = q.alloc_cache(c, "cpu"), torch.zeros(5, dtype=torch.uint8)
    held = (x, flat, c, s, data, short, torch.float16, torch.uint8)

    def calls():
        for args in ((short, x, flat, s), (data, x[:1], x, s), (data, x.float(), x, s), (data, x, flat, s.int())):
            with pytest.raises(ValueError):
                q.cache_write(c, *args)
        with pytest.raises(TypeError):                                 # past the tensors' checks
            q.cache_write(c, data, x, flat, s, stream="none")

    calls()
    before = [sys.getrefcount(o) for o in held]
    for _ in range(50):
        calls()
    assert all(abs(sys.getrefcount(o) - b) < 10 for o, b in zip(held, before))


# ----------------------------------------------------------------------------- plans
@pytest.mark.parametrize("hint", [0, 1, 2])
@pytest.mark.parametrize("dim,group,dtype", [(64, 32, 0), (128, 128, 0), (128, 32, 1), (256, 64, 0), (256, 256, 1)])
def test_plans_hold_their_limits(dim, group, dtype, hint):
    # grids, parts and workspaces over the range of calls: tickets for every workgroup that may join,
    # partial results for all of them
    g = np.random.default_rng([9, dim, group, dtype, hint])
    for _ in range(200):
        hk = int(g.choice([1, 2, 3, 8, 16]))
        batch, max_q = int(2 ** g.uniform(0, 9)), int(2 ** g.uniform(0, 13))
        total = int(g.integers(max_q, batch * max_q + 1))
        c = q.cache(1 << 20, 16, hk, dim, dtype, group_size=group)
        p = q.attention_problem(c, batch, total, hk * int(g.choice([1, 2, 5, 8])), max_q, int(2 ** g.uniform(0, 14)),
                                causal=bool(g.random() < 0.8), kernel_hint=hint)
        try:
            kind, *fields = q.attention_describe(p).split()
        except q.QgemmError as e:                                      # more units than a launch divides: only on request
            assert hint == 1 and e.status == UNS and "row tiles" in e.detail
            continue
        f = {k: int(v) for k, v in (x.split("=") for x in fields)}
        ws = q.attention_workspace_bytes(p)
        assert f["groups"] == dim // group and (hint == 0 or kind == ("rows", "tiles")[hint - 1])
        if kind == "rows":
            assert f["grid"] in (512, 2048) and ws == 32768 + 2 * f["grid"] * (16 // f["pack"]) * (dim + 4) * 4
        elif f["splits"] == 1:
            assert ws == 0
        else:
            assert 2 <= f["splits"] <= 32 and f["grid"] <= 8192 and f["grid"] % f["splits"] == 0
            assert ws == 32768 + f["grid"] * f["rows"] * (dim + 16) * 4
