"""The 8-bit operators on the CPU: descriptors, sizes and refusals of the C ABI and of the binding (nothing is
launched), the weights' quantizer against the oracle's codecs, and pins of the oracle the GPU tests hold the kernels to."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import weight_only_quantized_qgemm_amd as q
from oracle import codecs, w8a8

INV, UNS, MIS, SMALL = q.ERR_INVALID_ARGUMENT, q.ERR_UNSUPPORTED, q.ERR_MISALIGNED, q.ERR_WORKSPACE_TOO_SMALL
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_declared_function_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "qgemm_w8a8.h")).read(), flags=re.S)
    names = re.findall(r"^qgemm_status_t\s+(qgemm_[a-z0-9_]+)\s*\(", text, flags=re.M)
    assert len(names) == 5
    for n in names:
        assert hasattr(q.lib, n), n


# ----------------------------------------------------------------------------- add_norm
def _norm(**kw):
    d = dict(tokens=4, dim=256, dtype=q.DT_F16, out_dtype=q.DT_F16, norm=1, eps=1e-6, reserved=0)
    c = dict(x=0x10000, xs=256, r=0x20000, rs=256, w=0x30000, sum=0x40000, ss=256, y=0x50000, ys=None)
    for n, v in kw.items():
        (d if n in d else c)[n] = v
    p = q.AddNorm(*(d[n] for n in ("tokens", "dim", "dtype", "out_dtype", "norm", "eps", "reserved")))
    return q.lib.qgemm_add_norm(ctypes.byref(p), c["x"], c["xs"], c["r"], c["rs"], c["w"], c["sum"], c["ss"], c["y"], c["ys"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(tokens=-1), INV, "tokens"), (dict(tokens=(1 << 24) + 1), INV, "tokens"), (dict(dim=0), INV, "dim"),
    (dict(dim=252), INV, "dim"), (dict(dim=32776), INV, "dim"), (dict(dtype=q.DT_F32, out_dtype=q.DT_F32), UNS, "dtype"),
    (dict(dtype=77), INV, "dtype"), (dict(out_dtype=q.DT_BF16), UNS, "out_dtype"), (dict(out_dtype=-1), INV, "out_dtype"),
    (dict(out_dtype=q.DT_INT4), UNS, "out_dtype"), (dict(dim=264, out_dtype=q.DT_FP8_E4M3, ys=0x60000), INV, "dim"),
    (dict(norm=2), INV, "norm"), (dict(eps=-1.0), INV, "eps"), (dict(eps=float("nan")), INV, "eps"),
    (dict(eps=float("inf")), INV, "eps"), (dict(reserved=1), INV, "reserved"), (dict(x=None), INV, "x"), (dict(y=None), INV, "y"),
    (dict(out_dtype=q.DT_FP8_E4M3), INV, "y_scales"), (dict(ys=0x60000), INV, "y_scales"), (dict(x=0x10008), MIS, "x"),
    (dict(r=0x20008), MIS, "residual"), (dict(w=0x30002), MIS, "weight"), (dict(sum=0x40004), MIS, "sum_out"),
    (dict(y=0x50008), MIS, "y"), (dict(out_dtype=q.DT_FP8_E4M3, ys=0x60002), MIS, "y_scales"), (dict(xs=248), INV, "x token stride"),
    (dict(rs=260), INV, "residual token stride"), (dict(ss=0), INV, "sum_out token stride"), (dict(xs=(1 << 31) + 8), INV, "stride"),
    (dict(sum=0x10000, ss=512), INV, "in place"), (dict(sum=0x20000, ss=264), INV, "in place"), (dict(y=0x10000), INV, "overlap"),
    (dict(y=0x40000), INV, "overlap"), (dict(tokens=1 << 24, dim=2048, xs=2048, rs=2048, ss=2048), UNS, "launch")])
def test_add_norm_refusals(kw, status, text):
    assert _norm(**kw) == status and text in q.last_error(), q.last_error()


def test_add_norm_empty_and_null():
    assert _norm(tokens=0, x=None, y=None, r=None, sum=None) == q.OK
    assert q.lib.qgemm_add_norm(None, 16, 256, None, 0, None, None, 0, 16, None, None) == INV


# ----------------------------------------------------------------------------- products
def _w8a8(**kw):
    d = dict(M=4, N=256, K=256, out_dtype=q.DT_BF16, gate=0, kernel_hint=0, split_hint=0, tile_hint=0, reserved=0)
    d.update(kw)
    return q.W8A8(*d.values())


BAD = [(dict(M=-1), INV, "M must"), (dict(M=(1 << 24) + 1), INV, "M must"), (dict(N=0), INV, "N must"), (dict(N=24), INV, "N must"),
       (dict(N=(1 << 24) + 16), INV, "N must"), (dict(K=0), INV, "K must"), (dict(K=192), INV, "K must"),
       (dict(K=(1 << 22) + 128), INV, "K must"), (dict(gate=3), INV, "gate"), (dict(gate=-1), INV, "gate"),
       (dict(out_dtype=99), INV, "out_dtype"), (dict(out_dtype=q.DT_INT4), UNS, "out_dtype"),
       (dict(out_dtype=q.DT_FP8_E4M3), UNS, "needs a gate"), (dict(out_dtype=q.DT_FP8_E4M3, gate=1, N=272), INV, "N must"),
       (dict(kernel_hint=3), INV, "kernel_hint"), (dict(kernel_hint=q.W8A8_ROWS, M=65), UNS, "rows kernel"),
       (dict(split_hint=33), INV, "split_hint"), (dict(split_hint=-1), INV, "split_hint"), (dict(tile_hint=32), INV, "tile_hint"),
       (dict(reserved=5), INV, "reserved"), (dict(M=1 << 24, N=1 << 24), UNS, "launch"),
       (dict(M=16, N=1 << 24, split_hint=32, K=8192, kernel_hint=q.W8A8_ROWS, out_dtype=q.DT_FP8_E4M3, gate=1), UNS, "launch")]


@pytest.mark.parametrize("kw,status,text", BAD)
def test_product_descriptor_refusals(kw, status, text):
    p, n, buf = _w8a8(**kw), ctypes.c_size_t(7), ctypes.create_string_buffer(256)
    assert q.lib.qgemm_w8a8_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == status and text in q.last_error(), q.last_error()
    assert n.value == 7
    assert q.lib.qgemm_w8a8_describe(ctypes.byref(p), buf, 256) == status
    os_ = 0x60000 if p.out_dtype == q.DT_FP8_E4M3 else None
    assert q.lib.qgemm_w8a8_run(ctypes.byref(p), 0x1000, 0x2000, 0x3000, 0x4000, 0x5000, os_, None, 0, None) == status
    if "launch" not in text:
        assert q.lib.qgemm_w8a8_quantize(ctypes.byref(p), 16, 16, 16) == status


def _run(p=None, **kw):
    c = dict(A=0x1000, sa=0x2000, W=0x3000, sw=0x4000, out=0x5000, so=None, ws=None, n=0)
    c.update(kw)
    return q.lib.qgemm_w8a8_run(ctypes.byref(p or _w8a8()), c["A"], c["sa"], c["W"], c["sw"], c["out"], c["so"], c["ws"], c["n"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(A=None), INV, "A"), (dict(sa=None), INV, "a_scales"), (dict(W=None), INV, "W"), (dict(sw=None), INV, "w_scales"),
    (dict(out=None), INV, "out"), (dict(A=0x1008), MIS, "A"), (dict(sa=0x2002), MIS, "a_scales"), (dict(W=0x3004), MIS, "W"),
    (dict(sw=0x4001), MIS, "w_scales"), (dict(out=0x5008), MIS, "out"), (dict(so=0x6000), INV, "out_scales")])
def test_product_call_refusals(kw, status, text):
    assert _run(**kw) == status and text in q.last_error()


def test_product_outputs_and_workspace():
    g = _w8a8(gate=1, out_dtype=q.DT_FP8_E4M3)
    assert _run(g) == INV and "out_scales" in q.last_error()
    assert _run(g, so=0x6002) == MIS and "out_scales" in q.last_error()
    need = q.w8a8_workspace_bytes(g)
    assert need > 0 and _run(g, so=0x6000) == SMALL and str(need) in q.last_error()
    assert _run(g, so=0x6000, ws=0x7000, n=need - 1) == SMALL
    assert _run(g, so=0x6000, ws=0x7010, n=need) == MIS and "workspace" in q.last_error()
    assert _run(_w8a8(M=0), A=None, sa=None, W=None, sw=None, out=None) == q.OK
    assert q.lib.qgemm_w8a8_run(None, 16, 16, 16, 16, 16, None, None, 0, None) == INV
    assert q.lib.qgemm_w8a8_workspace_bytes(ctypes.byref(g), None) == INV
    buf = ctypes.create_string_buffer(8)
    assert q.lib.qgemm_w8a8_describe(ctypes.byref(g), buf, 8) == INV and "needs" in q.last_error()
    assert q.w8a8_describe(_w8a8(M=0)) == "empty" and q.w8a8_workspace_bytes(_w8a8(M=0, gate=1, out_dtype=q.DT_FP8_E4M3)) == 0


def test_plans_cover_every_size():
    """Whatever the sizes and hints: the splits share all k blocks, none of them empty, and the workspace holds the partial
    results that the kernels number."""
    g = np.random.default_rng(0)
    for _ in range(3000):
        m = int(2 ** g.uniform(0, 15))
        n, k = 16 * int(2 ** g.uniform(0, 11)), 128 * int(2 ** g.uniform(0, 8))
        gate = int(g.integers(0, 3))
        out = q.DT_F16
        if gate and g.random() < 0.5:
            n, out = -(-n // 128) * 128, q.DT_FP8_E4M3
        p = q.w8a8_problem(m, n, k, out, gate=gate, kernel_hint=int(g.choice([0, 0, 1, 2])) if m <= 64 else int(g.choice([0, 2])),
                           split_hint=int(g.choice([0, 0, 1, 2, 7, 32])), tile_hint=int(g.choice([0, 0, 64, 128, 256])))
        head, *rest = q.w8a8_describe(p).split()
        f = {a: int(b) for a, b in (x.split("=") for x in rest)}
        ws, kb = q.w8a8_workspace_bytes(p), k // 128
        per = -(-kb // f["splits"])
        assert 1 <= f["splits"] <= 32 and per * (f["splits"] - 1) < kb <= per * f["splits"]
        if head == "rows":
            members = f["splits"] * (8 if out == q.DT_FP8_E4M3 else 1)
            assert f["members"] == members and f["grid"] == n // 16 * f["splits"] and m <= 64
            assert ws == (0 if members == 1 else (4 << 17) + f["grid"] * (2 if gate else 1) * 1024 * -(-m // 16))
        else:
            cols = 128 if gate else 256
            tiles = -(-m // f["tokens"]) * -(-n // cols)
            assert f["whole"] <= tiles and f["grid"] == f["whole"] + (tiles - f["whole"]) * f["splits"]
            assert (f["splits"] == 1) == (f["whole"] == tiles) or f["splits"] == 1
            assert ws == (0 if f["splits"] == 1 else (4 << 17) + (tiles - f["whole"]) * f["splits"] * f["tokens"] * 1024)


# ----------------------------------------------------------------------------- the quantizer
@pytest.mark.parametrize("n,k,gate", [(16, 128, 0), (272, 384, 0), (128, 256, 1), (144, 128, 2)])
def test_quantize(n, k, gate):
    g = np.random.default_rng([n, k])
    parts = 2 if gate else 1
    w = (g.standard_normal((parts * n, k)) * np.exp(g.standard_normal((parts * n, 1)))).astype(np.float32)
    w[:16, :128] = 0 if n == 16 else w[:16, :128]
    codes, scales = q.w8a8_quantize(q.w8a8_problem(1, n, k, gate=gate), w)
    per = -(-n // 128)
    assert scales.shape == (parts * per, k // 128)
    for p in range(parts):
        for b in range(per):
            for c in range(k // 128):
                at = np.s_[p * n + 128 * b:p * n + min(n, 128 * b + 128), 128 * c:128 * c + 128]
                s = np.float32(np.abs(w[at]).max()) / np.float32(448)
                assert scales[p * per + b, c] == s
                want = codecs.e4m3_encode(np.clip(w[at].astype(np.float64) / float(s), -448, 448)) if s else np.zeros(w[at].shape, np.uint8)
                assert np.array_equal(codes[at], want)
    v = w8a8.weight_values(codes, scales, parts)
    s = np.abs(w).reshape(parts * n, -1, 128).max(-1)
    assert np.all(np.abs(v - w) <= w8a8.half_step(np.abs(w), np.repeat(scales.max() * np.ones_like(s), 128, 1)) * (1 + 2.0 ** -20))


def test_quantize_refuses_what_is_not_finite():
    p = q.w8a8_problem(1, 16, 128)
    w = np.zeros((16, 128), np.float32)
    for bad in (np.inf, -np.inf, np.nan):
        w[3, 5] = bad
        with pytest.raises(q.QgemmError, match=r"w\[389\] is not finite"):
            q.w8a8_quantize(p, w)
    w[3, 5] = 1e-44                                           # a scale that rounds to zero holds zeros
    codes, scales = q.w8a8_quantize(p, w)
    assert scales[0, 0] == 0 and not codes.any()
    assert q.lib.qgemm_w8a8_quantize(ctypes.byref(p), None, 16, 16) == INV


# ----------------------------------------------------------------------------- the oracle
def test_oracle_pins():
    a = np.array([[0x38] * 128 + [0xB8] * 128], np.uint8)                     # 1 and -1
    s = np.array([[2.0], [0.5]], np.float32)
    v = w8a8.activation_values(a, s)
    assert (v[0, :128] == 2).all() and (v[0, 128:] == -0.5).all()
    w = np.full((130, 128), 0x40, np.uint8)                                   # 2
    x = w8a8.weight_values(w, np.array([[1.0], [3.0]], np.float32))
    assert (x[:128] == 2).all() and (x[128:] == 6).all()
    y = w8a8.weight_values(w, np.array([[1.0], [5.0]], np.float32), 2)        # two projections of 65 rows
    assert (y[:65] == 2).all() and (y[65:] == 10).all()
    x = np.zeros((2, 256))
    x[0, 3], x[0, 200], x[1, 0] = -896, 2.0 ** -110, np.inf
    t = w8a8.activation_scales(x)
    assert t[0, 0] == 2 and t[1, 0] == 2.0 ** -100 / 448 and np.isnan(t[0, 1]) and t[1, 1] == 2.0 ** -100 / 448
    total, y = w8a8.add_norm(np.array([[3.0, 4.0]]), np.array([[0.0, 0.0]]), np.array([1.0, 2.0]), True, 0.0)
    assert np.allclose(y, [[3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5]]) and (total == [[3, 4]]).all()
    assert w8a8.act(np.float64(0), "silu") == 0 and abs(w8a8.act(np.float64(1), "silu") - 0.7310585786300049) < 1e-15
    assert abs(w8a8.act(np.float64(1), "gelu") - 0.8411919906082768) < 1e-12
    assert w8a8.half_step(16.0, 1.0) == 1 and w8a8.half_step(0.0, 1.0) == 2.0 ** -10


# ----------------------------------------------------------------------------- the binding
class Elsewhere:
    """A tensor that says it lies on another device; its memory is the host's, which the checks must keep from the library."""

    def __init__(self, x, device, pinned=False):
        self.x, self.device, self.pinned = x, device, pinned

    def is_pinned(self):
        return self.pinned

    def get_device(self):
        return self.device

    def __getattr__(self, name):
        return getattr(self.x, name)


def norm_call(**kw):
    f8 = kw.pop("f8", False)
    h = lambda: torch.zeros(3, 256).half()
    d = dict(x=h(), residual=h(), weight=torch.ones(256).half(), sum_out=h(), y=h().to(torch.float8_e4m3fn) if f8 else h(),
             y_scales=torch.zeros(2, 3) if f8 else None)
    return dict(p=q.add_norm_problem(3, 256, out_dtype=q.DT_FP8_E4M3 if f8 else None), **d, **kw)


def run_call(gated=False, **kw):
    f8 = torch.float8_e4m3fn
    parts = 2 if gated else 1
    d = dict(A=torch.zeros(3, 256).to(f8), a_scales=torch.zeros(2, 3), W=torch.zeros(parts * 128, 256).to(f8),
             w_scales=torch.zeros(parts, 2), out=torch.zeros(3, 128).to(f8) if gated else torch.zeros(3, 128).bfloat16(),
             out_scales=torch.zeros(1, 3) if gated else None, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    p = q.w8a8_problem(3, 128, 256, q.DT_FP8_E4M3 if gated else q.DT_BF16, gate=q.GATE_SILU if gated else q.GATE_NONE)
    return dict(p=p, **d, **kw)


@pytest.mark.parametrize("f,make,kw", [(q.add_norm, norm_call, {}), (q.add_norm, norm_call, dict(f8=True)), (q.w8a8_run, run_call, {}),
                                       (q.w8a8_run, run_call, dict(gated=True))])
def test_binding_checks_every_tensor(f, make, kw):
    with pytest.raises(ValueError, match="on the GPU"):
        f(**make(**kw))
    names = [n for n, v in make(**kw).items() if isinstance(v, torch.Tensor)]
    at = lambda **odd: {n: odd.get(n, Elsewhere(v, 0)) if isinstance(v, torch.Tensor) else v for n, v in make(**kw).items()}
    for n in names:
        v = make(**kw)[n]
        for device, text in ((-1, f"{n} must be on the GPU"), (1, "on device")):
            with pytest.raises(ValueError, match=text):
                f(**at(**{n: Elsewhere(v, device)}), stream=0)
        if n == "workspace":
            continue
        wrong = [v.double(), v[:1] if n != "weight" else v[:8]]                 # another type, another shape
        if v.dim() == 2:
            wrong.append(torch.zeros(v.shape[1], v.shape[0]).to(v.dtype).t())   # another order
        for bad in wrong:
            if bad.shape == v.shape and bad.is_contiguous() and bad.dtype == v.dtype:
                continue
            with pytest.raises(ValueError, match=f"^{n} must be"):
                f(**at(**{n: Elsewhere(bad, 0)}), stream=0)
    with pytest.raises(TypeError, match="descriptor"):
        f(**dict(at(), p=b"123"), stream=0)


def test_binding_refuses_loose_workspaces_and_odd_sizes():
    at = {n: Elsewhere(v, 0) if isinstance(v, torch.Tensor) else v for n, v in run_call(gated=True).items()}
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        q.w8a8_run(**dict(at, workspace=Elsewhere(torch.zeros(2 << 20, dtype=torch.uint8)[::2], 0)), stream=0)
    with pytest.raises(ValueError, match="must be in"):
        q.w8a8_run(**dict(at, p=q.w8a8_problem(1 << 40, 128, 256)), stream=0)
    with pytest.raises(q.QgemmError, match="workspace"):
        q.w8a8_run(**dict(at, workspace=None), stream=0)
