"""How products enter the sums of the 8-bit products: whole, except behind 16-bit outputs of the tiles kernel that did not ask.

Activations of one and weights of +-448 that cancel beside weights of 2^-6: every partial sum is a whole number of 2^-6 below 2^18,
so fp32 sums are exact in any order, while a sum of eight products cut at 2^-13 of the largest loses the small ones."""
import numpy as np
import pytest

from gpu_cases import say
from oracle import w8a8
from test_gpu_w8a8 import F8, T16, U24, STEP, dt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

N, KB = 256, 8
EXACT = 112 * 2.0 ** -6                                                      # a block's sum over the cancelling weights


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_qgemm_amd as q
    return q


def inputs(m, cancels):
    """Codes and scales: activations 1 (tokens scaled by powers of two), weights of each projection that cancel or are all 2^-6; the
    weights' scale divides by the number of blocks."""
    hard = torch.full((N, 128 * KB), 2.0 ** -6)
    hard[:, ::16], hard[:, 8::16] = 448, -448
    plain = torch.full((N, 128 * KB), 2.0 ** -6)
    a_scales = 2.0 ** -(torch.arange(m) % 3).float().expand(KB, m).contiguous()
    w = torch.cat([hard if c else plain for c in cancels])
    return [x.cuda() for x in (torch.ones(m, 128 * KB).to(F8), a_scales, w.to(F8), torch.full((2 * len(cancels), KB), 1.0 / KB))]


def want(m, cancels, gate):
    t = 2.0 ** -(np.arange(m) % 3)
    p = [(EXACT if c else 2.0) * t for c in cancels]
    y = p[0] if gate == "none" else w8a8.act(p[0], gate) * p[1]
    # the sums are exact; the gate's exponential and what follows it, as in product_want
    tol = 0 * y if gate == "none" else (12 * p[0] + 10 + (4 * p[0] ** 3 if gate == "gelu" else 0)) * U24 * np.abs(y)
    return y[:, None], tol[:, None]


def launches(q, m):
    """Hints for every tile, unsplit and with splits of both hand-offs, and for the rows kernel."""
    out = [dict(kernel_hint=q.W8A8_TILES, tile_hint=t, split_hint=s) for t in (64, 128, 256) for s in (1, 2, 4, 8)]
    return out + ([dict(kernel_hint=q.W8A8_ROWS, split_hint=s) for s in (1, 4)] if m <= 64 else []) + [{}]


def call(q, ins, m, gate, out, **hints):
    gates = {"none": q.GATE_NONE, "silu": q.GATE_SILU, "gelu": q.GATE_GELU_TANH}
    p = q.w8a8_problem(m, N, 128 * KB, dt(q, out), gate=gates[gate], **hints)
    y = torch.empty((m, N), dtype=F8 if out == "e4m3" else torch.float32 if out == "f32" else T16[out], device="cuda")
    scales = torch.empty((N // 128, m), device="cuda") if out == "e4m3" else None
    say(f"case sums {m} {gate} {out} {q.w8a8_describe(p)}")
    q.w8a8_run(p, *ins, y, scales, q.alloc_w8a8_workspace(p))
    torch.cuda.synchronize()
    return y.double().cpu().numpy(), scales


@pytest.mark.parametrize("m", [1, 40, 130])
@pytest.mark.parametrize("gate,cancels", [("none", (True,)), ("silu", (True, False)), ("silu", (False, True)), ("silu", (True, True)),
                                          ("gelu", (True, False)), ("gelu", (False, True))])
def test_every_product_enters_whole(q, m, gate, cancels):
    ins, (y64, tol) = inputs(m, cancels), want(m, cancels, gate)
    for out in ["f32", "f16", "bf16"] + (["e4m3"] if gate != "none" else []):
        sums = q.W8A8_SUMS_WHOLE if out in T16 else q.W8A8_SUMS_AUTO
        for h in launches(q, m):
            y, scales = call(q, ins, m, gate, out, sums=sums, **h)
            if out == "e4m3":                                                 # all outputs of a token are alike: the largest, code 448
                assert (y == 448).all(), h
                s = scales.double().cpu().numpy()
                assert np.all(np.abs(s * 448 - y64.T) <= tol.T + 3 * U24 * (y64 + tol).T), h
            else:
                assert np.all(np.abs(y - y64) <= tol + STEP[out] * (np.abs(y64) + tol)), (out, h, np.abs(y / y64 - 1).max())


@pytest.mark.parametrize("gate", ["none", "silu"])
@pytest.mark.parametrize("m", [20, 200])
def test_whole_sums_leave_the_other_outputs_as_they_are(q, m, gate):
    """Where sums are whole without being asked for, asking changes no bit, and the planner says which operands it takes."""
    ins = inputs(m, (True,) if gate == "none" else (True, False))
    for out in ["f32"] + (["e4m3"] if gate != "none" else []):
        for h in launches(q, m):
            a, b = (call(q, ins, m, gate, out, sums=s, **h)[0] for s in (q.W8A8_SUMS_AUTO, q.W8A8_SUMS_WHOLE))
            assert np.array_equal(a, b), (out, h)
    gates = {"none": q.GATE_NONE, "silu": q.GATE_SILU}
    operands = lambda out, s: q.w8a8_describe(q.w8a8_problem(m, N, 1024, dt(q, out), gate=gates[gate], kernel_hint=q.W8A8_TILES,
                                                             sums=s)).split("operands=")[1]
    assert [operands(o, q.W8A8_SUMS_AUTO) for o in ("f16", "bf16", "f32")] == ["8", "8", "16"]
    assert [operands(o, q.W8A8_SUMS_WHOLE) for o in ("f16", "bf16", "f32")] == ["16", "16", "16"]


@pytest.mark.parametrize("m", [65, 300])
@pytest.mark.parametrize("gate", ["none", "silu", "gelu"])
def test_random_16_bit_products_with_whole_sums(q, m, gate):
    from test_gpu_w8a8 import on_gpu, product_check, product_inputs, product_want, run_product
    for n, k in ((272, 1152), (640, 384)):
        host = product_inputs(m, n, k, 1 if gate == "none" else 2, m + n)
        ref, tol = product_want(*host, gate, 1 if gate == "none" else 2)
        ins = on_gpu(*host)
        for out in ("f16", "bf16"):
            for t in (64, 128, 256):
                for s in (1, 3):
                    y, scales, _, _ = run_product(q, ins, n, gate, out, tile_hint=t, split_hint=s, kernel_hint=q.W8A8_TILES,
                                                  sums=q.W8A8_SUMS_WHOLE)
                    product_check(y, scales, ref, tol, out)
