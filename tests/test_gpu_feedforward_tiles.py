"""The 8-bit operators together where the tiles kernel's workgroups share a tile (splits along K): captured and replayed, with two
layers on two streams at once, and beside whole tiles in one launch."""
import numpy as np
import pytest

from gpu_cases import say
from test_gpu_feedforward import FeedForward, inputs
from test_gpu_w8a8 import F8, product_check, product_want, run_product

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_qgemm_amd as q
    return q


# tokens, width, inner width, tile and split hints (0: the plan's own): tiles handed over whole (64 tokens by two or three) and in parts
LAYERS = [(40, 512, 896, 64, 3), (40, 512, 896, 64, 4), (150, 512, 896, 128, 3), (300, 512, 896, 256, 2), (70, 2048, 2816, 0, 0)]


def layer(q, tokens, width, inner, tile, split, seed):
    f = FeedForward(q, tokens, width, inner, seed)
    for p in (f.up, f.down):
        p.kernel_hint, p.tile_hint, p.split_hint = q.W8A8_TILES, tile, split
        head, *fields = q.w8a8_describe(p).split()
        shared = dict(x.split("=") for x in fields)
        assert head == "tiles" and int(shared["splits"]) > 1 and shared["whole"] == "0", (head, shared)
    f.ws = q.alloc_w8a8_workspace([f.up, f.down])
    return f


@pytest.mark.parametrize("tokens,width,inner,tile,split", LAYERS)
def test_captured_replays_equal_eager_calls(q, tokens, width, inner, tile, split):
    say(f"case shared tiles graph {tokens} {tile} {split}")
    f = layer(q, tokens, width, inner, tile, split, 6)
    x, r = inputs(tokens, width, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f(x, r)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(x, r)
    for seed in range(2, 7):
        x1, r1 = inputs(tokens, width, seed)
        x.copy_(x1), r.copy_(r1)
        y = f(x, r).clone()
        total, after = r.clone(), f.after.clone()
        torch.cuda.synchronize()
        f.y.zero_(), f.after.zero_()
        x.copy_(x1), r.copy_(r1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(f.y, y) and torch.equal(r, total) and torch.equal(f.after, after), seed
        assert bool((f.ws[:4 << 17] == 0).all()), "tickets"


def test_two_streams_at_once(q):
    """Layers of every hand-off that overlap, each with a workspace of its own."""
    say("case shared tiles streams")
    layers = [layer(q, *at, 7 + i) for i, at in enumerate(LAYERS)]
    ins = [inputs(f.tokens, f.width, 3) for f in layers]
    alone = [f(x, r.clone()).clone() for f, (x, r) in zip(layers, ins)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(20):
        at = [(i + j) % len(layers) for j in (0, 1 + i // len(layers))]       # every pair
        for k, s in zip(at, streams):
            with torch.cuda.stream(s):
                layers[k](ins[k][0], ins[k][1].clone())
        torch.cuda.synchronize()
        for k in at:
            assert torch.equal(layers[k].y, alone[k]), (i, k)


@pytest.mark.parametrize("m,n,k,tile,whole", [(130, 22016, 1280, 64, 512), (130, 16512, 1280, 128, 256), (300, 16512, 1280, 256, 256)])
def test_whole_and_shared_tiles_gated_to_e4m3(q, m, n, k, tile, whole):
    """More tiles than compute units: whole ones, and those of the last round shared by four or more workgroups."""
    g = torch.Generator(device="cuda").manual_seed(n)
    codes = lambda rows, size: (torch.randn((rows, k), generator=g, device="cuda") * size).clamp(-448, 448).to(F8)
    scales = lambda *s: torch.exp(0.5 * torch.randn(s, generator=g, device="cuda")) / 60
    ins = (codes(m, 60), scales(k // 128, m), codes(2 * n, 100), scales(2 * n // 128, k // 128) * k ** -0.5)
    p = q.w8a8_problem(m, n, k, q.DT_FP8_E4M3, gate=q.GATE_SILU, tile_hint=tile)
    assert f"whole={whole} " in q.w8a8_describe(p) and int(q.w8a8_describe(p).split("splits=")[1].split()[0]) >= 4
    y, s, p, ws = run_product(q, ins, n, "silu", "e4m3", tile_hint=tile)
    byte = lambda t: t.view(torch.uint8).cpu().numpy()
    want, tol = product_want(byte(ins[0]), ins[1].cpu().numpy(), byte(ins[2]), ins[3].cpu().numpy(), "silu", 2)
    product_check(y, s, want, tol, "e4m3")
    first, first_s = y.view(torch.uint8).clone(), s.clone()
    for _ in range(3):
        y.view(torch.uint8).zero_(), s.zero_()
        q.w8a8_run(p, *ins, y, s, ws)
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.uint8), first) and torch.equal(s, first_s)
    assert bool((ws[:4 << 17] == 0).all()), "tickets"
