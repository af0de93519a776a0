"""The 8-bit operators together, as the feed-forward half of a decoder layer:

  residual addition + RMS norm -> e4m3 -> gated pair -> e4m3 -> product -> residual addition + RMS norm (16 bits)

each against the 64-bit oracle on what the one before it gave, eager and as a captured graph that is replayed with new
tokens, with the calls of two layers on two streams at once, and beside the 4-bit attention layer's products."""
import numpy as np
import pytest

from gpu_cases import say
from oracle import w8a8
from test_gpu_w8a8 import F8, f64, norm_check, product_check, product_want

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_qgemm_amd as q
    return q


class FeedForward:
    """Weights laid out once; buffers and workspace of one number of tokens."""

    def __init__(self, q, tokens, width, inner, seed):
        g = np.random.default_rng(seed)
        self.q, self.tokens, self.width, self.inner = q, tokens, width, inner
        self.up = q.w8a8_problem(tokens, inner, width, q.DT_FP8_E4M3, gate=q.GATE_SILU)
        self.down = q.w8a8_problem(tokens, width, inner, q.DT_BF16)
        self.first = q.add_norm_problem(tokens, width, q.DT_BF16, q.DT_FP8_E4M3)
        self.last = q.add_norm_problem(tokens, width, q.DT_BF16)
        put = lambda p, w: [torch.from_numpy(x).cuda() for x in q.w8a8_quantize(p, w.astype(np.float32))]
        self.w_up, self.s_up = put(self.up, g.standard_normal((2 * inner, width)) * width ** -0.5)
        self.w_down, self.s_down = put(self.down, g.standard_normal((width, inner)) * inner ** -0.5)
        self.w_up, self.w_down = self.w_up.view(F8), self.w_down.view(F8)
        self.g1, self.g2 = (torch.from_numpy(1 + 0.2 * g.standard_normal(width)).bfloat16().cuda() for _ in range(2))
        new = lambda n, t=torch.bfloat16: torch.empty((tokens, n), dtype=t, device="cuda")
        self.h, self.h_s = new(width, F8), torch.empty((width // 128, tokens), device="cuda")
        self.m, self.m_s = new(inner, F8), torch.empty((inner // 128, tokens), device="cuda")
        self.o, self.y, self.after = new(width), new(width), new(width)
        self.ws = torch.zeros(max(q.w8a8_workspace_bytes(p) for p in (self.up, self.down)) or 256, dtype=torch.uint8, device="cuda")

    def __call__(self, x, stream_of_residual):
        """x is added to the residual stream in place; y gets the next part's input."""
        q = self.q
        q.add_norm(self.first, x, stream_of_residual, self.g1, stream_of_residual, self.h, self.h_s)
        q.w8a8_run(self.up, self.h, self.h_s, self.w_up, self.s_up, self.m, self.m_s, self.ws)
        q.w8a8_run(self.down, self.m, self.m_s, self.w_down, self.s_down, self.o, None, self.ws)
        q.add_norm(self.last, self.o, stream_of_residual, self.g2, self.after, self.y)
        return self.y


def inputs(tokens, width, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn((tokens, width), generator=g).bfloat16().cuda() for _ in range(2)]


@pytest.mark.parametrize("tokens", [1, 7, 16, 33, 200])
def test_stage_by_stage(q, tokens):
    say(f"case feed-forward {tokens}")
    f = FeedForward(q, tokens, 512, 896, 5)
    x, r = inputs(tokens, 512, tokens)
    x0, r0 = x.cpu(), r.cpu()
    f(x, r)
    torch.cuda.synchronize()
    norm_check(x0, r0, f.g1.cpu(), True, 1e-6, "bf16", "e4m3", r, f.h, f.h_s)
    byte = lambda t: t.view(torch.uint8).cpu().numpy()
    want, tol = product_want(byte(f.h), f.h_s.cpu().numpy(), byte(f.w_up), f.s_up.cpu().numpy(), "silu", 2)
    product_check(f.m, f.m_s, want, tol, "e4m3")
    want, tol = product_want(byte(f.m), f.m_s.cpu().numpy(), byte(f.w_down), f.s_down.cpu().numpy(), "none", 1)
    product_check(f.o, None, want, tol, "bf16")
    norm_check(f.o.cpu(), r.cpu(), f.g2.cpu(), True, 1e-6, "bf16", "bf16", f.after, f.y, None)
    # and the whole of it near the unquantized formula: e4m3 rounds to 2^-4 at most, its errors average over the sums
    xs = f64(x0) + f64(r0)
    h = xs / np.sqrt((xs * xs).mean(1, keepdims=True) + 1e-6) * f64(f.g1.cpu())
    w = w8a8.weight_values(byte(f.w_up), f.s_up.cpu().numpy(), 2)
    p = h @ w.T
    m = w8a8.act(p[:, :896], "silu") * p[:, 896:]
    o = m @ w8a8.weight_values(byte(f.w_down), f.s_down.cpu().numpy()).T
    assert np.linalg.norm(f64(f.o) - o) <= 2.0 ** -4 * np.linalg.norm(o)


@pytest.mark.parametrize("tokens", [1, 16, 40, 300])
def test_captured_replays_equal_eager_calls(q, tokens):
    say(f"case feed-forward graph {tokens}")
    f = FeedForward(q, tokens, 384, 640, 6)
    x, r = inputs(tokens, 384, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f(x, r)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(x, r)
    for seed in range(2, 6):
        x1, r1 = inputs(tokens, 384, seed)
        x.copy_(x1), r.copy_(r1)
        y = f(x, r).clone()
        total, after = r.clone(), f.after.clone()
        torch.cuda.synchronize()
        f.y.zero_(), f.after.zero_()
        x.copy_(x1), r.copy_(r1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(f.y, y) and torch.equal(r, total) and torch.equal(f.after, after), seed


def test_two_streams_at_once(q):
    """Calls that overlap, each with a workspace of its own."""
    say("case feed-forward streams")
    layers = [FeedForward(q, t, 512, 896, 7 + t) for t in (40, 16)]
    ins = [inputs(f.tokens, 512, 3) for f in layers]
    alone = []
    for f, (x, r) in zip(layers, ins):
        alone.append(f(x, r.clone()).clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(20):
        for f, (x, r), s in zip(layers, ins, streams):
            with torch.cuda.stream(s):
                f(x, r.clone())
        torch.cuda.synchronize()
        for f, want in zip(layers, alone):
            assert torch.equal(f.y, want)


def test_norm_feeds_a_4_bit_product(q):
    """The 16-bit form between two weight-only products: the same bytes as the product of the norm's output."""
    say("case norm into int4")
    t, width, n = 19, 256, 512
    g = np.random.default_rng(2)
    p = q.problem(t, n, width, "int4", group_size=128)
    codes, scales, _ = q.quantize(p, (g.standard_normal((n, width)) * 0.05).astype(np.float32))
    w, s = (torch.from_numpy(a).cuda() for a in q.pack(p, codes, scales))
    x = torch.from_numpy(g.standard_normal((t, width)).astype(np.float16)).cuda()
    r = torch.from_numpy(g.standard_normal((t, width)).astype(np.float16)).cuda()
    y, total = torch.empty_like(x), torch.empty_like(x)
    out = torch.empty((t, n), dtype=torch.float16, device="cuda")
    q.add_norm(q.add_norm_problem(t, width), x, r, None, total, y)
    q.run(p, y, w, s, None, out, q.alloc_workspace(p))
    torch.cuda.synchronize()
    norm_check(x.cpu(), r.cpu(), None, True, 1e-6, "f16", "f16", total, y, None)
    sd = scales.view(np.float16).astype(np.float64)                            # [K / 128, N]
    v = np.stack([codes & 15, codes >> 4], -1).reshape(n, width).astype(np.float64) - 8
    wd = (v * np.repeat(sd.T, 128, 1)).astype(np.float16).astype(np.float64)
    want = f64(y) @ wd.T
    assert np.all(np.abs(f64(out) - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + width * 2.0 ** -24 * (np.abs(f64(y)) @ np.abs(wd).T))
