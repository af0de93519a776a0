"""One attention layer of a language model in 4 bits, from the library's operators:

  INT4 product (q, k and v of every token) -> head norm and rotation -> 4-bit paged cache ->
  attention over the cache -> INT4 product (output)

run for prompts of different lengths at once and then token by token, as a serving program would:
the lengths, slots and pages lie in device memory, so one captured graph serves every decode step.

  python example_attention.py [--batch 8] [--prompt 1000] [--steps 64]

prints the time of the prompt pass and of a decode step, eager and from the graph.  Weights and
hidden states are random.
"""
import argparse
import time

import numpy as np
import torch

import weight_only_quantized_qgemm_amd as q


class Linear:
    """An INT4 weight laid out once; the descriptors and workspaces of each row count are kept."""

    def __init__(self, w_nk, group=128):
        self.n, self.k = w_nk.shape
        self.group, self.plans = group, {}
        p = q.problem(1, self.n, self.k, "int4", group_size=group)
        codes, scales, _ = q.quantize(p, w_nk)
        self.w, self.s = (torch.from_numpy(a).cuda() for a in q.pack(p, codes, scales))

    def __call__(self, x, out):
        m = x.shape[0]
        if m not in self.plans:
            p = q.problem(m, self.n, self.k, "int4", group_size=self.group)
            self.plans[m] = p, q.alloc_workspace(p)
        p, ws = self.plans[m]
        q.run(p, x, self.w, self.s, None, out, ws)
        return out


def rotation_table(rot, max_pos, base=10000.0):
    """cos | sin of every position's rot / 2 angles, fp32 [max_pos, rot]."""
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    return torch.cat((angle.cos(), angle.sin()), -1).float().cuda()


class Tokens:
    """The new tokens of a batch of requests and where their context lies, all in device memory."""

    def __init__(self, table, q_lens, k_lens, page):
        """table [batch, pages] int32: each request's pages in order.  k_lens count the new tokens too."""
        n = [j for k, m in zip(k_lens, q_lens) for j in range(k - m, k)]
        row = [b for b, m in enumerate(q_lens) for _ in range(m)]
        self.page, self.table, self.max_q = page, table, max(q_lens)
        self.batch, self.total = len(q_lens), len(n)
        self.lens = torch.tensor(k_lens, dtype=torch.int32, device="cuda")
        self.starts = torch.tensor(np.concatenate(([0], np.cumsum(q_lens))), dtype=torch.int32, device="cuda")
        self.positions = torch.tensor(n, dtype=torch.int32, device="cuda")
        at = torch.tensor(n, device="cuda")
        self.slots = table[torch.tensor(row, device="cuda"), at // page].long() * page + at % page

    def advance(self):
        """One more token for every request (decode): three small device updates, no host value."""
        self.positions.copy_(self.lens)
        at = self.lens.long()
        self.slots.copy_(self.table.gather(1, (at // self.page)[:, None])[:, 0].long() * self.page + at % self.page)
        self.lens.add_(1)


class AttentionLayer:
    def __init__(self, w_qkv, w_out, q_norm, k_norm, table, q_heads, kv_heads, head_dim, pages, page_size, group_size=None,
                 window=0):
        self.heads, self.dim, self.window = (q_heads, kv_heads), head_dim, window
        self.qkv, self.out = Linear(w_qkv), Linear(w_out)
        self.q_norm, self.k_norm, self.table = q_norm, k_norm, table
        self.cache = q.cache(pages, page_size, kv_heads, head_dim, q.DT_F16, group_size=group_size)
        self.data = q.alloc_cache(self.cache)
        self.plans = {}

    def plan(self, t):
        """Descriptors, workspace and buffers of a call's shape (the lengths themselves may change)."""
        key = t.batch, t.total, t.max_q, t.table.shape[1]
        if key not in self.plans:
            hq, hk = self.heads
            rope = q.norm_rope_problem(t.total, hq, hk, self.dim, rot_dim=self.table.shape[1], max_pos=self.table.shape[0])
            attn = q.attention_problem(self.cache, t.batch, t.total, hq, t.max_q, t.table.shape[1], causal=True,
                                       window=self.window)
            qkv = torch.empty((t.total, hq + 2 * hk, self.dim), dtype=torch.float16, device="cuda")
            self.plans[key] = dict(
                rope=rope, attn=attn, ws=q.alloc_attention_workspace(attn), qkv=qkv, q=qkv[:, :hq], k=qkv[:, hq:hq + hk],
                v=qkv[:, hq + hk:], heads=torch.empty((t.total, hq, self.dim), dtype=torch.float16, device="cuda"),
                out=torch.empty((t.total, self.out.n), dtype=torch.float16, device="cuda"))
        return self.plans[key]

    def project(self, b, x):
        self.qkv(x, b["qkv"].view(x.shape[0], -1))

    def rotate(self, b, t):                                  # in place, inside the product's output
        q.qk_norm_rope(b["rope"], b["q"], b["k"], self.q_norm, self.k_norm, t.positions, self.table, b["q"], b["k"])

    def store(self, b, t):
        q.cache_write(self.cache, self.data, b["k"], b["v"], t.slots)

    def attend(self, b, t):
        q.attention(b["attn"], b["q"], self.data, t.table, t.lens, t.starts, b["heads"], b["ws"])

    def output(self, b):
        return self.out(b["heads"].view(b["heads"].shape[0], -1), b["out"])

    def __call__(self, x, t):
        """x [total, width] of the new tokens -> [total, width]; their keys and values join the cache."""
        b = self.plan(t)
        self.project(b, x)
        self.rotate(b, t)
        self.store(b, t)
        self.attend(b, t)
        return self.output(b)


def random_layer(width, q_heads, kv_heads, head_dim, pages, page_size, group_size=None, rot=None, max_pos=32768, window=0, seed=0):
    g = np.random.default_rng(seed)
    n = (q_heads + 2 * kv_heads) * head_dim
    norm = [torch.from_numpy((1 + 0.2 * g.standard_normal(head_dim)).astype(np.float16)).cuda() for _ in "qk"]
    w = [(g.standard_normal(s, dtype=np.float32) * s[1] ** -0.5) for s in ((n, width), (width, q_heads * head_dim))]
    return AttentionLayer(*w, *norm, rotation_table(head_dim if rot is None else rot, max_pos), q_heads, kv_heads, head_dim, pages,
                          page_size, group_size, window)


def capture(layer, x, t):
    """A graph of one decode step: advance, then the layer.  Returns it and its output buffer."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = [a.clone() for a in (t.lens, t.positions, t.slots)]
    with torch.cuda.stream(side):                            # plans and workspaces exist before the capture
        t.advance()
        layer(x, t)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.advance()
        out = layer(x, t)
    for a, b in zip((t.lens, t.positions, t.slots), keep):       # the slots written so far are written again
        a.copy_(b)
    return graph, out


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1000, help="longest prompt; the requests' lengths fall from there to a half")
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--page", type=int, default=64)
    a = ap.parse_args()
    width, hq, hk, dim = 4096, 32, 8, 128
    each = -(-(a.prompt + 2 * a.steps + 2) // a.page)
    layer = random_layer(width, hq, hk, dim, each * a.batch, a.page)
    table = torch.randperm(each * a.batch, device="cuda").to(torch.int32).view(a.batch, each)
    lens = [max(1, a.prompt - i * a.prompt // (2 * a.batch)) for i in range(a.batch)]
    hidden = torch.randn((sum(lens), width), device="cuda").half()

    def timed(run, n):
        torch.cuda.synchronize()
        start = time.perf_counter()
        for _ in range(n):
            run()
        torch.cuda.synchronize()
        return (time.perf_counter() - start) / n * 1e6

    prompt = Tokens(table, lens, lens, a.page)
    layer(hidden, prompt)
    print(f"prompt: {sum(lens)} tokens of {a.batch} requests, {timed(lambda: layer(hidden, prompt), 5):.0f} us")
    x = hidden[:a.batch].contiguous()
    step = Tokens(table, [1] * a.batch, lens, a.page)        # lens: the context before the first step

    def eager():
        step.advance()
        layer(x, step)

    eager()
    print(f"decode: {timed(eager, a.steps):.1f} us a step, each operator called on its own")
    graph, out = capture(layer, x, step)
    print(f"decode: {timed(graph.replay, a.steps):.1f} us a step from a captured graph; output finite: "
          f"{bool(torch.isfinite(out).all())}")


if __name__ == "__main__":
    main()
