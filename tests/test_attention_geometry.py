"""Which tokens and rows a workgroup of the attention kernels takes (csrc/qgemm_attention_geometry.h, the
functions that the kernels themselves use), on the CPU against the same rules on whole numbers without a limit."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import weight_only_quantized_qgemm_amd as q

HERE = os.path.dirname(os.path.abspath(__file__))
LARGEST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def geometry(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("geometry") / "geometry.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-Wall", "-shared", "-fPIC", os.path.join(HERE, "attention_geometry.cpp"),
                    "-o", lib], check=True)
    lib = ctypes.CDLL(lib)

    def call(f, n, *args):
        out = (ctypes.c_int * n)()
        f(*args, out)
        return list(out)

    lib.geometry_claimed.restype = ctypes.c_uint
    return (lambda *a: call(lib.geometry_seq, 5, *a)), (lambda *a: call(lib.geometry_tile, 5, *a)), lib.geometry_claimed


def windows(g):
    return int(g.choice([0, 1, int(g.integers(2, 3000)), 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 1, LARGEST - 300, LARGEST - 1, LARGEST]))


def test_sequences_see_what_their_windows_leave(geometry):
    seq = geometry[0]
    g = np.random.default_rng(50)
    for _ in range(4000):
        n, length = (int(2 ** g.uniform(0, top)) - 1 for top in (24, 30))
        window = windows(g)
        start, count, tokens, lo, hi = seq(5, 5 + n, length, 2 ** 24, 2 ** 24, 2 ** 30, window)
        assert (start, count, tokens, hi) == (5, min(n, 2 ** 24 - 5), length, length)
        # the first token that the first query's window leaves, or 0
        want = max(length - count - window + 1, 0) if window else 0
        assert lo == min(want // 16, hi // 16) * 16, (n, length, window)


@pytest.mark.parametrize("step", [32, 64])
def test_parts_cover_each_row_tile(geometry, step):
    # every token that a row of the tile sees lies in one of the parts, and there are no more parts than workgroups
    tile = geometry[1]
    g = np.random.default_rng([51, step])
    for _ in range(6000):
        BM, ratio, splits = int(g.choice([128, 256])), int(g.choice([1, 2, 3, 5, 8, 16, 64])), int(g.integers(1, 33))
        n, length = int(2 ** g.uniform(0, 13)), int(2 ** g.uniform(0, 17)) - 1
        row0 = int(g.integers(0, -(-ratio * n // BM))) * BM
        causal = bool(g.random() < 0.8)
        window = windows(g) if causal else 0
        lo, hi, per, active, seen = tile(n, length, row0, BM, ratio, int(causal), window, step, splits)
        rows = range(row0, min(ratio * n, row0 + BM))
        places = [length - n + r // ratio for r in (rows[0], rows[-1])]
        last = max(min(length, places[1] + 1), 0) if causal else length
        first = max(places[0] - window + 1, 0) if window else 0
        case = (BM, ratio, splits, n, length, row0, causal, window)
        assert hi == last and lo % 16 == 0 and 0 <= lo <= hi, case
        assert seen == first and (lo <= first or first >= hi), case
        assert 1 <= active <= splits and per >= 1, case
        assert lo + per * active * step >= hi, case
        assert active == 1 or lo + per * (active - 1) * step < hi, case


def test_the_largest_window_is_no_window(geometry):
    # 2048 queries of four heads a kv head, one part: all 32 steps of the last row tile are in it
    seq, tile, _ = geometry
    for window in (0, LARGEST - 100, LARGEST):
        assert tile(2048, 2048, 7936, 256, 4, 1, window, 64, 1) == [0, 2048, 32, 1, 0]
        assert tile(200, 100, 0, 256, 1, 1, window, 64, 1) == [0, 100, 2, 1, 0]   # more queries than tokens
        assert seq(0, 200, 100, 200, 200, 1 << 20, window) == [0, 200, 100, 0, 100]


def planned(batch, total_q, max_q, q_heads, kv_heads, dim, group, dtype, max_pages, hint):
    """Rows of a row tile, and the row tiles per kv head that the launch and its workspace are made for."""
    p = q.attention_problem(q.cache(64, 16, kv_heads, dim, dtype, group_size=group), batch, total_q, q_heads, max_q, max_pages,
                            kernel_hint=hint)
    f = dict(x.split("=") for x in q.attention_describe(p).split()[1:])
    return int(f["rows"]), int(f["grid"]) // kv_heads // int(f["splits"])


def claimed(geometry, n):
    return geometry[2]((ctypes.c_int * len(n))(*n), len(n))


def test_row_tiles_fit_the_launch_unless_too_many_rows_are_claimed(geometry):
    # whatever stands in q_start: no more row tiles than planned, so none's tickets or partial results lie past
    # the workspace, or more rows than total_q, where the kernels compute nothing
    seq = geometry[0]
    g = np.random.default_rng(52)
    over = 0
    for case in range(3000):
        batch, max_q = int(2 ** g.uniform(0, 6)), int(2 ** g.uniform(0, 11))
        total = int(g.integers(max_q, batch * max_q + 1))
        ratio, kv, dim = int(g.choice([1, 3, 4, 8])), int(g.choice([1, 2, 8])), int(g.choice([64, 128, 256]))
        rows, tiles = planned(batch, total, max_q, ratio * kv, kv, dim, dim, int(g.integers(0, 2)), int(2 ** g.uniform(0, 10)),
                              q.ATTENTION_TILES)
        starts = g.integers(-100, total + 100, batch + 1)
        if case % 3:
            starts = np.sort(starts)
        if case % 3 == 1:                                             # padded with zeros
            starts[int(g.integers(1, batch + 1)):] = 0
        if g.random() < 0.2:
            starts[-1] = LARGEST
        n = [seq(int(a), int(b), 500, total, max_q, 1 << 20, 0)[1] for a, b in zip(starts, starts[1:])]
        rising = bool(np.all(np.diff(starts) >= 0))
        assert min(n) >= 0 and claimed(geometry, n) == sum(n) and (sum(n) <= total or not rising)
        if sum(n) > total:
            over += 1
        else:
            assert sum(-(-ratio * x // rows) for x in n) <= tiles
    assert over > 100
    # sums far past 32 bits stay above any total_q
    assert claimed(geometry, [1 << 24] * 65535) == 1 << 30 and claimed(geometry, [1 << 24] * 64) == 1 << 30


@pytest.mark.parametrize("starts,total,max_q", [([0, 1000, 0, 1000, 0], 1000, 1000), ([0, 900, 0, 900, 0, 900, 0, 900, 0], 1000, 900)])
def test_starts_that_claim_too_much_count_more_tiles_than_planned(geometry, starts, total, max_q):
    n = [geometry[0](a, b, 500, total, max_q, 1 << 20, 0)[1] for a, b in zip(starts, starts[1:])]
    rows, tiles = planned(len(starts) - 1, total, max_q, 32, 8, 128, 128, q.DT_F16, 200, q.ATTENTION_TILES)
    assert sum(-(-4 * x // rows) for x in n) > tiles and claimed(geometry, n) > total


# ----------------------------------------------------------------------------- the choice of kernel
@pytest.mark.parametrize("batch,kv_heads,pages", [(4096, 32, 1 << 16), (1024, 32, 1 << 18), (65535, 8, 1 << 15), (65535, 64, 1 << 13)])
def test_problems_beyond_the_rows_kernel_go_to_the_tiles_kernel(batch, kv_heads, pages):
    # one token a request over tables so wide that the rows kernel could not number all their units
    c = q.cache(1 << 20, 16, kv_heads, 128, q.DT_BF16)
    p = q.attention_problem(c, batch, batch, 4 * kv_heads, 1, pages)
    assert q.attention_describe(p).startswith("tiles ") and q.attention_workspace_bytes(p) == 0
    asked = q.attention_problem(c, batch, batch, 4 * kv_heads, 1, pages, kernel_hint=q.ATTENTION_ROWS)
    with pytest.raises(q.QgemmError, match="row tiles") as e:
        q.attention_describe(asked)
    assert e.value.status == q.ERR_UNSUPPORTED
    narrow = q.attention_problem(c, batch, batch, 4 * kv_heads, 1, pages // 64)
    assert q.attention_describe(narrow).startswith("rows ")


# ----------------------------------------------------------------------------- launch limits
def test_launches_of_too_many_work_items_are_refused():
    # a launch holds less than 2^32 work-items; calls beyond that are refused by the host, not by the runtime
    def text(status):
        assert status == q.ERR_UNSUPPORTED, q.last_error()
        assert "more than one launch allows" in q.last_error()

    tokens, a = 1 << 24, 0x100000
    for heads, dim in ((64, 128), (128, 64), (32, 256), (1024, 64)):
        p = q.NormRope(tokens, heads, heads, dim, 0, 0, q.DT_F16, 0, 1, 1e-6, 0)
        row = heads * dim
        text(q.lib.qgemm_qk_norm_rope(ctypes.byref(p), a, row, a, row, None, None, None, None, a, row, a, row, None))
    for heads, dim in ((16, 128), (32, 64), (8, 256), (1024, 64)):
        c, row = q.cache(1 << 20, 16, heads, dim, q.DT_F16), heads * dim
        text(q.lib.qgemm_cache_write(ctypes.byref(c), a, a, row, a, row, a, tokens, None))
        text(q.lib.qgemm_cache_read(ctypes.byref(c), a, a, tokens, a, a, None))
    for heads, dim, batch in ((512, 64, 65535), (1024, 128, 16384), (1024, 256, 65535)):
        p = q.attention_problem(q.cache(1 << 20, 16, heads, dim, q.DT_F16), batch, batch, heads, 1, 4, kernel_hint=q.ATTENTION_TILES)
        n = ctypes.c_size_t()
        text(q.lib.qgemm_attention_workspace_bytes(ctypes.byref(p), ctypes.byref(n)))
