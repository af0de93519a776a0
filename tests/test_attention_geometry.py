"""Which tokens and rows a workgroup of the attention kernels takes (csrc/qgemm_attention_geometry.h, the
functions that the kernels themselves use), on the CPU against the same rules on whole numbers without a limit."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

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

    return (lambda *a: call(lib.geometry_seq, 5, *a)), (lambda *a: call(lib.geometry_tile, 4, *a))


def windows(g):
    return int(g.choice([0, 1, int(g.integers(2, 3000)), 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 1, LARGEST - 300, LARGEST - 1, LARGEST]))


def test_sequences_see_what_their_windows_leave(geometry):
    seq, _ = geometry
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
    _, tile = geometry
    g = np.random.default_rng([51, step])
    for _ in range(6000):
        BM, ratio, splits = int(g.choice([128, 256])), int(g.choice([1, 2, 3, 5, 8, 16, 64])), int(g.integers(1, 33))
        n, length = int(2 ** g.uniform(0, 13)), int(2 ** g.uniform(0, 17)) - 1
        row0 = int(g.integers(0, -(-ratio * n // BM))) * BM
        causal = bool(g.random() < 0.8)
        window = windows(g) if causal else 0
        lo, hi, per, active = tile(n, length, row0, BM, ratio, int(causal), window, step, splits)
        rows = range(row0, min(ratio * n, row0 + BM))
        places = [length - n + r // ratio for r in (rows[0], rows[-1])]
        last = max(min(length, places[1] + 1), 0) if causal else length
        first = max(places[0] - window + 1, 0) if window else 0
        case = (BM, ratio, splits, n, length, row0, causal, window)
        assert hi == last and lo % 16 == 0 and 0 <= lo <= hi, case
        assert lo <= first or first >= hi, case
        assert 1 <= active <= splits and per >= 1, case
        assert lo + per * active * step >= hi, case
        assert active == 1 or lo + per * (active - 1) * step < hi, case


def test_the_largest_window_is_no_window(geometry):
    # 2048 queries of four heads a kv head, one part: all 32 steps of the last row tile are in it
    seq, tile = geometry
    for window in (0, LARGEST - 100, LARGEST):
        assert tile(2048, 2048, 7936, 256, 4, 1, window, 64, 1) == [0, 2048, 32, 1]
        assert tile(200, 100, 0, 256, 1, 1, window, 64, 1) == [0, 100, 2, 1]      # more queries than tokens
        assert seq(0, 200, 100, 200, 200, 1 << 20, window) == [0, 200, 100, 0, 100]
