"""The Python binding of the attention operators on the CPU: what it needs, and what it refuses before a pointer
reaches the library."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

import weight_only_quantized_qgemm_amd as q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "weight_only_quantized_qgemm_amd")


def test_products_do_not_need_the_compiled_calls(tmp_path):
    # a package without the _calls module: it imports and packs weights, and the first attention call says what is missing
    pkg = tmp_path / "weight_only_quantized_qgemm_amd"
    pkg.mkdir()
    shutil.copy(os.path.join(PKG, "__init__.py"), pkg)
    code = """
import numpy as np, torch
import weight_only_quantized_qgemm_amd as q
assert q.__file__.startswith(%r)
p = q.problem(1, 64, 256, "int4")
codes, scales, _ = q.quantize(p, np.ones((64, 256), np.float32))
assert q.pack(p, codes, scales)[0].size
c = q.cache(1, 16, 2, 64)
assert q.cache_bytes(c)
try:
    q.cache_read(c, torch.zeros(1), torch.zeros(1), None, None)
except ImportError as e:
    assert "_calls" in str(e) and "_build" in str(e)
    print("told")
""" % str(tmp_path)
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=str(tmp_path), QGEMM_LIB_PATH=q.LIB_PATH))
    assert r.returncode == 0 and "told" in r.stdout, r.stderr[-2000:]


def test_first_calls_of_many_threads():
    # the module is set up once, and no thread sees it before that
    code = """
import threading, torch
import weight_only_quantized_qgemm_amd as q
c = q.cache(1, 16, 2, 64)
seen, start = [], threading.Barrier(8)
def call():
    start.wait()
    try:
        q.cache_write(c, torch.zeros(5, dtype=torch.uint8), torch.zeros(1, 2, 64).half(), torch.zeros(1, 2, 64).half(), torch.zeros(1).long())
    except ValueError as e:
        seen.append(str(e))
t = [threading.Thread(target=call) for _ in range(8)]
[x.start() for x in t], [x.join() for x in t]
assert len(seen) == 8 and all("data must be" in s for s in seen), seen
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


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


def calls(at):
    """Each call's function and its arguments by name, at(name, tensor) in place of each tensor."""
    half, i32 = torch.float16, torch.int32
    x, kv = torch.zeros(3, 4, 64, dtype=half), torch.zeros(3, 2, 64, dtype=half)
    c = q.cache(4, 16, 2, 64)
    data, slots = torch.zeros(q.cache_bytes(c), dtype=torch.uint8), torch.zeros(3, dtype=torch.int64)
    w, lens = torch.ones(64, dtype=half), torch.zeros(2, dtype=i32)
    p = q.attention_problem(c, 1, 3, 4, 3, 2)
    r = q.norm_rope_problem(3, 4, 2, 64, max_pos=8)
    found = [
        (q.qk_norm_rope, dict(p=r), dict(q=x, k=kv, q_weight=w, k_weight=w, positions=torch.zeros(3, dtype=i32),
                                         cos_sin=torch.zeros(8, 64), q_out=x, k_out=kv)),
        (q.cache_write, dict(c=c), dict(data=data, k=kv, v=kv, slots=slots)),
        (q.cache_read, dict(c=c), dict(data=data, slots=slots, k_out=kv, v_out=kv)),
        (q.attention, dict(p=p), dict(q=x, data=data, page_table=torch.zeros(1, 2, dtype=i32), seq_lens=lens, q_start=lens, out=x,
                                      workspace=torch.zeros(1 << 20, dtype=torch.uint8)))]
    return [(f, dict(fixed, **{n: at(n, v) for n, v in t.items()}), list(t)) for f, fixed, t in found]


@pytest.mark.parametrize("stream", [None, 0])
def test_tensors_on_the_host_are_refused(stream):
    for f, args, names in calls(lambda n, t: t):
        with pytest.raises(ValueError, match="on the GPU"):
            f(**args, stream=stream)


def test_one_tensor_elsewhere_is_refused():
    for i in range(4):
        for odd in calls(lambda n, t: t)[i][2]:
            for device, text in ((-1, f"{odd} must be on the GPU"), (1, "on device")):
                f, args, _ = calls(lambda n, t: Elsewhere(t, device if n == odd else 0))[i]
                with pytest.raises(ValueError, match=text):
                    f(**args, stream=0)


def test_pinned_tensors_pass():
    # the GPU reads them where they lie: the next wrong tensor is named
    f, args, _ = calls(lambda n, t: Elsewhere(t, -1 if n == "seq_lens" else 0, n == "seq_lens"))[3]
    with pytest.raises(ValueError, match="^out is on device 1, q on device 0"):
        f(**dict(args, out=Elsewhere(args["out"].x, 1)), stream=0)


def test_page_tables_of_another_width_and_loose_workspaces_are_refused():
    f, args, _ = calls(lambda n, t: Elsewhere(t, 0))[3]
    # of several requests; one request's row may be longer, and a flat table is taken as it is
    two = dict(args, p=q.attention_problem(args["p"].cache, 2, 3, 4, 3, 2), q_start=Elsewhere(torch.zeros(3, dtype=torch.int32), 0))
    for wide in (torch.zeros(2, 3, dtype=torch.int32), torch.zeros(4, 1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="max_pages = 2 columns"):
            f(**dict(two, page_table=Elsewhere(wide, 0)), stream=0)
    loose = Elsewhere(torch.zeros(2 << 20, dtype=torch.uint8)[::2], 0)
    for taken in (dict(args, page_table=Elsewhere(torch.zeros(1, 3, dtype=torch.int32), 0)),
                  dict(two, page_table=Elsewhere(torch.zeros(4, dtype=torch.int32), 0))):
        with pytest.raises(ValueError, match="workspace"):               # the check after the table's
            f(**dict(taken, workspace=loose), stream=0)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        f(**dict(args, workspace=Elsewhere(torch.zeros(2 << 20, dtype=torch.uint8)[::2], 0)), stream=0)
