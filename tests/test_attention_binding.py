"""The Python binding of the attention operators on the CPU: what it needs, and what it refuses before a pointer
reaches the library."""
import os
import shutil
import subprocess
import sys

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
