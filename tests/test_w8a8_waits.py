"""The rows kernel's waits for its loads, read from the assembly that the build's flags give: a wait counts the loads issued
after those it is for, so it holds only as long as the compiler keeps the loads of one stage together."""
import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "weight_only_quantized_qgemm_amd")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """(wavefronts, loads of tokens, gate, 8-bit output) -> the kernel's instructions and labels."""
    if not shutil.which(HIPCC):
        pytest.skip("no hipcc")
    sys.path.insert(0, PKG)
    try:
        import _build
    finally:
        sys.path.pop(0)
    to = tmp_path_factory.mktemp("rows") / "rows.s"
    subprocess.run([HIPCC, *_build.HIPCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-S", "--offload-device-only",
                    os.path.join(PKG, "csrc", "qgemm_w8a8_rows.hip"), "-o", str(to)], check=True, capture_output=True, timeout=600)
    found = re.findall(r"^_ZN\S*rows_kernelILi(\d+)ELi(\d+)ELi(\d+)ELb(\d)\S*:\s.*?\n(.*?)s_endpgm", to.read_text(), re.S | re.M)
    return {tuple(map(int, f[:4])): [l.split(";")[0].strip() for l in f[4].splitlines()] for f in found}


def stage_loads(kernel):
    """Of one k block: (loads into LDS, loads of scales)."""
    _, tokens, gate, _ = kernel
    sides = 2 if gate else 1
    return 2 * sides + tokens, sides + (tokens + 1) // 2


def prologue_and_loop(lines):
    """Instructions before the k loop, and those of the loop: from the label that the first branch back goes to, to that branch."""
    at = {}
    for i, l in enumerate(lines):
        m = re.match(r"(\.LBB\w+):", l)
        if m:
            at[m[1]] = i
        m = re.match(r"s_cbranch_\w+ (\.LBB\w+)", l)
        if m and m[1] in at:
            return lines[:at[m[1]]], lines[at[m[1]]:i]
    raise AssertionError("no loop")


def loads(lines):
    """'L' for a load into LDS, 's' for one of a scale, in order."""
    return "".join("L" if l.endswith(" lds") else "s" for l in lines if l.startswith("buffer_load"))


def test_every_instance_was_found(kernels):
    assert len(kernels) == 3 * 6 + 2 * 5                                     # a gate has two outputs; without one, up to 32 tokens, 4 or 8 wavefronts
    for k, lines in kernels.items():
        _, loop = prologue_and_loop(lines)
        assert len(loads(loop)) == 2 * sum(stage_loads(k)), k                # two k blocks, none of their loads repeated
        assert not any("scratch_" in l for l in lines), k


def test_first_loads_come_stage_by_stage(kernels):
    for k, lines in kernels.items():
        into_lds, scales = stage_loads(k)
        order = loads(prologue_and_loop(lines)[0])
        first, second = order[:into_lds + scales], order[into_lds + scales:]
        assert len(order) == 2 * (into_lds + scales), (k, order)
        assert first.count("L") == second.count("L") == into_lds, (k, order)


def test_each_stage_waits_for_itself_alone(kernels):
    """In a round of the loop one wait for each stage, while all loads of the other are on their way: nothing else waits for loads
    (as it did where the scales' product was moved up to the other stage's)."""
    for k, lines in kernels.items():
        each, loop = sum(stage_loads(k)), prologue_and_loop(lines)[1]
        waits = [i for i, l in enumerate(loop) if l.startswith("s_waitcnt") and "vmcnt" in l]
        assert [re.search(r"vmcnt\((\d+)\)", loop[i])[1] for i in waits] == [str(each)] * 2, k
        assert not loads(loop[:waits[0]]) and len(loads(loop[waits[0]:waits[1]])) == each, k
