"""Calls of the 8-bit operators that the C ABI refuses beside those of a single argument (nothing is launched)."""
import ctypes

import numpy as np
import pytest

import weight_only_quantized_qgemm_amd as q

# M = 4, N = K = 256: where each argument of a gated call to e4m3 lies, and its bytes
AT = dict(A=0x100000, sa=0x200000, W=0x300000, sw=0x400000, out=0x500000, so=0x600000, ws=0x700000)
BYTES = dict(A=4 * 256, sa=4 * 2 * 4, W=512 * 256, sw=4 * 2 * 4, out=4 * 256, so=4 * 2 * 4, ws=0)
NAMES = dict(A="A", sa="a_scales", W="W", sw="w_scales", out="out", so="out_scales", ws="workspace")


def call(p, **at):
    c = dict(AT, **at)
    return q.lib.qgemm_w8a8_run(ctypes.byref(p), c["A"], c["sa"], c["W"], c["sw"], c["out"], c["so"], c["ws"], 1 << 24, None)


@pytest.mark.parametrize("written", ["out", "so", "ws"])
@pytest.mark.parametrize("other", list(AT))
def test_outputs_on_other_arguments_are_refused(written, other):
    """A gated product to e4m3 with N = K has outputs of its activations' shape and type."""
    if written == other:
        return
    p = q.w8a8_problem(4, 256, 256, q.DT_FP8_E4M3, gate=q.GATE_SILU)
    size = dict(BYTES, ws=q.w8a8_workspace_bytes(p))
    align = dict(out=16, so=4, ws=256)[written]
    last = (size[other] - 1) // align * align                                 # begins on the other's last bytes, or ends on its first
    before = -((size[written] - 1) // align * align)
    for distance in {0, last, before}:
        assert call(p, **{written: AT[other] + distance}) == q.ERR_INVALID_ARGUMENT, (written, other, distance)
        assert "overlaps" in q.last_error() and NAMES[written] in q.last_error() and NAMES[other] in q.last_error()


def test_a_16_bit_output_on_its_activations_is_refused():
    p = q.w8a8_problem(4, 128, 256, q.DT_BF16)
    assert call(p, out=AT["A"], so=None) == q.ERR_INVALID_ARGUMENT and "out overlaps A" in q.last_error()


def test_sums_are_checked():
    for bad in (-1, 2):
        p = q.w8a8_problem(4, 256, 256, sums=bad)
        assert call(p, so=None) == q.ERR_INVALID_ARGUMENT and "sums" in q.last_error()
        with pytest.raises(q.QgemmError, match="sums"):
            q.w8a8_describe(p)
    whole = q.w8a8_problem(200, 256, 256, sums=q.W8A8_SUMS_WHOLE)
    assert "operands=16" in q.w8a8_describe(whole) and "operands=8" in q.w8a8_describe(q.w8a8_problem(200, 256, 256))


def test_a_split_hint_leaves_the_kernel_and_its_tile():
    """The launch that is taken without the hint is the one that the hint splits."""
    for m in (1, 16, 17, 24, 40, 64, 65, 200, 333, 1000):
        for n, k in ((4096, 4096), (10240, 5120), (1024, 28672), (22016, 4096), (2048, 512)):
            for gate, out in ((q.GATE_NONE, q.DT_BF16), (q.GATE_NONE, q.DT_F32), (q.GATE_SILU, q.DT_FP8_E4M3)):
                def launch(split):
                    head, *f = q.w8a8_describe(q.w8a8_problem(m, n, k, out, gate=gate, split_hint=split)).split()
                    return head, [x for x in f if x.startswith("tokens=")]
                for split in (1, 2, 5, 32):
                    assert launch(split) == launch(0), (m, n, k, gate, out, split)


def test_one_workspace_for_every_number_of_tokens():
    """The largest number of tokens needs no workspace, smaller ones do: a workspace is allocated for all of them."""
    ps = [q.w8a8_problem(m, 11008, 4096, q.DT_FP8_E4M3, gate=q.GATE_SILU) for m in (1, 16, 40, 200, 333, 4096, 8192)]
    sizes = [q.w8a8_workspace_bytes(p) for p in ps]
    assert sizes[-1] == 0 and max(sizes) > 0 and sizes != sorted(sizes)
    ws = q.alloc_w8a8_workspace(ps, device="cpu")
    assert ws.numel() == max(sizes) and not ws.any()
    assert q.alloc_w8a8_workspace(ps[-1:], device="cpu") is None and q.alloc_w8a8_workspace([], device="cpu") is None
    assert q.alloc_w8a8_workspace(ps[1], device="cpu").numel() == sizes[1]


def test_the_faster_kernel_is_taken_up_to_64_tokens():
    """Where one kernel takes at least a tenth longer than the other (measured with weights from memory, us)."""
    silu = q.GATE_SILU
    for m, n, k, gate, out, rows, tiles in (
            (17, 4096, 4096, 0, q.DT_F16, 6.1, 12.2), (64, 4096, 11008, 0, q.DT_BF16, 20.2, 23.4), (32, 6144, 8192, 0, q.DT_BF16, 17.7, 19.6),
            (24, 28672, 8192, 0, q.DT_BF16, 58.4, 66.2), (48, 16384, 2048, 0, q.DT_F16, 13.3, 16.1), (64, 2816, 4096, silu, q.DT_FP8_E4M3, 16.1, 19.3),
            (40, 10240, 5120, 0, q.DT_BF16, 22.2, 19.8), (64, 28672, 8192, 0, q.DT_BF16, 86.5, 67.9), (64, 6144, 8192, 0, q.DT_BF16, 25.5, 20.2),
            (40, 11008, 4096, silu, q.DT_FP8_E4M3, 32.2, 26.8), (64, 11008, 4096, silu, q.DT_BF16, 32.4, 23.8), (47, 14336, 4096, 0, q.DT_F16, 23.3, 20.2)):
        taken = q.w8a8_describe(q.w8a8_problem(m, n, k, out, gate=gate)).split()[0]
        assert taken == ("rows" if rows < tiles else "tiles"), (m, n, k, gate, out)


def test_few_tokens_split_along_k_only_where_it_pays():
    """The rows kernel's splits: as measured with weights from memory, the fastest of 1, 2, 4 and 8 but for a tenth."""
    for m, n, k, splits in ((4, 1024, 2048, 1), (16, 512, 4096, 1), (1, 2048, 4096, 1), (4, 1024, 8192, 2), (16, 1024, 8192, 2),
                            (16, 2048, 8192, 2), (40, 1024, 8192, 4), (16, 1024, 28672, 4), (64, 1024, 28672, 4), (1, 2048, 28672, 2), (1, 4096, 28672, 1)):
        assert f"rows grid={n // 16 * splits} " in q.w8a8_describe(q.w8a8_problem(m, n, k)), (m, n, k)


def test_quantize_refuses_weights_of_another_shape():
    """With an exception that optimized Python keeps: the library reads as many weights as the problem has."""
    for gate, shape in ((q.GATE_NONE, (32, 128)), (q.GATE_SILU, (16, 128)), (q.GATE_SILU, (32, 64)), (q.GATE_NONE, (16 * 128,))):
        with pytest.raises(ValueError, match="w must be"):
            q.w8a8_quantize(q.w8a8_problem(1, 16, 128, gate=gate), np.zeros(shape, np.float32))
