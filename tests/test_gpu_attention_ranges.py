"""The attention operators at the ends of their arguments' ranges, against the 64-bit oracle."""
import numpy as np
import pytest

from gpu_cases import say
from test_gpu_attention import _check, _run, _sequences
from test_gpu_attention_plans import scale_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_qgemm_amd as lib
    return lib


# kind, query lengths, context lengths, q_heads, kv_heads, dim, group, page
WIDE = [("f16", [700], [700], 4, 1, 64, 64, 16), ("bf16", [70, 3], [2100, 40], 1, 1, 128, 32, 48),
        ("f16", [200, 30], [100, 0], 2, 1, 128, 64, 16), ("bf16", [1, 5, 2], [900, 2, 64], 8, 2, 64, 32, 16)]


@pytest.mark.parametrize("hint", [0, 1, 2])
@pytest.mark.parametrize("case", range(len(WIDE)))
def test_windows_wider_than_any_context(q, case, hint):
    # windows up to the type's largest hide nothing, also where a sequence has more queries than tokens
    kind, qlens, klens, hq, hk, dim, group, page = WIDE[case]
    say(f"case attention wide windows {WIDE[case]} hint={hint}")
    s = _sequences(q, kind, qlens, klens, hq, hk, dim, group, page, 400 + case)
    outs = [_run(q, s, kind, hq, True, w, hint=hint) for w in (2 ** 31 - 1, 2 ** 31 - 200, 2 ** 30)]
    _check(s, outs[0], kind, hq, True, 0, scale_of(dim))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
