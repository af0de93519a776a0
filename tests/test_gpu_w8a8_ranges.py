"""The residual addition with RMS norm to e4m3 where its factors leave fp32's range one by one: a small eps beside rows, blocks
and weights that are zero or tiny.  The codes stay those of the definition, code = RNE(y / scale)."""
import numpy as np
import pytest

from gpu_cases import say
from test_gpu_w8a8 import F8, norm_check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_qgemm_amd as q
    return q


# eps as fp32 values; the last is the smallest normal number
EPS = [float(np.float32(e)) for e in (1e-6, 2.8e-12, 1e-12, 1e-20, 1e-30, 2.0 ** -126)]


@pytest.mark.parametrize("eps", EPS)
@pytest.mark.parametrize("dim", [384, 1152])                                  # a wavefront's rows, a workgroup's
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_add_norm_small_eps(q, dtype, dim, eps):
    say(f"case add_norm small eps {dtype} {dim} {eps}")
    t16 = dict(f16=torch.float16, bf16=torch.bfloat16)[dtype]
    g = torch.Generator().manual_seed(dim)
    t = 9
    x, w = torch.randn((t, dim), generator=g), 1 + 0.3 * torch.randn(dim, generator=g)
    x[0] = 0                                                                  # padding
    x[1, :128] = 0                                                            # a zero block in an ordinary row
    least = -24 if dtype == "f16" else -120
    x[2], x[3] = x[2] * 2.0 ** -10, x[3] * 2.0 ** -18
    x[4], x[5] = 0, 0
    x[4, 3], x[5, 130] = 2.0 ** least, -2.0 ** least                           # all but zero
    x[6], x[7] = x[6] * 2.0 ** max(least, -40), x[7] * 2.0 ** max(least, -105)
    x[8], x[8, 256:] = x[8] * 2.0 ** max(least, -118), 0
    w[-128:] = 0                                                              # a zero block of the weight
    w[128:256] *= 2.0 ** (-14 if dtype == "f16" else -100)
    x, w = x.to(t16), w.to(t16)
    y, scales = torch.empty((t, dim), dtype=F8, device="cuda"), torch.empty((dim // 128, t), device="cuda")
    p = q.add_norm_problem(t, dim, q.DT_F16 if dtype == "f16" else q.DT_BF16, q.DT_FP8_E4M3, eps=eps)
    for weight in (w, None):
        q.add_norm(p, x.cuda(), None, None if weight is None else weight.cuda(), None, y, scales)
        torch.cuda.synchronize()
        assert bool(torch.isfinite(scales).all()) and bool(torch.isfinite(y.float()).all())
        assert bool((y[0].float() == 0).all()) and bool((scales[:, 0] == np.float32(2.0 ** -100 / 448)).all())
        norm_check(x, None, weight, True, eps, dtype, "e4m3", None, y, scales)


def test_add_norm_without_eps(q):
    """eps = 0: rows of any size give the same codes; a row of zeros is 0 / 0."""
    say("case add_norm eps 0")
    dim = 384
    row = torch.randn(dim, generator=torch.Generator().manual_seed(1)).bfloat16()
    x = torch.stack([row.double() * 2.0 ** e for e in (0, 50, -20, -40, -50)] + [torch.zeros(dim).double()]).bfloat16()
    y, scales = torch.empty((6, dim), dtype=F8, device="cuda"), torch.empty((3, 6), device="cuda")
    q.add_norm(q.add_norm_problem(6, dim, q.DT_BF16, q.DT_FP8_E4M3, eps=0.0), x.cuda(), None, None, None, y, scales)
    torch.cuda.synchronize()
    norm_check(x[:5], None, None, True, 0.0, "bf16", "e4m3", None, y[:5], scales[:, :5].contiguous())
    assert bool((y[:5].view(torch.uint8) == y[0].view(torch.uint8)).all()) and bool((scales[:, :5] == scales[:, :1]).all())
    assert bool(torch.isnan(y[5].float()).all()) and bool(torch.isnan(scales[:, 5]).all())
