"""Oracle of the 8-bit operators in 64 bits (TEST INFRASTRUCTURE ONLY): the residual addition with RMS norm, e4m3
values with a scale per block of 128, their products and the gates.  Plain numpy, each from its definition:

  activations  value[t, k] = code[t, k] * scale[k / 128, t],  scale = max(max |x|, 2^-100) / 448, code = RNE(x / scale)
  weights      value[r, k] = code[r, k] * scale[r / 128, k / 128]
"""
import numpy as np

from . import codecs

BLOCK = 128
LEAST = 2.0 ** -100


def weight_values(codes, scales, parts=1):
    """codes uint8 [parts * N, K], scales [parts * ceil(N / 128), K / 128] -> float64 [parts * N, K]."""
    rows, k = codes.shape
    n = rows // parts
    v = codecs.e4m3_decode(codes)
    out = np.empty((rows, k))
    per = -(-n // BLOCK)
    for r in range(rows):
        s = scales[r // n * per + r % n // BLOCK].astype(np.float64)
        out[r] = v[r] * np.repeat(s, BLOCK)
    return out


def activation_values(codes, scales):
    """codes uint8 [tokens, K], scales [K / 128, tokens] -> float64 [tokens, K]."""
    return codecs.e4m3_decode(codes) * np.repeat(scales.astype(np.float64).T, BLOCK, axis=1)


def activation_scales(x):
    """float64 [tokens, K] -> scales [K / 128, tokens]; NaN where a block holds a value that is not finite."""
    y = np.abs(x.reshape(x.shape[0], -1, BLOCK))
    top = np.where(np.isfinite(y).all(-1), np.where(np.isfinite(y), y, 0).max(-1), np.nan)
    return np.where(np.isnan(top), np.nan, np.maximum(top, LEAST)).T / 448.0


def add_norm(x, residual, weight, norm, eps):
    """float64 rows -> (sum, y)."""
    s = x if residual is None else x + residual
    if not norm:
        return s, s
    y = s / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps)
    return s, y if weight is None else y * weight


def act(g, gate):
    if gate == "silu":
        return g / (1 + np.exp(-g))
    return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))


def half_step(v, scale):
    """Largest distance of a value from the e4m3 code times scale that it is rounded to."""
    return np.maximum(np.abs(v) * 2.0 ** -4, scale * 2.0 ** -10)
