"""Oracle of the attention operators, in 64 bits (numpy): head norm and rotation, the 4-bit cache,
attention over the cache's values, and the error bounds the GPU results are held to.

Written from the definitions in include/qgemm_attention.h, without code of the library.  16-bit
arrays are passed as float64 values that a 16-bit type holds; `kind` is 'f16' or 'bf16'.
"""
import numpy as np

# largest relative error of one rounding to the type
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def round16(x, kind):
    """float64 -> nearest-even value of the 16-bit type (as float64); overflow goes to infinity."""
    x = np.asarray(x, np.float64)
    if kind == "f16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16).astype(np.float64)
    finite = np.isfinite(x)
    a = np.where(finite, x, 0.0)
    e = np.maximum(np.frexp(a)[1] - 1, -126)
    step = np.ldexp(1.0, e - 7)
    r = np.rint(a / step) * step
    r = np.where(np.abs(r) > 3.3895313892515355e38, np.copysign(np.inf, r), r)
    return np.where(finite, r, x)


def bits16(x, kind):
    """The uint16 pattern of values that the 16-bit type holds."""
    if kind == "f16":
        return np.asarray(x, np.float64).astype(np.float16).view(np.uint16)
    return (np.asarray(x, np.float64).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def from_bits16(b, kind):
    b = np.asarray(b, np.uint16)
    if kind == "f16":
        return b.view(np.float16).astype(np.float64)
    with np.errstate(invalid="ignore"):                              # signalling NaN patterns
        return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


# ----------------------------------------------------------------------------- norm and rotation
def norm_rope(x, weight, positions, table, rot, interleaved, norm=True, eps=1e-6):
    """x [T, H, D] -> y in 64 bits and the sum of magnitudes behind each y (for the error bound)."""
    y = np.array(x, np.float64)
    if norm:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + np.float64(np.float32(eps)))
        if weight is not None:
            y = y * weight
    mag = np.abs(y)
    if rot:
        row = np.asarray(table, np.float64)[np.clip(positions, 0, len(table) - 1)]
        c, s = row[:, None, :rot // 2], row[:, None, rot // 2:]
        a, b = (np.s_[..., 0:rot:2], np.s_[..., 1:rot:2]) if interleaved else (np.s_[..., :rot // 2], np.s_[..., rot // 2:rot])
        ya, yb = y[a].copy(), y[b].copy()
        y[a], y[b] = ya * c - yb * s, yb * c + ya * s
        mag[a], mag[b] = np.abs(ya * c) + np.abs(yb * s), np.abs(yb * c) + np.abs(ya * s)
    return y, mag


def norm_rope_bound(y, mag, dim, kind):
    """One rounding to 16 bits (or half the smallest subnormal step), plus fp32: the sum of `dim`
    squares (dim roundings, halved by the root) and eight operations after it."""
    tiny = 2.0 ** -25 if kind == "f16" else 0.0
    return UNIT[kind] * np.abs(y) + (dim / 2 + 8) * 2.0 ** -24 * mag * (1 + UNIT[kind]) + tiny


# ----------------------------------------------------------------------------- the cache
def quantize(x, group, kind):
    """x [..., D] -> codes uint8 [..., D], scale and zero [..., D / group] (values of the type).

    The steps are fp32, each rounded once, as the definition says."""
    x32 = np.asarray(x, np.float64).astype(np.float32)
    g = x32.reshape(*x32.shape[:-1], x32.shape[-1] // group, group)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        span = hi - lo
        bad = ~np.isfinite(span)
        s = round16((span / np.float32(15)).astype(np.float64), kind)
        c = np.rint((g - lo[..., None]) / s.astype(np.float32)[..., None])
    c = np.where((s > 0)[..., None] & ~bad[..., None], np.clip(np.nan_to_num(c), 0, 15), 0).astype(np.uint8)
    nan = np.float64("nan")
    return c.reshape(x32.shape), np.where(bad, nan, s), np.where(bad, nan, lo.astype(np.float64))


def dequantize(codes, scale, zero, group):
    """The values the codes stand for, exactly."""
    return codes * np.repeat(scale, group, -1) + np.repeat(zero, group, -1)


def block_bytes(page, dim, group):
    return page * (dim + 8 * (dim // group))


def pack_block(kc, ks, kz, vc, vs, vz, kind):
    """One page of one kv head: codes [P, D], scale / zero [P, NG] of both sides -> its bytes."""
    P, D = kc.shape
    NG, u = ks.shape[1], D // 32
    out = np.zeros(P * (D + 8 * NG), np.uint8)
    for t in range(P):
        for d in range(D):
            b, n = divmod(d, 8)
            i, g = divmod(b, 4)
            out[t * (D // 2) + 4 * (u * g + i) + n // 2] |= kc[t, d] << (4 * (n % 2))
            i, r = divmod(d, 16)
            out[P * D // 2 + ((t // 4) * 16 + r) * 4 * u + (t % 4) * u + i // 2] |= vc[t, d] << (4 * (i % 2))
    for side, (s, z) in enumerate(((ks, kz), (vs, vz))):
        par = np.stack((bits16(s.T, kind), bits16(z.T, kind)), -1).reshape(-1)        # [NG][P][2]
        at = P * D + side * P * NG * 4
        out[at:at + P * NG * 4] = par.view(np.uint8)
    return out




# ----------------------------------------------------------------------------- attention
def attention(q, k, v, length, causal, window, scale):
    """q [n, D], k, v [length, D] of one sequence and head -> out [n, D], weights [n, length]."""
    n = q.shape[0]
    t = np.arange(length)[None, :]
    pos = length - n + np.arange(n)[:, None]
    seen = np.ones((n, length), bool)
    if causal:
        seen = t <= pos
        if window:
            seen &= t > pos - window
    out, w = np.zeros((n, q.shape[1])), np.zeros((n, length))
    for i in range(n):
        at = np.flatnonzero(seen[i])
        if not at.size:
            continue
        s = (k[at] @ q[i]) * scale
        with np.errstate(invalid="ignore"):                            # NaN tokens
            e = np.exp(s - s.max())
        w[i, at] = e / e.sum()
        out[i] = w[i, at] @ v[at]
    return out, w


def attention_bound(q, w, out, ks, kz, vs, vz, kmax, group, scale, kind):
    """Largest error of a result with fp32 accumulation and code weights rounded to 11 bits.

    out = sum_t w_t v_t.  (1) one rounding to the type; (2) each w_t * scale_t rounded to 11 bits,
    times a code no further than 8 from the middle; (3) a score off by ds moves every weight by a
    factor exp(+-ds), so the output by at most 2 ds sum w |v - out|: ds from D fp32 steps over the
    magnitudes |q| (15 scale + |zero|), and the exponential itself; (4) fp32 sums over the tokens."""
    n, D = q.shape
    vmax = np.repeat(15 * np.abs(vs) + np.abs(vz), group, -1)                          # [len, D]
    bound = UNIT[kind] * np.abs(out) + (2.0 ** -25 if kind == "f16" else 0.0)
    bound += 2.0 ** -11 * (w @ np.repeat(8 * np.abs(vs), group, -1))
    amount = np.abs(q) @ np.repeat(15 * np.abs(ks) + np.abs(kz), group, -1).T * abs(scale)   # [n, len]
    ds = (D + 16) * 2.0 ** -24 * amount + 2.0 ** -21
    spread = w @ vmax + np.abs(out)
    bound += 2 * np.max(np.where(w > 0, ds, 0), axis=1, keepdims=True, initial=0) * spread
    return bound + (kmax + 64) * 2.0 ** -24 * (w @ vmax)


def attention_weight_bound(q, w, v, out, ks, kz, vs, vz, group, scale, kind, floor, values16=False):
    """As attention_bound, with the weights' own range, the sums' real length and the values' real distance from the
    result.

    A token's weight times a group's scale, p, multiplies a code no further than 8 from the middle; it is
    rounded to 11 bits (half a unit: 2^-12 p), or, where it is far below the group's largest in the row, to
    `floor` of that one, or lost.  values16: the weight multiplies the whole value, itself rounded to 11 bits.
    A result is the sum of at most one rounding for eight tokens (32 enter a product at once, whose own
    sum rounds up to four times) and 64 at the joins."""
    n, D = q.shape
    ng = D // group
    vmax = np.repeat(15 * np.abs(vs) + np.abs(vz), group, -1)                          # [len, D]
    size = 15 * np.abs(vs) + np.abs(vz) if values16 else 8 * np.abs(vs)                # [len, NG]
    low = np.zeros((n, ng))
    for i in range(n):
        p = w[i][:, None] * size
        low[i] = (2.0 ** -12 * (2 if values16 else 1) * p + np.minimum(p, floor * p.max(0, initial=0.0))).sum(0)
    bound = UNIT[kind] * np.abs(out) + (2.0 ** -25 if kind == "f16" else 0.0) + np.repeat(low, group, -1)
    amount = np.abs(q) @ np.repeat(15 * np.abs(ks) + np.abs(kz), group, -1).T * abs(scale)   # [n, len]
    ds = (D + 16) * 2.0 ** -24 * amount + 2.0 ** -21
    spread = np.stack([w[i] @ np.abs(v - out[i]) for i in range(n)])
    bound += 2 * np.max(np.where(w > 0, ds, 0), axis=1, keepdims=True, initial=0) * spread
    return bound + (w.shape[1] / 8 + 64) * 2.0 ** -24 * (w @ vmax)
