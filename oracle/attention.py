"""Plain 64-bit forms of the attention side of a decode step (TEST
INFRASTRUCTURE ONLY), in numpy, sharing no code with the GPU path.

bf16 inputs come as float64 values, codes as uint8.  Besides each result the
functions give what the tests' tolerances need (sums of magnitudes).
"""
import numpy as np

FMAX = {"e5m2": 57344.0, "e4m3": 448.0}
_FRACTION = {"e5m2": (2, 15), "e4m3": (3, 7)}     # fraction bits, exponent bias


def code_values(fmt):
    """The values of the 256 codes, from sign, exponent and fraction."""
    bits, bias = _FRACTION[fmt]
    out = np.empty(256)
    for c in range(256):
        e, f = (c & 127) >> bits, c & ((1 << bits) - 1)
        v = (1 + f / (1 << bits)) * 2.0 ** (e - bias) if e else f / (1 << bits) * 2.0 ** (1 - bias)
        if fmt == "e5m2" and e == 31:
            v = np.nan if f else np.inf
        if fmt == "e4m3" and (c & 127) == 127:
            v = np.nan
        out[c] = -v if c & 128 else v
    return out


def round_bf16(x):
    """float64 to the nearest bf16 value, ties to even (no overflow)."""
    m, e = np.frexp(np.asarray(x, np.float64))
    e = np.maximum(e, -125)
    return np.ldexp(np.rint(np.ldexp(x, 8 - e)), e - 8)


def norm_rope(x, weight, eps, cos_sin, positions, interleaved):
    """x [T, H, D] -> (normed and rotated, magnitude): the magnitude bounds
    each output's terms, |a c| + |b s|."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    mag = np.abs(x)
    if cos_sin is None:
        return x, mag
    h = cos_sin.shape[1] // 2
    c = cos_sin[positions, None, :h].astype(np.float64)
    s = cos_sin[positions, None, h:].astype(np.float64)
    ia = np.arange(0, 2 * h, 2) if interleaved else np.arange(h)
    ib = ia + 1 if interleaved else ia + h
    y = x.copy()
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = np.abs(a * c) + np.abs(b * s)
    mag[..., ib] = np.abs(b * c) + np.abs(a * s)
    return y, mag


def quantise(x, fmt):
    """Rows x [..., D] (bf16 values) -> (codes, float32 scales [...]): the
    nearest code, ties to even, to the fp32 quotient by the fp32 scale."""
    x = np.asarray(x, np.float32)
    amax = np.abs(x).max(-1)
    d = np.where(amax == 0, np.float32(1), amax / np.float32(FMAX[fmt]))
    q = (x / d[..., None]).astype(np.float64).clip(-FMAX[fmt], FMAX[fmt])
    bits, bias = _FRACTION[fmt]
    _, e = np.frexp(q)
    e = np.where(q == 0, 2 - bias, np.maximum(e, 2 - bias))    # subnormals share the smallest normal's step
    n = np.rint(np.ldexp(np.abs(q), bits + 1 - e)).astype(np.int64)    # in units of the step
    code = ((e + bias - 2) << bits) + n          # a carry moves on to the next exponent
    return (code | np.where(np.signbit(q), 128, 0)).astype(np.uint8), d.astype(np.float32)


def attention(q, k, v, scale, window=0):
    """One sequence: q [Hq, D], k, v [n, H, D] values.  Returns (out [Hq, D],
    lse [Hq], weight-averaged magnitude of v [Hq, D], the largest sum of
    |q k| scale of a seen score [Hq])."""
    n, H, D = k.shape
    Hq = q.shape[0]
    lo = max(0, n - window) if window else 0
    out, lse = np.zeros((Hq, D)), np.full(Hq, -np.inf)
    mag, big = np.zeros((Hq, D)), np.zeros(Hq)
    if n - lo <= 0:
        return out, lse, mag, big
    for h in range(Hq):
        kk, vv = k[lo:, h // (Hq // H)], v[lo:, h // (Hq // H)]
        s = scale * (kk @ q[h])
        m = s.max()
        p = np.exp(s - m)
        out[h], mag[h] = p @ vv / p.sum(), p @ np.abs(vv) / p.sum()
        lse[h] = m + np.log(p.sum())
        big[h] = abs(scale) * (np.abs(kk) @ np.abs(q[h])).max()
    return out, lse, mag, big
