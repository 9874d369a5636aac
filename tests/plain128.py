"""The operators with 128-element scales from their definitions, in float64
numpy: what the tests of the kernels compare with."""

import numpy as np

MAXV = {1: 448.0, 2: 57344.0}     # by format: E4M3 1, E5M2 2
MANT = {1: 3, 2: 2}               # mantissa bits
LOW = {1: -6, 2: -14}             # smallest normal exponent
BIAS = {1: 7, 2: 15}
TINY = 2.0 ** -126


def decode(codes, fmt):
    """Value of each code byte."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    m, b = MANT[fmt], BIAS[fmt]
    e = (c & 0x7F) >> m
    f = c & ((1 << m) - 1)
    v = np.where(e == 0, f * 2.0 ** (1 - b - m), (1 + f * 2.0 ** -m) * 2.0 ** (e - b))
    top = (1 << (7 - m)) - 1
    if fmt == 1:
        v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    else:
        v = np.where(e == top, np.where(f == 0, np.inf, np.nan), v)
    return np.where(c & 0x80, -v, v)


def encode(x, fmt):
    """Code byte of each float64 value: nearest, ties to the even code,
    saturating, sign kept; NaN 0x7F."""
    x = np.asarray(x, np.float64)
    m, b = MANT[fmt], BIAS[fmt]
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), MAXV[fmt])
    e = np.maximum(np.frexp(np.where(a == 0, 1.0, a))[1] - 1, LOW[fmt])
    k = np.rint(a / 2.0 ** (e - m)).astype(np.int64)      # in steps of 2^(e - m)
    # k in [0, 2^(m+1)]: 2^(m+1) is the next exponent's first code; a
    # subnormal (e = LOW, k < 2^m) is its own code
    code = np.where(k >= (1 << m), ((e + b) << m) + (k - (1 << m)), k)
    code = np.minimum(code, int(0x7E if fmt == 1 else 0x7B)) | (np.signbit(x) * 0x80)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def scale_of(amax, fmt, pow2):
    """Scale (float32 values) of tiles' largest magnitudes (float64)."""
    amax = np.asarray(amax, np.float64)
    bad = ~np.isfinite(amax)
    a = np.where(bad, 1.0, amax)
    if pow2:
        q = a / MAXV[fmt]                       # exact comparisons: maxv = 7 * 2^n
        e = np.ceil(np.log2(np.where(q == 0, TINY, q)))
        for _ in range(2):                      # log2 may be off by one at a boundary
            e = np.where(MAXV[fmt] * 2.0 ** (e - 1) >= a, e - 1, e)
            e = np.where(MAXV[fmt] * 2.0 ** e < a, e + 1, e)
        s = 2.0 ** np.maximum(e, -126)
    else:
        # a float64 quotient of two floats rounds to the float quotient
        s = np.maximum((a / MAXV[fmt]).astype(np.float32).astype(np.float64), TINY)
    return np.where(bad, np.nan, s).astype(np.float32)


def amax_of(x, block):
    """Largest magnitudes of 1 x 128 tiles or 128 x 128 blocks (NaN kept)."""
    x = np.abs(np.asarray(x, np.float64))
    rows, cols = x.shape
    t = np.stack([x[:, c:c + 128].max(1) for c in range(0, cols, 128)], 1)
    return np.stack([t[r:r + 128].max(0) for r in range(0, rows, 128)], 0) if block else t


def spread(scales, rows, cols, block):
    s = np.repeat(np.asarray(scales, np.float64), 128, 1)[:, :cols]
    return np.repeat(s, 128, 0)[:rows] if block else s


def quantize(x, fmt, block, pow2):
    """(codes, scales) of float64 x along its rows."""
    s = scale_of(amax_of(x, block), fmt, pow2)
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        q = (np.asarray(x, np.float64) / spread(s, *x.shape, block)).astype(np.float32)
    return encode(q, fmt), s


def norm(x, residual, weight, eps):
    """(h, y) in float64."""
    h = x if residual is None else x + residual
    return h, h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * weight


def norm_bwd(gy, h, weight, eps, gres):
    r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    n, g = h * r, gy * weight
    gh = r * (g - n * (g * n).mean(1, keepdims=True))
    return gh + (0 if gres is None else gres), (gy * n).sum(0)
