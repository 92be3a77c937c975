"""8-bit floating point and block quantization, by definition.

A format has `mant` mantissa bits and the smallest normal exponent `emin`; its
values are +-m 2^e. e4m3: bias 7, no infinity, NaN 0x7F/0xFF, top 448. e5m2:
bias 15, infinity 0x7C, top 57344; saturating conversions never make it.
"""

import numpy as np

E4M3 = dict(mant=3, emin=-6, bias=7, top=448.0)
E5M2 = dict(mant=2, emin=-14, bias=15, top=57344.0)
FORMATS = {0: E4M3, 1: E5M2}
LEAST = np.float32(2.0 ** -100)
NAN_CODE = 0x7F


def decode(codes, fmt):
    """fp64 values of uint8 codes."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    mant, emin, bias = fmt["mant"], fmt["emin"], fmt["bias"]
    frac, exp = c & ((1 << mant) - 1), (c & 0x7F) >> mant
    v = np.where(exp == 0, np.ldexp(frac.astype(np.float64), emin - mant),
                 np.ldexp((frac + (1 << mant)).astype(np.float64), exp - bias - mant))
    if fmt is E4M3:
        v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    else:
        v = np.where(exp == 31, np.where(frac == 0, np.inf, np.nan), v)
    return np.where(c >= 128, -v, v)


def encode(x, fmt):
    """Nearest code, ties to even, saturating; not-a-number for NaN."""
    x = np.asarray(x, np.float64)
    mant, emin, bias = fmt["mant"], fmt["emin"], fmt["bias"]
    mag = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), fmt["top"])
    _, e = np.frexp(mag)                       # mag = f 2^e, f in [1/2, 1)
    e = np.maximum(e - 1, emin)
    steps = np.rint(np.ldexp(mag, mant - e)).astype(np.int64)      # units of 2^(e - mant)
    over = steps == (2 << mant)                # rounded up to the next power of two
    steps, e = np.where(over, 1 << mant, steps), np.where(over, e + 1, e)
    normal = steps >= (1 << mant)
    code = np.where(normal, ((e + bias) << mant) + steps - (1 << mant), steps)
    code = code | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isnan(x), NAN_CODE, code).astype(np.uint8)


def block_scale(v, fmt, axis=-1):
    """(scale, inverse) fp32 of blocks laid out along `axis`."""
    v = np.asarray(v, np.float32)
    amax = np.max(np.where(np.isfinite(v), np.abs(v), np.float32(0)), axis=axis).astype(np.float32)
    amax = np.maximum(amax, LEAST)
    top = np.float32(fmt["top"])
    return amax / top, top / amax


def scaled(v, inv):
    """fl32(v inv) where v is finite, else NaN; zeros keep their sign."""
    v = np.asarray(v, np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        return np.where(np.isfinite(v), v * inv, np.float32(np.nan)).astype(np.float32)


def quantize_rows(x, fmt, block=128):
    """(codes, scales) of fp32 rows, one scale per `block` columns."""
    rows, cols = x.shape
    nb = -(-cols // block)
    t = np.zeros((rows, nb * block), np.float32)
    t[:, :cols] = x
    t = t.reshape(rows, nb, block)
    scale, inv = block_scale(t, fmt)
    return encode(scaled(t, inv[:, :, None]), fmt).reshape(rows, -1)[:, :cols], scale


def quantize_weight(w, fmt=E4M3, block=128):
    """(codes, scales) of an fp32 matrix, one scale per block x block."""
    n, k = w.shape
    nn, nk = -(-n // block), -(-k // block)
    t = np.zeros((nn * block, nk * block), np.float32)
    t[:n, :k] = w
    b = t.reshape(nn, block, nk, block).transpose(0, 2, 1, 3).reshape(nn, nk, -1)
    scale, inv = block_scale(b, fmt)
    wide = np.repeat(np.repeat(inv, block, 0), block, 1)[:n, :k]
    return encode(scaled(w, wide), fmt), scale


def rows_values(codes, scales, fmt, block=128):
    return decode(codes, fmt) * np.repeat(scales.astype(np.float64), block, 1)[:, :codes.shape[1]]


def weight_values(codes, scales, block=128):
    n, k = codes.shape
    return decode(codes, E4M3) * np.repeat(np.repeat(scales.astype(np.float64), block, 0), block, 1)[:n, :k]
