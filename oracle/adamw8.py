"""The states of the 8-bit AdamW step, operation by operation in fp32.

m and r = sqrt(v) are e4m3 codes with one scale per 256 values of a tensor.
Every operation below is rounded to fp32 by itself, so that a state after any
number of steps is one set of bits:

    m <- b1 (code scale) + (1 - b1) g
    v <- b2 r^2 + (1 - b2) g^2,  r = code scale
    amax  = max |value| of the block, at least 2^-100
    scale = amax fl(1/448)
    code  = e4m3(clamp(value (448 fl(1/amax)), -448, 448)); of a root above zero at least 2^-9
"""

import numpy as np

from oracle import fp8

BLOCK = 256
F = np.float32


def decode(codes, scales):
    """fp32 values of a tensor's codes [n] under scales [ceil(n/256)]."""
    n = codes.size
    return fp8.decode(codes, fp8.E4M3).astype(F) * np.repeat(scales.astype(F), BLOCK)[:n]


def encode(values, root):
    """(codes [n], scales [ceil(n/256)]) of finite fp32 values."""
    n = values.size
    t = np.zeros(-(-n // BLOCK) * BLOCK, F)
    t[:n] = values
    t = t.reshape(-1, BLOCK)
    amax = np.maximum(np.abs(t).max(1), F(2.0 ** -100))
    c = t * (F(448) * (F(1) / amax))[:, None]
    if root:
        c = np.where(t > 0, np.maximum(c, F(2.0 ** -9)), c)
    return fp8.encode(c, fp8.E4M3).reshape(-1)[:n], amax * (F(1) / F(448))


def states(m, r, g, beta1, beta2):
    """(m, sqrt(v)) after a gradient, fp32, from the fp32 values of the states."""
    m, r, g, b1, b2 = (np.asarray(a, F) for a in (m, r, g, beta1, beta2))
    m = m * b1 + g * (F(1) - b1)
    v = (r * r) * b2 + (g * g) * (F(1) - b2)
    return m, np.sqrt(v)


def step(m, m_scales, r, r_scales, g, beta1, beta2):
    """The next (m, m_scales, r, r_scales) of one tensor: codes and scales."""
    m, r = states(decode(m, m_scales), decode(r, r_scales), g, beta1, beta2)
    return encode(m, False) + encode(r, True)
