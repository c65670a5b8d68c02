"""Plain CPU reference of the AdamW operators (numpy, float64, with the
definition's float32 roundings made explicit where they are part of it).

The step is algorithm 2 of Loshchilov and Hutter, "Decoupled Weight Decay
Regularization" (ICLR 2019). moments() forms m', v' and r' = sqrt(v') with
every operation rounded to float32 on its own: each is computed in float64
from float32 operands and rounded once, which is that rounding (a product of
two 24-bit significands fits 53 bits; for the sum and the square root 53 >=
2 * 24 + 2 bits make the double rounding innocuous).

The 8-bit format: blocks of 256 consecutive entries; one exponent byte per
block; codes of E4M3 (sign, 4 exponent bits with bias 7, 3 mantissa bits).
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 256


def f32(x):
    """One rounding to float32, kept in float64."""
    with np.errstate(over="ignore", invalid="ignore"):
        return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


class Roots(np.ndarray):
    """Second moments' roots: encode() keeps those that are not zero."""


def moments(m, v, g, beta1, beta2, scale=None):
    """(m', v', r') of float32 moments and gradients, with the definition's float32 roundings."""
    b1, c1, b2, c2 = f32(beta1), f32(1 - beta1), f32(beta2), f32(1 - beta2)
    with np.errstate(over="ignore", invalid="ignore"):
        g = np.asarray(g, np.float64)
        if scale is not None:
            g = f32(f32(scale) * g)
        m = f32(f32(b1 * m) + f32(c1 * g))
        v = f32(f32(b2 * v) + f32(c2 * f32(g * g)))
        return m, v, f32(np.sqrt(v)).view(Roots)


def direction(m, r, t, beta1, beta2, eps):
    """The step's direction before weight decay, in float64, from m' and r'."""
    with np.errstate(over="ignore", invalid="ignore"):
        return (m / (1 - beta1 ** t)) / (r / math.sqrt(1 - beta2 ** t) + eps)


def step64(w, g, m, v, t, lr, beta1, beta2, eps, wd, scale=1.0):
    """The whole step in float64 without any rounding: (W', m', v')."""
    g = scale * np.asarray(g, np.float64)
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    return w - lr * (wd * w + direction(m, np.sqrt(v), t, beta1, beta2, eps)), m, v


# ---------------------------------------------------------------- 8-bit moments
def code_values():
    """Value of each of the 256 codes."""
    out = np.zeros(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = (math.nan if c & 127 == 127 else x) * (-1 if c & 128 else 1)
    return out


_VALUES = code_values()


def _nearest_code(y):
    """E4M3 code nearest to each y (|y| <= 448), ties to the even mantissa."""
    a = np.abs(y)
    _, e = np.frexp(a)
    grid = np.exp2(np.maximum(e - 1, -6).astype(np.float64) - 3)
    a = np.rint(a / grid) * grid
    mant, e = np.frexp(a)  # a = mant 2^e, mant in [1/2, 1)
    sub = a < 2.0 ** -6
    code = np.where(sub, a * 512, (e - 1 + 7) * 8 + (mant * 2 - 1) * 8).astype(np.int64)
    return (code | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def _random_code(y, rnd):
    """E4M3 code of each y (|y| < 256): the code below |y| or the next one, up where |y|'s place between the two (in 2^20
    parts, and |y| < 2^-6 to multiples of 2^-29) and rnd / 2^16 together reach one."""
    a = f32(np.abs(y) * 2.0 ** -120) * 2.0 ** 120
    grid = np.exp2(np.maximum(np.frexp(a)[1] - 1, -6).astype(np.float64) - 3)
    below = np.floor(a / grid)
    up = a / grid - below + np.asarray(rnd, np.float64) * 2.0 ** -16 >= 1
    return _nearest_code(np.copysign((below + up) * grid, y))


def exponent_bytes(x):
    """Exponent byte of each block of a flat array of float32 values."""
    n = x.size
    pad = np.zeros(-(-n // BLOCK) * BLOCK)
    pad[:n] = x
    out = []
    for row in pad.reshape(-1, BLOCK):
        top = np.max(np.abs(row)) if not np.isnan(row).any() else math.nan
        if not np.isfinite(top):
            out.append(255)
        else:
            out.append(0 if top < 2.0 ** -119 else math.frexp(top)[1] - 1 + 127 - 7)
    return np.array(out, np.uint8)


def encode(x, rnd=None):
    """(codes, exponent bytes) of a flat array; rnd: 16 random bits per entry, None: to nearest. Roots that are not zero
    get at least the smallest code (in a block that is held)."""
    least = isinstance(x, Roots)
    x = np.asarray(x, np.float64).reshape(-1)
    byte = exponent_bytes(x)
    per = np.repeat(byte.astype(np.int64), BLOCK)[:x.size]
    live = (per > 0) & (per < 255)
    y = np.where(live, np.where(live, x, 0.0) * np.exp2(np.where(live, 127.0 - per, 0.0)), 0.0)
    code = _nearest_code(y) if rnd is None else _random_code(y, rnd)
    if least:
        code = np.where(x > 0, np.maximum(code, 1), code)
    return np.where(live, code, 0).astype(np.uint8), byte


def decode(codes, byte):
    """float32 values of codes and exponent bytes (in float64)."""
    per = np.repeat(np.asarray(byte).astype(np.int64), BLOCK)[:codes.size]
    val = _VALUES[codes] * np.exp2(np.where((per > 0) & (per < 255), per - 127.0, 0.0))
    return f32(np.where(per == 0, 0.0 * val, np.where(per == 255, math.nan, val)))


def rounding_bits(n, tensor, seed, t, first=0):
    """The 16 random bits of entries first..first + n - 1 (first a multiple of 8) of a tensor at step t
    (Philox4x32-10 in Python integers)."""
    low = 0xFFFFFFFF
    out = np.empty(-(-n // 8) * 8, np.uint32)
    for e in range(-(-n // 8)):
        grp = first // 8 + e
        c, k = [grp & low, grp >> 32, t & low, 1], [seed & low, tensor & low]
        for r in range(10):
            if r:
                k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
            p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
            c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & low, (p0 >> 32) ^ c[3] ^ k[1], p0 & low]
        for i in range(4):
            out[8 * e + 2 * i], out[8 * e + 2 * i + 1] = c[i] & 0xFFFF, c[i] >> 16
    return out[:n]


# ---------------------------------------------------------------- gradient norm
def grad_norm(gs, max_norm):
    """(norm, clip factor) in float64."""
    norm = math.sqrt(math.fsum(float(np.sum(np.asarray(g, np.float64) ** 2)) for g in gs))
    return norm, min(1.0, max_norm / (norm + 1e-6))
