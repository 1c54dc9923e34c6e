"""AdamW in fp64, and the 8-bit states as plain arithmetic on real numbers.

A code c of `mant` mantissa bits under a block exponent E stands for

    (1 + (c mod 2^mant) / 2^mant) * 2^(c div 2^mant + E - 15 - 127),   c = 0 for 0,

and a value x is rounded to floor(|x| / unit + draw) units, the unit being that of
x's own binade; E is the (biased) exponent of the block's largest magnitude rounded
up to `mant` bits, at least 16, and 255 for a block with an infinity or NaN.
"""
from __future__ import annotations

import numpy as np

BLOCK = 256
MUL1, MUL2 = 0xBB67AE85, 0x3C6EF373


def mix(x):
    x = (np.asarray(x, dtype=np.uint64) * np.uint64(MUL1)) & np.uint64(0xFFFFFFFF)
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(MUL2)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def draws(n, first, seed, step):
    """Draws in [0, 1) (multiples of 2^-16) for m, sqrt(v) and the parameter."""
    M = np.uint64(0xFFFFFFFF)
    key = mix((np.uint64(seed) + mix(step)) & M)
    h = mix((np.arange(first, first + n, dtype=np.uint64) + key) & M)
    h2 = (h * np.uint64(MUL1)) & M
    s = 2.0 ** -16
    return (h & np.uint64(0xFFFF)) * s, (h >> np.uint64(16)) * s, (h2 >> np.uint64(16)) * s


def step(param, grad, m, v, t, lr, beta1, beta2, eps, weight_decay, grad_scale=1.0):
    """(param, m, v) after step t, unrounded."""
    g = grad_scale * grad
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    w = param * (1 - lr * weight_decay)
    w = w - lr * (m / (1 - beta1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return w, m, v


def _blocks(x):
    n = len(x)
    pad = -n % BLOCK
    return np.concatenate([x, np.zeros(pad)]).reshape(-1, BLOCK), n


def exponents(x, mant):
    mag, _ = _blocks(np.abs(x))
    top = mag.max(axis=1)
    bad = ~np.isfinite(mag).all(axis=1)
    fr, ex = np.frexp(np.where(bad, 0.0, top))
    up = fr > 1 - 2.0 ** -(mant + 1)
    e = np.where(top > 0, ex - 1 + up + 127, 0)
    return np.where(bad, 255, np.maximum(e, 16)).astype(np.int64)


def encode(x, draw, mant):
    """(codes, exponents, slack): slack is how far x / unit + draw is from the next
    whole number, in units: a value computed in fp32 may fall on its other side."""
    exp = exponents(x, mant)
    e = np.repeat(exp, BLOCK)[: len(x)]
    mag = np.where(np.isfinite(x), np.abs(x), 0.0)
    ex = np.frexp(mag)[1] - 1                     # binade of x
    real = mag / np.exp2(ex - mant) + draw        # in units of that binade
    q = np.floor(real)
    slack = np.abs(real - np.rint(real))
    k = (ex + 127 - (e - 15)) * 2 ** mant + (q - 2 ** mant)
    k = np.where(mag > 0, np.maximum(k, 0), 0).astype(np.int64)
    if mant == 4:
        k = np.where((mag > 0) & (k == 0), 1, k)
    else:
        k = np.where((x < 0) & (k > 0), k + 128, k)
    return np.where(e == 255, 0, k), exp, slack


def decode(codes, exp, mant):
    codes = np.asarray(codes, dtype=np.int64)
    e = np.repeat(np.asarray(exp, dtype=np.int64), BLOCK)[: len(codes)]
    mag = codes & (16 * 2 ** mant - 1)
    x = (1 + (mag % 2 ** mant) / 2 ** mant) * np.exp2(mag // 2 ** mant + e - 15 - 127.0)
    x = np.where(mag == 0, 0.0, x)
    if mant == 3:
        x = np.where(codes >= 128, -x, x)
    return np.where(e == 255, np.nan, x)
