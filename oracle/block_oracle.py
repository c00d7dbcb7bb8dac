"""The gated feed-forward block and the AdamW step in fp64 numpy, from their formulas.

Test infrastructure only.
"""

from __future__ import annotations

import math

import numpy as np

BLOCK = 128
TOP = 448.0
LEAST = 2.0 ** -118


# ------------------------------------------------------- gated feed-forward ----


def act(name, g):
    """(act(g), act'(g))."""
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-np.clip(g, -700, 700)))
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        phi = np.vectorize(lambda v: 0.5 * math.erfc(-v / math.sqrt(2)), otypes=[np.float64])(g)
        return g * phi, phi + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 0.134145 * g * g)
    if name == "relu":
        return np.maximum(g, 0), (g > 0).astype(np.float64)
    raise ValueError(name)


def _live(x, mask):
    return x if mask is None else np.where(np.asarray(mask)[:, None] != 0, x, 0.0)


def glu_fwd(x, wg, wu, name, mask=None):
    """(h, g, u)."""
    x = _live(x, mask)
    g, u = x @ wg.T, x @ wu.T
    return act(name, g)[0] * u, g, u


def glu_bwd(dh, g, u, name, mask=None):
    """(dgate, dup, h) from the projections."""
    dh, g, u = _live(dh, mask), _live(g, mask), _live(u, mask)
    a, slope = act(name, g)
    return dh * u * slope, dh * a, a * u


# --------------------------------------------------------------------- AdamW ----

_U = np.uint64
_LOW = _U(0xFFFFFFFF)


def _mul(x, k):
    return (x * _U(k)) & _LOW


def _mix(x):
    x = x ^ (x >> _U(16))
    x = _mul(x, 0x6A09E667)
    x ^= x >> _U(15)
    x = _mul(x, 0xBB67AE85)
    return x ^ (x >> _U(16))


def random_bits(places, seed, step):
    """For each place: 16 bits for m, for v and for the parameter."""
    a = _mix((_U(seed) & _LOW) ^ _mix(((_U(seed) >> _U(32)) + _U(0x3C6EF372)) & _LOW))
    k0 = _mix((_U(step) & _LOW) ^ _mix(((_U(step) >> _U(32)) + a) & _LOW))
    k1 = _mix((k0 + _U(0x510E527F)) & _LOW)
    i = np.asarray(places).astype(np.uint64)
    far = _mix(i >> _U(32))  # each 2^32 places have keys of their own; 0 for the first
    k0, k1 = k0 ^ far, (k1 + _mix(_mul(far, 0x1F83D9AB))) & _LOW
    x = (i & _LOW) ^ k0
    x ^= x >> _U(16)
    x = _mul(x, 0x6A09E667)
    x ^= x >> _U(15)
    x = (x + k1) & _LOW
    x = _mul(x, 0xBB67AE85)
    x ^= x >> _U(16)
    y = _mul(x ^ k1, 0x5BE0CD19)
    y ^= y >> _U(16)
    low = _U(0xFFFF)
    return (x & low).astype(np.float64), (x >> _U(16)).astype(np.float64), (y & low).astype(
        np.float64)


def e4m3_values():
    """The 127 finite values from 0 to 448, in the order of their codes."""
    c = np.arange(127)
    e, f = c >> 3, c & 7
    return np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))


def to_8(y, power, u):
    """A moment (packed, fp64) in 8 bits: (code, chance of the upper neighbour, the
    lower neighbour's code, scales). power 2: by the squares."""
    n = y.size
    blocks = -(-n // BLOCK)
    pad = np.zeros(blocks * BLOCK)
    pad[:n] = y
    pad = pad.reshape(blocks, BLOCK)
    size = np.where(np.isfinite(pad), np.abs(pad), 0.0)
    top = size.max(1)
    top = np.where(top >= LEAST, top, 0.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        a = np.where(top[:, None] > 0, size * TOP / top[:, None], 0.0).clip(0, TOP).reshape(-1)[:n]
    grid = e4m3_values()
    lo = np.clip(np.searchsorted(grid, a, side="right") - 1, 0, 125)
    chance = (a ** power - grid[lo] ** power) / (grid[lo + 1] ** power - grid[lo] ** power)
    code = lo + (u / 65536 < chance)
    if power == 2:
        some = (y > 0) & np.repeat(top > 0, BLOCK)[:n]
        code = np.where(some, np.maximum(code, 1), code)
    else:
        code = code | np.where(y < 0, 0x80, 0)
    code = np.where(np.isfinite(y), code, 0x7F)
    return code, chance, lo, top / TOP


def adamw(p, g, m, v, t, lr, betas=(0.9, 0.999), eps=1e-8, decay=0.0, scale=1.0):
    """(p, m, v) after step t."""
    g = g * scale
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    mh, vh = m / (1 - betas[0] ** t), v / (1 - betas[1] ** t)
    return p * (1 - lr * decay) - lr * mh / (np.sqrt(vh) + eps), m, v
