"""fp64 CPU oracle of the norms and the 8-bit activation checkpoint.

Plain definitions in numpy; nothing of the package is used. Inputs are numpy
arrays (any float type; callers widen bf16 exactly).

The package's library adds these next to the chunked selective log-softmax of
"GRPO with 7x longer context" (Unsloth docs, section "Offloading activations
for log-softmax": activations of the backward pass are what memory goes to).
"""

from __future__ import annotations

import numpy as np

BLOCK = 32
MIN_EXP = -117
BIAS = 127


def e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 (ties to even) of |v| <= 448, as float64; NaN stays NaN."""
    v = np.asarray(v, np.float64)
    _, e = np.frexp(v)  # |v| in [2^(e-1), 2^e)
    step = np.ldexp(1.0, np.maximum(e, -5) - 4)
    return np.rint(v / step) * step


def ckpt_pack(x: np.ndarray, type_max: float, mask=None):
    """(q float64 [N, D], exponents int [N, ceil(D / 32)], biased by 127)."""
    x = np.array(x, np.float64)
    n, d = x.shape
    if mask is not None:
        x[np.asarray(mask) == 0] = 0.0
    nb = -(-d // BLOCK)
    q = np.zeros((n, d))
    ex = np.zeros((n, nb), np.int64)
    for b in range(nb):
        s = slice(b * BLOCK, min(d, (b + 1) * BLOCK))
        blk = x[:, s]
        fin = np.isfinite(blk)
        a = np.max(np.where(fin, np.abs(blk), 0.0), axis=1, initial=0.0)
        m, e = np.frexp(a)  # a = (2 m) 2^(e - 1)
        k = np.where(2 * m <= 1.75, e - 1 - 8, e - 1 - 7)
        k = np.maximum(np.where(a > 0, k, MIN_EXP), MIN_EXP)
        v = np.where(fin, blk, 0.0)
        v = np.ldexp(v, -k[:, None])
        r = e4m3(v)
        over = np.ldexp(np.abs(r), k[:, None]) > type_max
        r = np.where(over, np.sign(r) * 240.0, r)
        q[:, s] = np.where(fin, r, np.nan)
        ex[:, b] = k + BIAS
    return q, ex


def ckpt_expand(q: np.ndarray, ex: np.ndarray) -> np.ndarray:
    d = q.shape[1]
    return np.ldexp(q, np.repeat(ex - BIAS, BLOCK, axis=1)[:, :d])


def norm_fwd(z, weight, bias, kind, eps, mask=None):
    """y, mean, rstd of the stream z (mean 0 for kind "rms"); masked rows 0."""
    z = np.array(z, np.float64)
    n, d = z.shape
    live = np.ones(n, bool) if mask is None else np.asarray(mask) != 0
    z[~live] = 0.0
    mean = z.mean(axis=1) if kind == "layer" else np.zeros(n)
    c = z - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1) + eps)
    w = np.ones(d) if weight is None else np.asarray(weight, np.float64)
    b = np.zeros(d) if bias is None else np.asarray(bias, np.float64)
    y = c * rstd[:, None] * w + b
    return y * live[:, None], mean * live, rstd * live


def norm_bwd(dy, z, weight, mean, rstd, kind, dres=None, mask=None):
    """dx, dweight, dbias from the statistics given."""
    dy, z = np.array(dy, np.float64), np.array(z, np.float64)
    n, d = dy.shape
    live = np.ones(n, bool) if mask is None else np.asarray(mask) != 0
    dy[~live] = 0.0
    z[~live] = 0.0
    rstd = np.where(live, np.asarray(rstd, np.float64), 0.0)[:, None]
    mu = np.zeros((n, 1)) if mean is None else np.where(live, np.asarray(mean, np.float64), 0.0)[:, None]
    w = np.ones(d) if weight is None else np.asarray(weight, np.float64)
    h = (z - mu) * rstd
    u = dy * w
    dx = u - h * (u * h).mean(axis=1, keepdims=True)
    if kind == "layer":
        dx = dx - u.mean(axis=1, keepdims=True)
    dx = dx * rstd
    if dres is not None:
        r = np.array(dres, np.float64)
        r[~live] = 0.0
        dx = dx + r
    return dx, (dy * h).sum(axis=0), dy.sum(axis=0)


def wgrad(dy, x, add=None):
    dw = np.asarray(dy, np.float64).T @ np.asarray(x, np.float64)
    return dw if add is None else dw + np.asarray(add, np.float64)
