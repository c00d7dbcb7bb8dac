"""ctypes binding of the norm and 8-bit activation checkpoint calls of
include/grpo_gb300.h (argument marshalling only, like ``_binding``).

Tensors are 2-D with the last dimension contiguous; rows may be any distance
apart. Outputs are allocated when not given.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import NamedTuple

import torch

from ._binding import GRPO_OK, GrpoError, GrpoNormDesc, _check, _ptr, _stream, lib

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_KINDS = {"layer": 0, "rms": 1}


@dataclass(frozen=True)
class Checkpoint8:
    """An activation [n_tokens, hidden] in 8 bits: e4m3 values, one power of two
    per 32 columns of a row. ``data`` is the library's buffer (uint8); ``q`` and
    ``exponents`` are views of it: x is about q * 2^(exponents - 127)."""

    data: torch.Tensor
    n_tokens: int
    hidden: int

    def _layout(self):
        out = [ctypes.c_int64() for _ in range(3)]
        _raise(lib.grpo_ckpt_layout(self.n_tokens, self.hidden, *map(ctypes.byref, out)),
               "grpo_ckpt_layout")
        return [int(v.value) for v in out]

    @property
    def q(self) -> torch.Tensor:
        """float8_e4m3fn [n_tokens, hidden]."""
        ldq, _, _ = self._layout()
        return self.data.view(torch.float8_e4m3fn).as_strided((self.n_tokens, self.hidden),
                                                              (ldq, 1))

    @property
    def exponents(self) -> torch.Tensor:
        """uint8 [n_tokens, ceil(hidden / 32)]: k + 127."""
        _, off, lde = self._layout()
        return self.data.as_strided((self.n_tokens, -(-self.hidden // 32)), (lde, 1),
                                    self.data.storage_offset() + off)


class NormForward(NamedTuple):
    y: torch.Tensor
    z: torch.Tensor  # the stream after the residual add (x itself without one)
    mean: torch.Tensor | None
    rstd: torch.Tensor | None
    ckpt: Checkpoint8 | None


class NormBackward(NamedTuple):
    dx: torch.Tensor
    dweight: torch.Tensor | None
    dbias: torch.Tensor | None


def _raise(rc, where):
    if rc != GRPO_OK:
        raise GrpoError(rc, where)


def _check_rows(t, name, dtype, shape, device):
    """Like ``_check``, for a tensor whose rows may be apart."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    if t.numel() and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: rows overlap (stride {t.stride(0)} < {t.shape[1]} columns)")


def _row_stride(t):
    # A single row has no distance to the next; torch may report any.
    return 0 if t is None or t.shape[0] <= 1 else t.stride(0)


def _need_cuda(device):
    if device.type != "cuda":
        raise ValueError(f"expected tensors on a CUDA device, got {device}")


def _rows_shape(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected 2 dimensions, got {t.dim()}")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name}: expected bfloat16, float16 or float32, got {t.dtype}")
    return t.shape


def _kind(kind):
    if kind not in _KINDS:
        raise ValueError(f"kind: expected 'layer' or 'rms', got {kind!r}")
    return _KINDS[kind]


def _check_weight(weight, bias, x):
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            if t.dtype not in (x.dtype, torch.float32):
                raise TypeError(f"{name}: expected {x.dtype} or torch.float32, got {t.dtype}")
            _check(t, name, t.dtype, (x.shape[1],), x.device)
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError(f"bias: expected weight's type {weight.dtype}, got {bias.dtype}")
    p = weight if weight is not None else bias
    return _DTYPES[p.dtype if p is not None else torch.float32]


def _check_ckpt(ckpt, n, d, device):
    if not isinstance(ckpt, Checkpoint8):
        raise TypeError(f"ckpt: expected Checkpoint8, got {type(ckpt).__name__}")
    if (ckpt.n_tokens, ckpt.hidden) != (n, d):
        raise ValueError(f"ckpt: expected shape {(n, d)}, got {(ckpt.n_tokens, ckpt.hidden)}")
    need = grpo_ckpt_size(n, d)
    t = ckpt.data
    if t.dtype != torch.uint8 or t.dim() != 1 or not t.is_contiguous() or t.numel() < need:
        raise ValueError(f"ckpt: data must be contiguous uint8 of at least {need} bytes")
    if t.device != device:
        raise ValueError(f"ckpt: expected device {device}, got {t.device}")


def grpo_ckpt_size(n_tokens, hidden) -> int:
    out = ctypes.c_size_t(0)
    _raise(lib.grpo_ckpt_size(int(n_tokens), int(hidden), ctypes.byref(out)), "grpo_ckpt_size")
    return int(out.value)


def alloc_ckpt(n_tokens, hidden, device=None) -> Checkpoint8:
    data = torch.empty(grpo_ckpt_size(n_tokens, hidden), dtype=torch.uint8, device=device)
    return Checkpoint8(data, int(n_tokens), int(hidden))


def grpo_norm_fwd(x, weight=None, bias=None, *, residual=None, kind="rms", eps=1e-6, mask=None,
                  want_stats=True, want_ckpt=False, y=None, z=None, mean=None, rstd=None,
                  ckpt=None) -> NormForward:
    """Layer norm (kind="layer") or RMS norm of z = x + residual, row by row.

    Returns (y, z, mean, rstd, ckpt): mean and rstd (fp32 [N], mean for layer
    norm only) are what ``grpo_norm_bwd`` needs; ckpt is z's 8-bit checkpoint.
    """
    n, d = _rows_shape(x, "x")
    dev, dt = x.device, x.dtype
    k = _kind(kind)
    wt = _check_weight(weight, bias, x)
    if residual is not None:
        _check_rows(residual, "residual", dt, (n, d), dev)
        if z is None:
            z = torch.empty((n, d), dtype=dt, device=dev)
        else:
            _check_rows(z, "z", dt, (n, d), dev)
    elif z is not None:
        raise ValueError("z: is x itself without a residual")
    if mask is not None:
        _check(mask, "mask", torch.uint8, (n,), dev)
    if y is None:
        y = torch.empty((n, d), dtype=dt, device=dev)
    else:
        _check_rows(y, "y", dt, (n, d), dev)
    if mean is not None:
        if k:
            raise ValueError("mean: RMS norm has none")
        _check(mean, "mean", torch.float32, (n,), dev)
    elif want_stats and not k:
        mean = torch.empty(n, dtype=torch.float32, device=dev)
    if rstd is not None:
        _check(rstd, "rstd", torch.float32, (n,), dev)
    elif want_stats:
        rstd = torch.empty(n, dtype=torch.float32, device=dev)
    if ckpt is not None:
        _check_ckpt(ckpt, n, d, dev)
    elif want_ckpt:
        ckpt = alloc_ckpt(n, d, dev)
    _need_cuda(dev)
    desc = GrpoNormDesc(n, d, _DTYPES[dt], wt, k, eps, 0, _row_stride(x), _row_stride(residual),
                        _row_stride(y), _row_stride(z), 0, 0, 0)
    _raise(lib.grpo_norm_fwd(_ptr(x), _ptr(residual), _ptr(weight), _ptr(bias), _ptr(mask),
                             _ptr(y), _ptr(z), _ptr(mean), _ptr(rstd),
                             _ptr(ckpt.data) if ckpt is not None else None,
                             ctypes.byref(desc), _stream(dev)), "grpo_norm_fwd")
    return NormForward(y, x if residual is None else z, mean, rstd, ckpt)


def grpo_norm_workspace_size(n_tokens, hidden) -> int:
    out = ctypes.c_size_t(0)
    desc = GrpoNormDesc(int(n_tokens), int(hidden), 0, 0, 0, 0.0, 0, 0, 0, 0, 0, 0, 0, 0)
    _raise(lib.grpo_norm_workspace_size(ctypes.byref(desc), ctypes.byref(out)),
           "grpo_norm_workspace_size")
    return int(out.value)


def grpo_norm_bwd(dy, x, weight, mean, rstd, *, dres=None, kind="rms", mask=None,
                  want_dweight=None, want_dbias=False, add_dweight=None, add_dbias=None, dx=None,
                  dweight=None, dbias=None, workspace=None) -> NormBackward:
    """Gradients of ``grpo_norm_fwd``. ``x`` is the normed stream z, or its
    Checkpoint8; ``dres`` is the gradient that reaches z past the norm.

    Returns (dx, dweight, dbias): dx is the gradient of x and of residual;
    dweight and dbias are fp32 [D], added to add_dweight and add_dbias (which
    may be the outputs themselves). dweight is left out without a weight.
    """
    n, d = _rows_shape(dy, "dy")
    dev, dt = dy.device, dy.dtype
    k = _kind(kind)
    wt = _check_weight(weight, None, dy)
    from_ckpt = isinstance(x, Checkpoint8)
    if from_ckpt:
        _check_ckpt(x, n, d, dev)
    else:
        _check_rows(x, "x", dt, (n, d), dev)
    if k and mean is not None:
        raise ValueError("mean: RMS norm has none")
    if not k:
        if mean is None:
            raise ValueError("mean: needed by layer norm")
        _check(mean, "mean", torch.float32, (n,), dev)
    _check(rstd, "rstd", torch.float32, (n,), dev)
    if mask is not None:
        _check(mask, "mask", torch.uint8, (n,), dev)
    if dres is not None:
        _check_rows(dres, "dres", dt, (n, d), dev)
    if dx is None:
        dx = torch.empty((n, d), dtype=dt, device=dev)
    else:
        _check_rows(dx, "dx", dt, (n, d), dev)
    if want_dweight is None:
        want_dweight = weight is not None
    if dweight is None and (want_dweight or add_dweight is not None):
        dweight = torch.empty(d, dtype=torch.float32, device=dev)
    if dbias is None and (want_dbias or add_dbias is not None):
        dbias = torch.empty(d, dtype=torch.float32, device=dev)
    for t, name in ((dweight, "dweight"), (dbias, "dbias"), (add_dweight, "add_dweight"),
                    (add_dbias, "add_dbias")):
        if t is not None:
            _check(t, name, torch.float32, (d,), dev)
    if workspace is None and (dweight is not None or dbias is not None):
        workspace = torch.empty(grpo_norm_workspace_size(n, d), dtype=torch.uint8, device=dev)
    _need_cuda(dev)
    desc = GrpoNormDesc(n, d, _DTYPES[dt], wt, k, 0.0, 0, 0 if from_ckpt else _row_stride(x), 0, 0,
                        0, _row_stride(dy), _row_stride(dres), _row_stride(dx))
    _raise(lib.grpo_norm_bwd(_ptr(dy), None if from_ckpt else _ptr(x),
                             _ptr(x.data) if from_ckpt else None, _ptr(weight), _ptr(mean),
                             _ptr(rstd), _ptr(mask), _ptr(dres), _ptr(dx), _ptr(dweight),
                             _ptr(dbias), _ptr(add_dweight), _ptr(add_dbias), ctypes.byref(desc),
                             _ptr(workspace), workspace.numel() if workspace is not None else 0,
                             _stream(dev)), "grpo_norm_bwd")
    return NormBackward(dx, dweight, dbias)


def grpo_ckpt_pack(x, *, mask=None, ckpt=None) -> Checkpoint8:
    """The 8-bit checkpoint of x [N, D]; masked rows are kept as zeros, unread."""
    n, d = _rows_shape(x, "x")
    _check_rows(x, "x", x.dtype, (n, d), x.device)
    if mask is not None:
        _check(mask, "mask", torch.uint8, (n,), x.device)
    if ckpt is None:
        ckpt = alloc_ckpt(n, d, x.device)
    else:
        _check_ckpt(ckpt, n, d, x.device)
    _need_cuda(x.device)
    _raise(lib.grpo_ckpt_pack(_ptr(x), _ptr(mask), _ptr(ckpt.data), n, d, _DTYPES[x.dtype],
                              _row_stride(x), _stream(x.device)), "grpo_ckpt_pack")
    return ckpt


def grpo_ckpt_unpack(ckpt, dtype=torch.bfloat16, *, out=None) -> torch.Tensor:
    """The values a checkpoint stands for, rounded once to ``dtype``."""
    dev = ckpt.data.device
    n, d = ckpt.n_tokens, ckpt.hidden
    _check_ckpt(ckpt, n, d, dev)
    if out is None:
        out = torch.empty((n, d), dtype=dtype, device=dev)
    _rows_shape(out, "out")
    _check_rows(out, "out", dtype, (n, d), dev)
    _need_cuda(dev)
    _raise(lib.grpo_ckpt_unpack(_ptr(ckpt.data), _ptr(out), n, d, _DTYPES[out.dtype],
                                _row_stride(out), _stream(dev)), "grpo_ckpt_unpack")
    return out


def grpo_ckpt_wgrad_workspace_size(n_tokens, out_features, in_features) -> int:
    out = ctypes.c_size_t(0)
    _raise(lib.grpo_ckpt_wgrad_workspace_size(int(n_tokens), int(out_features), int(in_features),
                                              ctypes.byref(out)),
           "grpo_ckpt_wgrad_workspace_size")
    return int(out.value)


def grpo_ckpt_wgrad(dy, ckpt, *, add=None, dW=None, workspace=None) -> torch.Tensor:
    """dW = add + dy^T X of a linear layer whose input X was kept as ``ckpt``.

    dy is bf16 [N, out]; dW and add are fp32 [out, in] and may be the same.
    """
    if dy.dim() != 2:
        raise ValueError(f"dy: expected 2 dimensions, got {dy.dim()}")
    n, out = dy.shape
    dev = dy.device
    _check_rows(dy, "dy", torch.bfloat16, (n, out), dev)
    if not isinstance(ckpt, Checkpoint8):
        raise TypeError(f"ckpt: expected Checkpoint8, got {type(ckpt).__name__}")
    d = ckpt.hidden
    _check_ckpt(ckpt, n, d, dev)
    if dW is None:
        dW = torch.empty((out, d), dtype=torch.float32, device=dev)
    else:
        _check(dW, "dW", torch.float32, (out, d), dev)
    if add is not None:
        _check(add, "add", torch.float32, (out, d), dev)
    if workspace is None:
        workspace = torch.empty(grpo_ckpt_wgrad_workspace_size(n, out, d), dtype=torch.uint8,
                                device=dev)
    _need_cuda(dev)
    _raise(lib.grpo_ckpt_wgrad(_ptr(dy), _ptr(ckpt.data), _ptr(add), _ptr(dW), n, out, d,
                               _row_stride(dy), _ptr(workspace), workspace.numel(), _stream(dev)),
           "grpo_ckpt_wgrad")
    return dW
