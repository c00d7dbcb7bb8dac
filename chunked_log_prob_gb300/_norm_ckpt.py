"""ctypes binding of the norm and 8-bit activation checkpoint calls of
include/grpo_gb300.h (argument marshalling only, like ``_binding``).

Tensors are 2-D with the last dimension contiguous; rows may be any distance
apart. Outputs are allocated when not given.

The calls are short (a decoded token's norm takes the GPU 3 us), so the common
case of every check is one expression; what it refuses is looked at again for
the message.
"""

from __future__ import annotations

import ctypes
from functools import lru_cache
from typing import NamedTuple

import torch

from ._binding import GRPO_OK, GrpoError, GrpoNormDesc, call_on, lib

_F32 = torch.float32
_U8 = torch.uint8
_BF16 = torch.bfloat16
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_KINDS = {"layer": 0, "rms": 1}
_byref = ctypes.byref
_empty, _empty_like = torch.empty, torch.empty_like


class Checkpoint8:
    """An activation [n_tokens, hidden] in 8 bits: e4m3 values, one power of two
    per 32 columns of a row. ``data`` is the library's buffer (uint8); ``q`` and
    ``exponents`` are views of it: x is about q * 2^(exponents - 127)."""

    __slots__ = ("data", "n_tokens", "hidden")

    def __init__(self, data: torch.Tensor, n_tokens: int, hidden: int):
        self.data, self.n_tokens, self.hidden = data, n_tokens, hidden

    def __repr__(self):
        return f"Checkpoint8(n_tokens={self.n_tokens}, hidden={self.hidden}, data={self.data.device})"

    def _layout(self):
        return _ckpt_layout(self.n_tokens, self.hidden)[:3]

    @property
    def q(self) -> torch.Tensor:
        """float8_e4m3fn [n_tokens, hidden]."""
        n, d = self.n_tokens, self.hidden
        ldq = _ckpt_layout(n, d)[0]
        return self.data.view(torch.float8_e4m3fn).as_strided((n, d), (ldq, 1))

    @property
    def exponents(self) -> torch.Tensor:
        """uint8 [n_tokens, ceil(hidden / 32)]: k + 127."""
        n, d = self.n_tokens, self.hidden
        _, off, lde, _ = _ckpt_layout(n, d)
        data = self.data
        return data.as_strided((n, -(-d // 32)), (lde, 1), data.storage_offset() + off)


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


# ------------------------------------------------------------------ checks ----


def _type_of_rows(t, name):
    """The library's code for the type of a 2-D tensor."""
    if t.dim() != 2:
        raise ValueError(f"{name}: expected 2 dimensions, got {t.dim()}")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected bfloat16, float16 or float32, got {t.dtype}")
    return code


def _rows(t, name, dtype, shape, device):
    """Checks a tensor whose rows may be apart; its row stride (0: packed)."""
    if t.dtype is dtype and t.shape == shape and t.device == device:
        if t.is_contiguous():
            return 0
        n, d = shape
        if n <= 1 and (d <= 1 or t.stride(1) == 1):
            return 0  # a single row has no distance to the next
        if d <= 1 or t.stride(1) == 1:
            s = t.stride(0)
            if s >= d:
                return s
            raise ValueError(f"{name}: rows overlap (stride {s} < {d} columns)")
        raise ValueError(f"{name}: the last dimension must be contiguous")
    _refuse(t, name, dtype, shape, device)


def _packed(t, name, dtype, shape, device):
    """Checks a contiguous tensor; its address."""
    if (t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        return t.data_ptr()
    _refuse(t, name, dtype, shape, device)


def _refuse(t, name, dtype, shape, device):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    raise ValueError(f"{name}: must be contiguous")


def _kind(kind):
    k = _KINDS.get(kind)
    if k is None:
        raise ValueError(f"kind: expected 'layer' or 'rms', got {kind!r}")
    return k


def _param(t, name, dtype, d, device):
    """Checks a weight or bias (of the rows' type or fp32); its address."""
    wt = t.dtype
    if wt is not dtype and wt is not _F32:
        raise TypeError(f"{name}: expected {dtype} or torch.float32, got {wt}")
    return _packed(t, name, wt, (d,), device)


def _like(t, stride):
    """A packed tensor of the shape and type of `t`, whose row stride is known."""
    return _empty_like(t) if stride == 0 else _empty(t.shape, dtype=t.dtype, device=t.device)


@lru_cache(maxsize=512)
def _ckpt_layout(n, d):
    """(bytes from row to row of q, where the exponents begin, bytes from row to
    row of them, bytes in all)."""
    out = [ctypes.c_int64() for _ in range(3)]
    _raise(lib.grpo_ckpt_layout(n, d, *map(_byref, out)), "grpo_ckpt_layout")
    return (*(v.value for v in out), grpo_ckpt_size(n, d))


def _ckpt(ckpt, n, d, device):
    """Checks a checkpoint; its address."""
    if not isinstance(ckpt, Checkpoint8):
        raise TypeError(f"ckpt: expected Checkpoint8, got {type(ckpt).__name__}")
    if ckpt.n_tokens != n or ckpt.hidden != d:
        raise ValueError(f"ckpt: expected shape {(n, d)}, got {(ckpt.n_tokens, ckpt.hidden)}")
    t = ckpt.data
    need = _ckpt_layout(n, d)[3]
    if t.dtype is not _U8 or t.dim() != 1 or not t.is_contiguous() or t.numel() < need:
        raise ValueError(f"ckpt: data must be contiguous uint8 of at least {need} bytes")
    if t.device != device:
        raise ValueError(f"ckpt: expected device {device}, got {t.device}")
    return t.data_ptr()


# ------------------------------------------------------------------- calls ----


def grpo_ckpt_size(n_tokens, hidden) -> int:
    out = ctypes.c_size_t(0)
    _raise(lib.grpo_ckpt_size(int(n_tokens), int(hidden), _byref(out)), "grpo_ckpt_size")
    return int(out.value)


def alloc_ckpt(n_tokens, hidden, device=None) -> Checkpoint8:
    n, d = int(n_tokens), int(hidden)
    return Checkpoint8(torch.empty(_ckpt_layout(n, d)[3], dtype=_U8, device=device), n, d)


def grpo_norm_fwd(x, weight=None, bias=None, *, residual=None, kind="rms", eps=1e-6, mask=None,
                  want_stats=True, want_ckpt=False, y=None, z=None, mean=None, rstd=None,
                  ckpt=None) -> NormForward:
    """Layer norm (kind="layer") or RMS norm of z = x + residual, row by row.

    Returns (y, z, mean, rstd, ckpt): mean and rstd (fp32 [N], mean for layer
    norm only) are what ``grpo_norm_bwd`` needs; ckpt is z's 8-bit checkpoint.
    Masked rows (mask 0) are not read; their outputs are zeros.
    """
    code = _type_of_rows(x, "x")
    shape, dt, dev = x.shape, x.dtype, x.device
    n, d = shape
    k = _kind(kind)
    sx = _rows(x, "x", dt, shape, dev)
    pw = pb = pr = pz = pm = ps = pmask = pc = None
    wt = 2
    sr = sz = 0
    if weight is not None:
        pw = _param(weight, "weight", dt, d, dev)
        wt = _DTYPES[weight.dtype]
    if bias is not None:
        pb = _param(bias, "bias", dt, d, dev)
        if weight is not None and weight.dtype is not bias.dtype:
            raise TypeError(f"bias: expected weight's type {weight.dtype}, got {bias.dtype}")
        wt = _DTYPES[bias.dtype]
    if residual is not None:
        sr = _rows(residual, "residual", dt, shape, dev)
        pr = residual.data_ptr()
        if z is None:
            z = _like(x, sx)
        else:
            sz = _rows(z, "z", dt, shape, dev)
        pz = z.data_ptr()
    elif z is not None:
        raise ValueError("z: is x itself without a residual")
    if mask is not None:
        pmask = _packed(mask, "mask", _U8, (n,), dev)
    sy = 0
    if y is None:
        y = _like(x, sx)
    else:
        sy = _rows(y, "y", dt, shape, dev)
    if mean is not None:
        if k:
            raise ValueError("mean: RMS norm has none")
        pm = _packed(mean, "mean", _F32, (n,), dev)
    elif want_stats and not k:
        mean = _empty(n, dtype=_F32, device=dev)
        pm = mean.data_ptr()
    if rstd is not None:
        ps = _packed(rstd, "rstd", _F32, (n,), dev)
    elif want_stats:
        rstd = _empty(n, dtype=_F32, device=dev)
        ps = rstd.data_ptr()
    if ckpt is None and want_ckpt:
        ckpt = Checkpoint8(_empty(_ckpt_layout(n, d)[3], dtype=_U8, device=dev), n, d)
        pc = ckpt.data.data_ptr()
    elif ckpt is not None:
        pc = _ckpt(ckpt, n, d, dev)
    desc = GrpoNormDesc(n, d, code, wt, k, eps, 0, sx, sr, sy, sz)
    rc = call_on(dev, lib.grpo_norm_fwd, x.data_ptr(), pr, pw, pb, pmask, y.data_ptr(), pz, pm, ps,
                 pc, _byref(desc))
    if rc:
        raise GrpoError(rc, "grpo_norm_fwd")
    return NormForward(y, x if residual is None else z, mean, rstd, ckpt)


@lru_cache(maxsize=512)
def _norm_workspace(n, d):
    out = ctypes.c_size_t(0)
    desc = GrpoNormDesc(n, d)
    _raise(lib.grpo_norm_workspace_size(_byref(desc), _byref(out)), "grpo_norm_workspace_size")
    return int(out.value)


def grpo_norm_workspace_size(n_tokens, hidden) -> int:
    return _norm_workspace(int(n_tokens), int(hidden))


def grpo_norm_bwd(dy, x, weight, mean, rstd, *, dres=None, kind="rms", mask=None,
                  want_dweight=None, want_dbias=False, add_dweight=None, add_dbias=None, dx=None,
                  dweight=None, dbias=None, workspace=None) -> NormBackward:
    """Gradients of ``grpo_norm_fwd``. ``x`` is the normed stream z, or its
    Checkpoint8; ``dres`` is the gradient that reaches z past the norm.

    Returns (dx, dweight, dbias): dx is the gradient of x and of residual;
    dweight and dbias are fp32 [D], added to add_dweight and add_dbias (which
    may be the outputs themselves). dweight is left out without a weight.
    """
    code = _type_of_rows(dy, "dy")
    shape, dt, dev = dy.shape, dy.dtype, dy.device
    n, d = shape
    k = _kind(kind)
    sdy = _rows(dy, "dy", dt, shape, dev)
    px = pc = pw = pmean = pmask = pr = pdw = pdb = paw = pab = pws = None
    wt = 2
    sx = sr = sdx = ws_bytes = 0
    if weight is not None:
        pw = _param(weight, "weight", dt, d, dev)
        wt = _DTYPES[weight.dtype]
    if isinstance(x, Checkpoint8):
        pc = _ckpt(x, n, d, dev)
    else:
        sx = _rows(x, "x", dt, shape, dev)
        px = x.data_ptr()
    if mean is not None:
        if k:
            raise ValueError("mean: RMS norm has none")
        pmean = _packed(mean, "mean", _F32, (n,), dev)
    elif not k:
        raise ValueError("mean: needed by layer norm")
    ps = _packed(rstd, "rstd", _F32, (n,), dev)
    if mask is not None:
        pmask = _packed(mask, "mask", _U8, (n,), dev)
    if dres is not None:
        sr = _rows(dres, "dres", dt, shape, dev)
        pr = dres.data_ptr()
    if dx is None:
        dx = _like(dy, sdy)
    else:
        sdx = _rows(dx, "dx", dt, shape, dev)
    if want_dweight is None:
        want_dweight = weight is not None
    vec = (d,)
    if dweight is not None:
        pdw = _packed(dweight, "dweight", _F32, vec, dev)
    elif want_dweight or add_dweight is not None:
        dweight = _empty(d, dtype=_F32, device=dev)
        pdw = dweight.data_ptr()
    if dbias is not None:
        pdb = _packed(dbias, "dbias", _F32, vec, dev)
    elif want_dbias or add_dbias is not None:
        dbias = _empty(d, dtype=_F32, device=dev)
        pdb = dbias.data_ptr()
    if add_dweight is not None:
        paw = _packed(add_dweight, "add_dweight", _F32, vec, dev)
    if add_dbias is not None:
        pab = _packed(add_dbias, "add_dbias", _F32, vec, dev)
    if workspace is None:
        if pdw is not None or pdb is not None:
            workspace = _empty(_norm_workspace(n, d), dtype=_U8, device=dev)
    if workspace is not None:
        if workspace.device != dev:
            raise ValueError(f"workspace: expected device {dev}, got {workspace.device}")
        pws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    desc = GrpoNormDesc(n, d, code, wt, k, 0.0, 0, sx, 0, 0, 0, sdy, sr, sdx)
    rc = call_on(dev, lib.grpo_norm_bwd, dy.data_ptr(), px, pc, pw, pmean, ps, pmask, pr,
                 dx.data_ptr(), pdw, pdb, paw, pab, _byref(desc), pws, ws_bytes)
    if rc:
        raise GrpoError(rc, "grpo_norm_bwd")
    return NormBackward(dx, dweight, dbias)


def grpo_ckpt_pack(x, *, mask=None, ckpt=None) -> Checkpoint8:
    """The 8-bit checkpoint of x [N, D]; masked rows are kept as zeros, unread."""
    code = _type_of_rows(x, "x")
    shape, dev = x.shape, x.device
    n, d = shape
    sx = _rows(x, "x", x.dtype, shape, dev)
    pmask = None if mask is None else _packed(mask, "mask", _U8, (n,), dev)
    if ckpt is None:
        ckpt = Checkpoint8(_empty(_ckpt_layout(n, d)[3], dtype=_U8, device=dev), n, d)
        pc = ckpt.data.data_ptr()
    else:
        pc = _ckpt(ckpt, n, d, dev)
    rc = call_on(dev, lib.grpo_ckpt_pack, x.data_ptr(), pmask, pc, n, d, code, sx)
    if rc:
        raise GrpoError(rc, "grpo_ckpt_pack")
    return ckpt


def grpo_ckpt_unpack(ckpt, dtype=torch.bfloat16, *, out=None) -> torch.Tensor:
    """The values a checkpoint stands for, rounded once to ``dtype``."""
    if not isinstance(ckpt, Checkpoint8):
        raise TypeError(f"ckpt: expected Checkpoint8, got {type(ckpt).__name__}")
    data = ckpt.data
    dev = data.device
    n, d = shape = ckpt.n_tokens, ckpt.hidden
    pc = _ckpt(ckpt, n, d, dev)
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"dtype: expected bfloat16, float16 or float32, got {dtype}")
    so = 0
    if out is None:
        out = _empty(shape, dtype=dtype, device=dev)
    else:
        so = _rows(out, "out", dtype, shape, dev)
    rc = call_on(dev, lib.grpo_ckpt_unpack, pc, out.data_ptr(), n, d, code, so)
    if rc:
        raise GrpoError(rc, "grpo_ckpt_unpack")
    return out


@lru_cache(maxsize=512)
def _wgrad_workspace(n, out_features, in_features):
    out = ctypes.c_size_t(0)
    _raise(lib.grpo_ckpt_wgrad_workspace_size(n, out_features, in_features, _byref(out)),
           "grpo_ckpt_wgrad_workspace_size")
    return int(out.value)


def grpo_ckpt_wgrad_workspace_size(n_tokens, out_features, in_features) -> int:
    return _wgrad_workspace(int(n_tokens), int(out_features), int(in_features))


def grpo_ckpt_wgrad(dy, ckpt, *, add=None, dW=None, workspace=None) -> torch.Tensor:
    """dW = add + dy^T X of a linear layer whose input X was kept as ``ckpt``.

    dy is bf16 [N, out]; dW and add are fp32 [out, in] and may be the same. A wait
    on the device that runs out leaves NaN (and its status in the workspace).
    """
    if dy.dim() != 2:
        raise ValueError(f"dy: expected 2 dimensions, got {dy.dim()}")
    dev = dy.device
    n, out = dy.shape
    sdy = _rows(dy, "dy", _BF16, dy.shape, dev)
    if not isinstance(ckpt, Checkpoint8):
        raise TypeError(f"ckpt: expected Checkpoint8, got {type(ckpt).__name__}")
    d = ckpt.hidden
    pc = _ckpt(ckpt, n, d, dev)
    shape = (out, d)
    if dW is None:
        dW = _empty(shape, dtype=_F32, device=dev)
        pdw = dW.data_ptr()
    else:
        pdw = _packed(dW, "dW", _F32, shape, dev)
    pa = None if add is None else _packed(add, "add", _F32, shape, dev)
    if workspace is None:
        workspace = _empty(_wgrad_workspace(n, out, d), dtype=_U8, device=dev)
    elif workspace.device != dev:
        raise ValueError(f"workspace: expected device {dev}, got {workspace.device}")
    rc = call_on(dev, lib.grpo_ckpt_wgrad, dy.data_ptr(), pc, pa, pdw, n, out, d, sdy,
                 workspace.data_ptr(), workspace.numel() * workspace.element_size())
    if rc:
        raise GrpoError(rc, "grpo_ckpt_wgrad")
    return dW


def grpo_selftest_lose_copy(index: int) -> None:
    """This thread's next ``grpo_norm_fwd`` or ``grpo_norm_bwd`` leaves out the copies
    of row ``index`` and of its CTA's later rows, or its next ``grpo_ckpt_wgrad``
    that of its first CTA's 64-token stage ``index`` (-1: none). The call gives up
    after about a second."""
    _raise(lib.grpo_selftest_lose_copy(int(index)), "grpo_selftest_lose_copy")
