"""ctypes binding of the gated feed-forward calls of include/grpo_gb300.h (argument
marshalling only, like ``_norm_ckpt``).

Tensors are 2-D with the last dimension contiguous; rows may be a multiple of 8
elements apart. Outputs are allocated when not given.
"""

from __future__ import annotations

import ctypes
from functools import lru_cache
from typing import NamedTuple

import torch

from ._binding import GRPO_OK, GrpoError, GrpoGluDesc, call_on, lib
from ._norm_ckpt import Checkpoint8, _ckpt, _ckpt_layout, _packed, _rows

_F32, _U8 = torch.float32, torch.uint8
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
_byref = ctypes.byref
_empty = torch.empty


class GluForward(NamedTuple):
    h: torch.Tensor
    gate: torch.Tensor | None  # the projections, where kept
    up: torch.Tensor | None
    ckpt: Checkpoint8 | None  # of h


class GluBackward(NamedTuple):
    dgate: torch.Tensor
    dup: torch.Tensor
    dx: torch.Tensor | None
    h: torch.Tensor | None


def _act(act):
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act: expected one of {', '.join(map(repr, _ACTS))}, got {act!r}")
    return code


def _type_of(t, name):
    """The library's code for the type of a 2-D tensor."""
    if t.dim() != 2:
        raise ValueError(f"{name}: expected 2 dimensions, got {t.dim()}")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected bfloat16 or float16, got {t.dtype}")
    return code


def _weights(w_gate, w_up, dt, dev, d):
    """Checks both weights; (inner, their row strides)."""
    if w_gate.dim() != 2:
        raise ValueError(f"w_gate: expected 2 dimensions, got {w_gate.dim()}")
    shape = w_gate.shape
    if shape[1] != d:
        raise ValueError(f"w_gate: expected {d} columns, got {shape[1]}")
    return shape[0], _rows(w_gate, "w_gate", dt, shape, dev), _rows(w_up, "w_up", dt, shape, dev)


def _both(a, b, names):
    if (a is None) != (b is None):
        raise ValueError(f"{names}: both or neither")


def grpo_glu_fwd(x, w_gate, w_up, *, act="silu", mask=None, want_gates=False, want_ckpt=False,
                 h=None, gate=None, up=None, ckpt=None) -> GluForward:
    """h = act(x w_gate^T) * (x w_up^T), x [N, D], weights [F, D], bf16 or fp16.

    Returns (h, gate, up, ckpt): the projections x w_gate^T and x w_up^T as
    ``grpo_glu_bwd`` reads them (with want_gates), and h's 8-bit checkpoint (with
    want_ckpt). Masked rows (mask 0) have no influence; their outputs are zeros.
    """
    code, k = _type_of(x, "x"), _act(act)
    n, d = x.shape
    dt, dev = x.dtype, x.device
    sx = _rows(x, "x", dt, x.shape, dev)
    f, swg, swu = _weights(w_gate, w_up, dt, dev, d)
    shape = (n, f)
    pg = pu = pc = pm = None
    sh = sg = su = 0
    if mask is not None:
        pm = _packed(mask, "mask", _U8, (n,), dev)
    if h is None:
        h = _empty(shape, dtype=dt, device=dev)
    else:
        sh = _rows(h, "h", dt, shape, dev)
    if gate is not None or up is not None:
        _both(gate, up, "gate and up")
        sg, su = _rows(gate, "gate", dt, shape, dev), _rows(up, "up", dt, shape, dev)
    elif want_gates:
        gate, up = _empty(shape, dtype=dt, device=dev), _empty(shape, dtype=dt, device=dev)
    if gate is not None:
        pg, pu = gate.data_ptr(), up.data_ptr()
    if ckpt is not None:
        pc = _ckpt(ckpt, n, f, dev)
    elif want_ckpt:
        ckpt = Checkpoint8(_empty(_ckpt_layout(n, f)[3], dtype=_U8, device=dev), n, f)
        pc = ckpt.data.data_ptr()
    desc = GrpoGluDesc(n, d, f, code, k, sx, swg, swu, sh, sg, su)
    rc = call_on(dev, lib.grpo_glu_fwd, x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), pm,
                 h.data_ptr(), pg, pu, pc, _byref(desc))
    if rc:
        raise GrpoError(rc, "grpo_glu_fwd")
    return GluForward(h, gate, up, ckpt)


def grpo_glu_bwd(dh, x, w_gate, w_up, *, gate=None, up=None, act="silu", mask=None, want_dx=True,
                 want_h=False, dgate=None, dup=None, dx=None, h=None, workspace=None) -> GluBackward:
    """Gradients of ``grpo_glu_fwd``: dgate, dup [N, F] of the projections, dx [N, D].

    ``gate`` and ``up`` are the projections that the forward pass kept (x may be None
    then); without them they are computed again from x. want_h: h again, for the
    weight gradient of the layer that it went into. dgate and dup may be given as dh,
    gate and up themselves, whose contents are lost then. The workspace
    (``grpo_glu_bwd_workspace_size`` bytes) is allocated when not given.
    """
    code, k = _type_of(dh, "dh"), _act(act)
    shape, dt, dev = dh.shape, dh.dtype, dh.device
    n, f = shape
    sdh = _rows(dh, "dh", dt, shape, dev)
    _both(gate, up, "gate and up")
    if w_gate.dim() != 2 or w_gate.shape[0] != f:
        raise ValueError(f"w_gate: expected [{f}, D], got {tuple(w_gate.shape)}")
    d = w_gate.shape[1]
    _, swg, swu = _weights(w_gate, w_up, dt, dev, d)
    px = pg = pu = pm = pdx = ph = None
    sx = sg = su = sdg = sdu = sdx = sh = 0
    if gate is not None:
        sg, su = _rows(gate, "gate", dt, shape, dev), _rows(up, "up", dt, shape, dev)
        pg, pu = gate.data_ptr(), up.data_ptr()
    elif x is None:
        raise ValueError("x: needed without gate and up")
    if x is not None:
        sx = _rows(x, "x", dt, (n, d), dev)
        px = x.data_ptr()
    if mask is not None:
        pm = _packed(mask, "mask", _U8, (n,), dev)
    if dgate is None:
        dgate = _empty(shape, dtype=dt, device=dev)
    else:
        sdg = _rows(dgate, "dgate", dt, shape, dev)
    if dup is None:
        dup = _empty(shape, dtype=dt, device=dev)
    else:
        sdu = _rows(dup, "dup", dt, shape, dev)
    if dx is not None:
        sdx = _rows(dx, "dx", dt, (n, d), dev)
        pdx = dx.data_ptr()
    elif want_dx:
        dx = _empty((n, d), dtype=dt, device=dev)
        pdx = dx.data_ptr()
    if h is not None:
        sh = _rows(h, "h", dt, shape, dev)
        ph = h.data_ptr()
    elif want_h:
        h = _empty(shape, dtype=dt, device=dev)
        ph = h.data_ptr()
    pw, nw = None, 0
    if pdx is not None:
        if workspace is None:
            nw = _bwd_workspace(n, f, d)
            if nw:
                workspace = _empty(nw, dtype=_U8, device=dev)
                pw = workspace.data_ptr()
        elif workspace.device != dev:
            raise ValueError(f"workspace: expected device {dev}, got {workspace.device}")
        else:
            pw, nw = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    desc = GrpoGluDesc(n, d, f, code, k, sx, swg, swu, sh, sg, su, sdh, sdg, sdu, sdx)
    rc = call_on(dev, lib.grpo_glu_bwd, dh.data_ptr(), px, w_gate.data_ptr(), w_up.data_ptr(), pg,
                 pu, pm, dgate.data_ptr(), dup.data_ptr(), pdx, ph, _byref(desc), pw, nw)
    if rc:
        raise GrpoError(rc, "grpo_glu_bwd")
    return GluBackward(dgate, dup, dx, h)


@lru_cache(maxsize=512)
def _bwd_workspace(n, f, d):
    out = ctypes.c_size_t(0)
    rc = lib.grpo_glu_bwd_workspace_size(n, f, d, _byref(out))
    if rc != GRPO_OK:
        raise GrpoError(rc, "grpo_glu_bwd_workspace_size")
    return int(out.value)


def grpo_glu_bwd_workspace_size(n_tokens, inner, hidden) -> int:
    return _bwd_workspace(int(n_tokens), int(inner), int(hidden))


@lru_cache(maxsize=512)
def _wgrad_workspace(n, f, d):
    out = ctypes.c_size_t(0)
    rc = lib.grpo_glu_wgrad_workspace_size(n, f, d, _byref(out))
    if rc != GRPO_OK:
        raise GrpoError(rc, "grpo_glu_wgrad_workspace_size")
    return int(out.value)


def grpo_glu_wgrad_workspace_size(n_tokens, inner, hidden) -> int:
    return _wgrad_workspace(int(n_tokens), int(inner), int(hidden))


def grpo_glu_wgrad(dgate, dup, x, *, add_gate=None, add_up=None, dw_gate=None, dw_up=None,
                   workspace=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(add_gate + dgate^T x, add_up + dup^T x), fp32 [F, D] each.

    add_gate and add_up may be the outputs themselves. Masked tokens: dgate and dup
    are 0 there, as ``grpo_glu_bwd`` leaves them, and x is finite.
    """
    code = _type_of(dgate, "dgate")
    n, f = dgate.shape
    dt, dev = dgate.dtype, dgate.device
    if x.dim() != 2:
        raise ValueError(f"x: expected 2 dimensions, got {x.dim()}")
    d = x.shape[1]
    sg = _rows(dgate, "dgate", dt, (n, f), dev)
    su = _rows(dup, "dup", dt, (n, f), dev)
    sx = _rows(x, "x", dt, (n, d), dev)
    shape = (f, d)
    if dw_gate is None:
        dw_gate = _empty(shape, dtype=_F32, device=dev)
    if dw_up is None:
        dw_up = _empty(shape, dtype=_F32, device=dev)
    pdg, pdu = _packed(dw_gate, "dw_gate", _F32, shape, dev), _packed(dw_up, "dw_up", _F32, shape,
                                                                      dev)
    pag = None if add_gate is None else _packed(add_gate, "add_gate", _F32, shape, dev)
    pau = None if add_up is None else _packed(add_up, "add_up", _F32, shape, dev)
    if workspace is None:
        workspace = _empty(_wgrad_workspace(n, f, d), dtype=_U8, device=dev)
    elif workspace.device != dev:
        raise ValueError(f"workspace: expected device {dev}, got {workspace.device}")
    desc = GrpoGluDesc(n, d, f, code, 0, sx, 0, 0, 0, 0, 0, 0, sg, su)
    rc = call_on(dev, lib.grpo_glu_wgrad, dgate.data_ptr(), dup.data_ptr(), x.data_ptr(), pag, pau,
                 pdg, pdu, _byref(desc), workspace.data_ptr(),
                 workspace.numel() * workspace.element_size())
    if rc:
        raise GrpoError(rc, "grpo_glu_wgrad")
    return dw_gate, dw_up
