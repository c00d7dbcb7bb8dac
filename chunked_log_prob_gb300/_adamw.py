"""The optimizer's step: ctypes binding of grpo_adamw_step and grpo_grad_norm of
include/grpo_gb300.h, with the moments of each parameter kept in ``AdamW``.
"""

from __future__ import annotations

import ctypes
from functools import lru_cache
from operator import attrgetter
from typing import NamedTuple, Sequence

import numpy as np
import torch

from ._binding import GRPO_OK, GrpoAdamwParams, GrpoAdamwTensor, GrpoError, GrpoGrad, call_on, lib

_F32, _U8, _E4M3 = torch.float32, torch.uint8, torch.float8_e4m3fn
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_PARAMS = (torch.float32, torch.bfloat16)
_COPIES = (torch.bfloat16, torch.float16)
_BLOCK = 128
_GRAD = np.dtype(GrpoGrad)
_byref = ctypes.byref
_data_ptr, _numel = torch.Tensor.data_ptr, torch.Tensor.numel
_packed, _device_index = torch.Tensor.is_contiguous, torch.Tensor.get_device
# (tensors, addresses, indices): whether those tensors lie there; a third faster than a map.
_lie_at = torch._C._tensors_data_ptrs_at_indices_equal
_dtype, _shape, _nbytes = attrgetter("dtype"), attrgetter("shape"), attrgetter("nbytes")


class GradNorm(NamedTuple):
    norm: torch.Tensor   # fp32, 0-d
    scale: torch.Tensor  # fp32, 0-d: min(1, max_norm / (norm + 1e-6)); NaN: not finite


class AdamState(NamedTuple):
    """Moments of one parameter, packed. 32 bits: m and v in fp32. 8 bits: e4m3 with a
    scale per 128 values: the moments are m m_scale and (v v_scale)^2."""

    m: torch.Tensor
    v: torch.Tensor
    m_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None

    def moments(self) -> tuple[torch.Tensor, torch.Tensor]:
        """(m, v) as fp32."""
        if self.m_scale is None:
            return self.m, self.v
        out = []
        for q, s in ((self.m, self.m_scale), (self.v, self.v_scale)):
            s = s.repeat_interleave(_BLOCK)[:q.numel()]
            out.append((q.float().reshape(-1) * s).reshape(q.shape))
        return out[0], out[1].square()


def alloc_adam_state(param, bits=32) -> AdamState:
    """The moments of a parameter before its first step: zeros."""
    if bits == 32:
        return AdamState(*(torch.zeros(param.shape, dtype=_F32, device=param.device)
                           for _ in range(2)))
    if bits != 8:
        raise ValueError(f"state bits: expected 8 or 32, got {bits!r}")
    q = [torch.zeros(param.shape, dtype=_U8, device=param.device).view(_E4M3) for _ in range(2)]
    s = [torch.zeros(-(-param.numel() // _BLOCK), dtype=_F32, device=param.device)
         for _ in range(2)]
    return AdamState(*q, *s)


# ----------------------------------------------------------- gradients' norm ----


@lru_cache(maxsize=64)
def _norm_workspace(count):
    out = ctypes.c_size_t(0)
    rc = lib.grpo_grad_norm_workspace_size(count, _byref(out))
    if rc != GRPO_OK:
        raise GrpoError(rc, "grpo_grad_norm_workspace_size")
    return int(out.value)


def grpo_grad_norm_workspace_size(count) -> int:
    return _norm_workspace(int(count))


def _grad_type(g, i, device):
    """The library's code for a gradient's type."""
    code = _DTYPES.get(g.dtype)
    if code is None:
        raise TypeError(f"grads[{i}]: expected bfloat16, float16 or float32, got {g.dtype}")
    if g.device != device:
        raise ValueError(f"grads[{i}]: expected device {device}, got {g.device}")
    if not g.is_contiguous():
        raise ValueError(f"grads[{i}]: must be contiguous")
    return code


def _quick(view, field, grads, device):
    """The gradients' addresses, with their types' codes put into the table, where all
    of them are what is expected; None otherwise: they are then looked at one by one.
    (A set of adapters has hundreds, at a few us each one by one.)"""
    try:
        types = list(map(_dtype, grads))
        same = types.count(types[0]) == len(types)
        codes = _DTYPES[types[0]] if same else [_DTYPES[t] for t in types]
        if set(map(_device_index, grads)) != {device.index} or not all(map(_packed, grads)):
            return None
        data = list(map(_data_ptr, grads))
    except (AttributeError, KeyError, TypeError, IndexError):  # None, or another type
        return None
    view[field] = codes
    return data


def grpo_grad_norm(grads: Sequence[torch.Tensor | None], *, max_norm=None, out=None,
                   workspace=None) -> GradNorm:
    """The 2-norm over all gradients (None ones add nothing), and what to scale them
    with so that it is at most max_norm: ``AdamW.step(grads, scale=...)`` takes it.
    out: fp32 [2]."""
    live = [g for g in grads if g is not None]
    if out is not None:
        dev = out.device
        if out.dtype is not _F32 or out.shape != (2,) or not out.is_contiguous():
            raise ValueError("out: expected contiguous float32 [2]")
    elif live:
        dev = live[0].device
        out = torch.empty(2, dtype=_F32, device=dev)
    else:
        raise ValueError("grads: none given, and no out")
    if max_norm is None:
        max_norm = 0.0
    elif not max_norm > 0:
        raise ValueError(f"max_norm: expected a positive number, got {max_norm!r}")
    n = len(live)
    table = (GrpoGrad * n)()
    if n:
        view = np.frombuffer(table, dtype=_GRAD)
        data = _quick(view, "dtype", live, dev)
        if data is None:
            view["dtype"] = [_grad_type(g, i, dev) for i, g in enumerate(live)]
            data = list(map(_data_ptr, live))
        view["data"] = data
        view["numel"] = list(map(_numel, live))
    if workspace is None:
        workspace = torch.empty(_norm_workspace(n), dtype=_U8, device=dev)
    elif workspace.device != dev:
        raise ValueError(f"workspace: expected device {dev}, got {workspace.device}")
    rc = call_on(dev, lib.grpo_grad_norm, table, n, max_norm, out.data_ptr(),
                 workspace.data_ptr(), workspace.numel() * workspace.element_size())
    if rc:
        raise GrpoError(rc, "grpo_grad_norm")
    return GradNorm(*out.unbind())


# --------------------------------------------------------------------- AdamW ----


def _per_tensor(value, n, name):
    """A number for all tensors, or one for each, as an array."""
    if isinstance(value, (int, float)):
        return np.full(n, value, np.float32)
    value = np.array([float(v) for v in value], np.float32)
    if len(value) != n:
        raise ValueError(f"{name}: expected {n} numbers, got {len(value)}")
    return value


def _device_scalar(t, name, dtype, device):
    if t.dtype is not dtype or t.numel() != 1:
        raise ValueError(f"{name}: expected one {dtype}, got {tuple(t.shape)} {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    return t.data_ptr()


def _cuda_device(t):
    if t.device.type != "cuda":
        raise ValueError(f"expected tensors on a CUDA device, got {t.device}")
    return t.device


class AdamW:
    """AdamW over many tensors, one launch per 256 of them.

    params: contiguous fp32 or bf16 tensors of one CUDA device. bf16 ones are rounded
    at random, so that steps far below their spacing are not lost. lr and
    weight_decay: a number, or one for each tensor. copies: per tensor None, or a bf16
    or fp16 tensor of its shape (fp32 parameters) that each step writes the rounded
    parameter to. states: the moments to go on from (``AdamState``); zeros when not
    given, of ``state_bits`` 8 or 32. steps_done: steps before the next one. seed: of
    the random rounding.

    ``step_tensor`` (int64, one value, on the device) takes the count's place, for
    steps that are captured in a graph: the program adds 1 to it before each.

    Parameters, moments and copies are written in place on the current stream, which
    autograd does not see. The ``.data`` of each may be exchanged between steps, for values
    of the same shape and type (a captured step keeps the addresses that it had). To go on
    later, keep ``states``, ``steps_done``, ``seed`` and the parameters, and make an AdamW
    of them.
    """

    def __init__(self, params: Sequence[torch.Tensor], *, lr, betas=(0.9, 0.999), eps=1e-8,
                 weight_decay=0.01, state_bits=32, states=None, copies=None, steps_done=0, seed=0,
                 step_tensor=None):
        self.params = tuple(params)
        n = len(self.params)
        if n == 0:
            raise ValueError("params: none given")
        self.device = _cuda_device(self.params[0])
        self.betas = (float(betas[0]), float(betas[1]))
        if not all(0.0 <= b < 1.0 for b in self.betas):
            raise ValueError(f"betas: expected numbers in [0, 1), got {betas!r}")
        self.eps = float(eps)
        if not self.eps >= 0.0:
            raise ValueError(f"eps: expected a number from 0 on, got {eps!r}")
        self.lr = _per_tensor(lr, n, "lr")
        self.weight_decay = _per_tensor(weight_decay, n, "weight_decay")
        if states is None:
            states = [alloc_adam_state(p, state_bits) for p in self.params]
        self.states = tuple(s if isinstance(s, AdamState) else AdamState(*s) for s in states)
        self.copies = (None,) * n if copies is None else tuple(copies)
        if len(self.states) != n or len(self.copies) != n:
            raise ValueError(f"states and copies: expected {n} of them, got {len(self.states)} "
                             f"and {len(self.copies)}")
        self.steps_done = int(steps_done)
        if self.steps_done < 0:
            raise ValueError(f"steps_done: expected a count, got {steps_done!r}")
        self.seed = int(seed) & 0xFFFFFFFFFFFFFFFF
        self.step_tensor = step_tensor
        if step_tensor is not None:
            _device_scalar(step_tensor, "step_tensor", torch.int64, self.device)
        self._table = (GrpoAdamwTensor * n)()
        self._view = np.frombuffer(self._table, dtype=GrpoAdamwTensor)
        self._describe()

    def _describe(self):
        self._described = False  # until all of it is: what is refused is looked at again
        for i in range(len(self.params)):
            self._fill(i)
        # All that the step writes, as the table has it.
        m, v, m_scale, v_scale = zip(*self.states)
        written = {"params": self.params, "states m": m, "states v": v,
                   "states m_scale": m_scale, "states v_scale": v_scale, "copies": self.copies}
        held = [(t, name, i) for name, part in written.items() for i, t in enumerate(part)
                if t is not None]
        # One value in two of them would be written twice at once.
        spans = sorted((t.data_ptr(), t.nbytes, f"{name}[{i}]") for t, name, i in held if t.numel())
        for (a, size, one), (b, _, other) in zip(spans, spans[1:]):
            if a + size > b:
                raise ValueError(f"{one} and {other} overlap")
        self._shapes = list(map(_shape, self.params))
        self._held = [t for t, _, _ in held]
        self._at = list(map(_data_ptr, self._held)), list(range(len(self._held)))
        self._rounded = [c for c in self.copies if c is not None]
        self._types = list(map(_dtype, self._rounded))
        self._model = [*self.params, *self._rounded]
        self._sizes = list(map(_nbytes, self._model))
        self._described = True

    def _moved(self):
        """Whether a tensor's storage was exchanged (`.data`), or fewer values of it taken,
        since it was described. At one address and of one size may be copies of either type;
        of the moments, which are the optimizer's, the address is enough."""
        return (not self._described or not _lie_at(self._held, *self._at)
                or list(map(_nbytes, self._model)) != self._sizes
                or list(map(_dtype, self._rounded)) != self._types)

    def _grad(self, i, g):
        """Checks one gradient; its address (0: none)."""
        if g is None:
            return 0
        self._table[i].grad_dtype = _grad_type(g, i, self.device)
        if g.shape != self._shapes[i]:
            raise ValueError(f"grads[{i}]: expected shape {tuple(self._shapes[i])}, "
                             f"got {tuple(g.shape)}")
        return g.data_ptr()

    def _fill(self, i):
        """Checks a tensor, its moments and its copy, and describes them."""
        p, s, c, e = self.params[i], self.states[i], self.copies[i], self._table[i]
        dev, n = self.device, p.numel()

        def check(t, name, dtypes, count):
            if t.dtype not in dtypes:
                raise TypeError(f"{name}[{i}]: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
            if t.device != dev:
                raise ValueError(f"{name}[{i}]: expected device {dev}, got {t.device}")
            if t.numel() != count:
                raise ValueError(f"{name}[{i}]: expected {count} values, got {t.numel()}")
            if not t.is_contiguous():
                raise ValueError(f"{name}[{i}]: must be contiguous")
            return t.data_ptr()

        e.param = check(p, "params", _PARAMS, n)
        eight = s.m_scale is not None
        if eight != (s.v_scale is not None):
            raise ValueError(f"states[{i}]: m_scale and v_scale: both or neither")
        kind = (_E4M3,) if eight else (_F32,)
        e.m, e.v = check(s.m, "states m", kind, n), check(s.v, "states v", kind, n)
        if eight:
            blocks = -(-n // _BLOCK)
            e.m_scale = check(s.m_scale, "states m_scale", (_F32,), blocks)
            e.v_scale = check(s.v_scale, "states v_scale", (_F32,), blocks)
        if c is not None:
            if p.dtype is not _F32:
                raise TypeError(f"copies[{i}]: only of float32 parameters, got {p.dtype}")
            e.copy = check(c, "copies", _COPIES, n)
            e.copy_dtype = _DTYPES[c.dtype]
        e.numel = n
        e.param_dtype, e.state_bits = _DTYPES[p.dtype], 8 if eight else 32

    def step(self, grads: Sequence[torch.Tensor | None] | None = None, *, scale=None, lr=None,
             lr_factor=None) -> None:
        """One step. grads: one for each parameter, bf16, fp16 or fp32 (None leaves the
        tensor as it is); by default their ``.grad``. scale: fp32 on the device,
        multiplies the gradients; where it is not finite the step changes nothing (and
        is counted all the same). lr: from this step on. lr_factor: fp32 on the device, multiplies it."""
        params, dev = self.params, self.device
        if grads is None:
            grads = [p.grad for p in params]
        if len(grads) != len(params):
            raise ValueError(f"grads: expected {len(params)} of them, got {len(grads)}")
        if lr is not None:
            self.lr = _per_tensor(lr, len(params), "lr")
        if self._moved():
            self._describe()
        view = self._view
        view["lr"], view["weight_decay"] = self.lr, self.weight_decay
        data = _quick(view, "grad_dtype", grads, dev)
        if data is None or list(map(_shape, grads)) != self._shapes:
            if list(map(_shape, params)) != self._shapes:  # or other values of it taken
                self._describe()
            data = [self._grad(i, g) for i, g in enumerate(grads)]
        view["grad"] = data
        q = GrpoAdamwParams(*self.betas, self.eps, self.steps_done + 1, self.seed)
        if scale is not None:
            q.scale = _device_scalar(scale, "scale", _F32, dev)
        if lr_factor is not None:
            q.lr_factor = _device_scalar(lr_factor, "lr_factor", _F32, dev)
        if self.step_tensor is not None:
            q.step_on_device = _device_scalar(self.step_tensor, "step_tensor", torch.int64, dev)
        rc = call_on(dev, lib.grpo_adamw_step, self._table, len(params), _byref(q))
        if rc:
            raise GrpoError(rc, "grpo_adamw_step")
        self.steps_done += 1
