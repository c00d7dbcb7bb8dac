"""Host-side checks of the gated feed-forward and optimizer calls: sizes and every
refusal, before anything is launched. No compute call runs (CPU)."""

import ctypes

import pytest
import torch

import __graft_entry__


@pytest.fixture(scope="module")
def clp():
    __graft_entry__.build()
    import chunked_log_prob_gb300 as m

    return m


class Buf:
    """Host memory standing in for device pointers that must not be touched."""

    def __init__(self):
        self.raw = ctypes.create_string_buffer(1 << 14)
        self.a = (ctypes.addressof(self.raw) + 255) // 256 * 256


def _desc(clp, n=4, d=16, f=24, dtype=0, act=0, **strides):
    e = clp._binding.GrpoGluDesc(n, d, f, dtype, act)
    for k, v in strides.items():
        setattr(e, k + "_stride", v)
    return e


def _ref(desc):
    return ctypes.byref(desc) if desc is not None else None


def _fwd(clp, desc, **kw):
    a = Buf().a
    p = dict(x=a, wg=a, wu=a, mask=None, h=a, gate=None, up=None, ckpt=None)
    p.update(kw)
    return clp.lib.grpo_glu_fwd(*p.values(), _ref(desc), None)


def _bwd(clp, desc, **kw):
    a = Buf().a
    p = dict(dh=a, x=a, wg=a, wu=a, gate=None, up=None, mask=None, dgate=a, dup=a, dx=a, h=None)
    ws, size = kw.pop("ws", None), kw.pop("size", 0)
    p.update(kw)
    return clp.lib.grpo_glu_bwd(*p.values(), _ref(desc), ws, size, None)


def _wgrad(clp, desc, ws=1 << 30, **kw):
    a = Buf().a
    p = dict(dgate=a, dup=a, x=a, ag=None, au=None, dwg=a, dwu=a)
    p.update(kw)
    wsp = p.pop("wsp", a)
    return clp.lib.grpo_glu_wgrad(*p.values(), _ref(desc), wsp, ws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), -1), (dict(d=0), -1), (dict(f=0), -1), (dict(f=-8), -1),
    (dict(dtype=2), -1), (dict(dtype=-1), -1), (dict(act=4), -1), (dict(act=-1), -1),
    (dict(d=20), -3), (dict(f=12), -3), (dict(n=(1 << 30) + 1), -3),
    (dict(d=(1 << 20) + 8), -3), (dict(f=(1 << 20) + 8), -3),
    (dict(n=1 << 30, f=1 << 20), -3),  # more tiles than 32 bits count
    (dict(x=8), -1), (dict(h=16), -1), (dict(dgate=16), -1), (dict(w_up=8), -1),
    (dict(x=20), -3), (dict(up=28), -3), (dict(dx=-8), -1),
])
def test_bad_descriptions_are_refused(clp, kw, want):
    d = _desc(clp, **kw)
    assert _fwd(clp, d) == want
    assert _bwd(clp, d) == want
    assert _wgrad(clp, d) == want


def test_glu_calls_refuse_bad_pointers(clp):
    a = Buf().a
    d = _desc(clp)
    assert _fwd(clp, None) == _bwd(clp, None) == _wgrad(clp, None) == -1
    for name in ("x", "wg", "wu", "h"):
        assert _fwd(clp, d, **{name: None}) == -1
        assert _fwd(clp, d, **{name: a + 8}) == -2
    assert _fwd(clp, d, gate=a) == -1  # both projections or neither
    assert _fwd(clp, d, up=a) == -1
    assert _fwd(clp, d, gate=a + 2, up=a) == -2
    assert _fwd(clp, d, ckpt=a + 16) == -2
    for name in ("dh", "x", "wg", "wu", "dgate", "dup"):
        assert _bwd(clp, d, **{name: None}) == -1
        assert _bwd(clp, d, **{name: a + 4}) == -2
    assert _bwd(clp, d, gate=a) == -1
    assert _bwd(clp, d, dx=a + 2) == -2
    assert _bwd(clp, d, h=a + 2) == -2
    assert _bwd(clp, d, ws=a + 16, size=1 << 30) == -2
    long = _desc(clp, f=4096)  # one tile of 128 stages: cut
    assert _bwd(clp, long, ws=a, size=256) == -4
    for name in ("dgate", "dup", "x", "dwg", "dwu"):
        assert _wgrad(clp, d, **{name: None}) == -1
        assert _wgrad(clp, d, **{name: a + 4}) == -2
    assert _wgrad(clp, d, ag=a + 4) == -2
    assert _wgrad(clp, d, wsp=None) == -1
    assert _wgrad(clp, d, wsp=a + 16) == -2
    assert _wgrad(clp, d, ws=64) == -4


def test_glu_workspace(clp):
    lib, out = clp.lib, ctypes.c_size_t()
    assert lib.grpo_glu_wgrad_workspace_size(4, 24, 16, None) == -1
    assert lib.grpo_glu_wgrad_workspace_size(-1, 24, 16, ctypes.byref(out)) == -1
    assert lib.grpo_glu_wgrad_workspace_size(4, 20, 16, ctypes.byref(out)) == -3
    assert lib.grpo_glu_bwd_workspace_size(4, 24, 16, None) == -1
    assert lib.grpo_glu_bwd_workspace_size(4, 24, -8, ctypes.byref(out)) == -1
    assert clp.grpo_glu_bwd_workspace_size(4, 24, 16) == 0
    assert clp.grpo_glu_bwd_workspace_size(0, 4096, 16) == 0
    assert clp.grpo_glu_bwd_workspace_size(4, 4096, 16) == 152 * 65536 * 4
    assert clp.grpo_glu_wgrad_workspace_size(4, 24, 16) == 256
    # Long sums over few tiles are cut into pieces: two tiles a pair at most.
    assert clp.grpo_glu_wgrad_workspace_size(1 << 20, 256, 256) == 256 + 152 * 65536 * 4


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_python_glu_refuses(clp):
    x, w, dh = _t(4, 16), _t(24, 16), _t(4, 24)
    with pytest.raises(TypeError, match="x: expected bfloat16 or float16"):
        clp.grpo_glu_fwd(x.float(), w, w)
    with pytest.raises(ValueError, match="x: expected 2 dimensions"):
        clp.grpo_glu_fwd(x[0], w, w)
    with pytest.raises(ValueError, match="act"):
        clp.grpo_glu_fwd(x, w, w, act="tanh")
    with pytest.raises(ValueError, match="w_gate: expected 16 columns"):
        clp.grpo_glu_fwd(x, _t(24, 8), w)
    with pytest.raises(ValueError, match="w_up"):
        clp.grpo_glu_fwd(x, w, _t(32, 16))
    with pytest.raises(TypeError, match="w_up"):
        clp.grpo_glu_fwd(x, w, w.half())
    with pytest.raises(ValueError, match="last dimension"):
        clp.grpo_glu_fwd(x, _t(16, 24).t(), w)
    with pytest.raises(ValueError, match="both or neither"):
        clp.grpo_glu_fwd(x, w, w, gate=dh)
    with pytest.raises(ValueError, match="h: expected shape"):
        clp.grpo_glu_fwd(x, w, w, h=_t(4, 16))
    with pytest.raises(TypeError, match="mask"):
        clp.grpo_glu_fwd(x, w, w, mask=torch.ones(4))
    with pytest.raises(ValueError, match="rows overlap"):
        clp.grpo_glu_fwd(_t(64).as_strided((4, 16), (8, 1)), w, w)
    with pytest.raises(ValueError, match="CUDA device"):
        clp.grpo_glu_fwd(x, w, w)
    with pytest.raises(ValueError, match="x: needed"):
        clp.grpo_glu_bwd(dh, None, w, w)
    with pytest.raises(ValueError, match="both or neither"):
        clp.grpo_glu_bwd(dh, x, w, w, gate=dh)
    with pytest.raises(ValueError, match="w_gate"):
        clp.grpo_glu_bwd(dh, x, _t(16, 16), w)
    with pytest.raises(ValueError, match="workspace"):
        clp.grpo_glu_bwd(dh, x, w, w, workspace=torch.empty(8, device="meta"))
    with pytest.raises(ValueError, match="dup: expected shape"):
        clp.grpo_glu_bwd(dh, x, w, w, dup=x)
    with pytest.raises(ValueError, match="x: expected shape"):
        clp.grpo_glu_wgrad(dh, dh, _t(5, 16))
    with pytest.raises(TypeError, match="dw_gate: expected torch.float32"):
        clp.grpo_glu_wgrad(dh, dh, x, dw_gate=w)


# ----------------------------------------------------------------- optimizer ----


def _tensor(clp, **kw):
    a = Buf().a
    e = clp._binding.GrpoAdamwTensor(a, a, a, a, None, None, None, 10, 1e-3, 0.0, 2, 2, 0, 32)
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def _params(clp, **kw):
    q = clp._binding.GrpoAdamwParams(0.9, 0.999, 1e-8, 1, 0)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


def _step(clp, t, q):
    return clp.lib.grpo_adamw_step(ctypes.byref(t) if t is not None else None, 1, _ref(q), None)


def test_adamw_refuses(clp):
    a, lib = Buf().a, clp.lib
    t, q = _tensor(clp), _params(clp)
    assert _step(clp, None, q) == -1
    assert _step(clp, t, None) == -1
    assert lib.grpo_adamw_step(ctypes.byref(t), -1, ctypes.byref(q), None) == -1
    for kw in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")),
               dict(eps=-1.0), dict(step=0)):
        assert _step(clp, t, _params(clp, **kw)) == -1
    assert _step(clp, t, _params(clp, scale=a + 2)) == -2
    assert _step(clp, t, _params(clp, step=0, step_on_device=a + 4)) == -2
    for kw in (dict(numel=-1), dict(param_dtype=1), dict(param_dtype=3), dict(grad_dtype=3),
               dict(state_bits=16), dict(lr=float("nan")), dict(weight_decay=float("inf")),
               dict(param=None), dict(m=None), dict(v=None), dict(state_bits=8),
               dict(copy=a, copy_dtype=2), dict(copy=a, param_dtype=0)):
        assert _step(clp, _tensor(clp, **kw), q) == -1, kw
    for kw in (dict(param=a + 2), dict(grad=a + 1), dict(m=a + 1), dict(v=a + 2),
               dict(copy=a + 1), dict(state_bits=8, m_scale=a + 2, v_scale=a)):
        assert _step(clp, _tensor(clp, **kw), q) == -2, kw
    assert _step(clp, _tensor(clp, numel=(1 << 44) + 1), q) == -3


def test_grad_norm_refuses(clp):
    a, lib = Buf().a, clp.lib
    G = clp._binding.GrpoGrad

    def norm(g, count=1, max_norm=1.0, out=a, ws=a, size=1 << 20):
        return lib.grpo_grad_norm(ctypes.byref(g) if g is not None else None, count, max_norm, out,
                                  ws, size, None)

    assert norm(None) == -1
    assert norm(G(a, 4, 2, 0), count=-1) == -1
    assert norm(G(a, -1, 2, 0)) == -1
    assert norm(G(a, 4, 3, 0)) == -1
    assert norm(G(a, 4, 2, 1)) == -1
    assert norm(G(a, 4, 2, 0), out=None) == -1
    assert norm(G(a, 4, 2, 0), ws=None) == -1
    assert norm(G(a, 4, 2, 0), max_norm=float("nan")) == -1
    assert norm(G(a + 2, 4, 2, 0)) == -2
    assert norm(G(a, 4, 2, 0), ws=a + 8) == -2
    assert norm(G(a, 4, 2, 0), size=128) == -4
    assert norm(G(a, (1 << 44) + 1, 2, 0)) == -3
    assert lib.grpo_grad_norm_workspace_size(-1, ctypes.byref(ctypes.c_size_t())) == -1
    assert lib.grpo_grad_norm_workspace_size(1, None) == -1


def test_python_optimizer_refuses(clp):
    p = _t(10, dtype=torch.float32)
    for bad, what in ((dict(params=[]), "none given"), (dict(params=[p]), "CUDA device")):
        with pytest.raises(ValueError, match=what):
            clp.AdamW(lr=1e-3, **bad)
    with pytest.raises(ValueError, match="state bits"):
        clp.alloc_adam_state(p, 16)
    with pytest.raises(ValueError, match="none given"):
        clp.grpo_grad_norm([None])
    with pytest.raises(ValueError, match="max_norm"):
        clp.grpo_grad_norm([p], max_norm=0.0)
    with pytest.raises(TypeError, match=r"grads\[0\]"):
        clp.grpo_grad_norm([p.double()])
    with pytest.raises(ValueError, match="contiguous"):
        clp.grpo_grad_norm([_t(4, 4).t()[1:]])


def test_states_before_the_first_step(clp):
    s = clp.alloc_adam_state(_t(3, 100), 8)
    assert s.m.dtype is s.v.dtype is torch.float8_e4m3fn and s.m.shape == (3, 100)
    assert s.m_scale.shape == s.v_scale.shape == (3,)
    for y in s.moments():
        assert y.dtype is torch.float32 and y.shape == (3, 100) and not y.any()
    s = clp.alloc_adam_state(_t(5))
    assert s.m_scale is None and s.moments()[0] is s.m
