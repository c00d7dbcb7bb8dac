"""Host-side checks of the norm and checkpoint calls: sizes, layout and every
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


def _desc(clp, n=4, d=16, dtype=0, wdtype=0, kind=1, eps=1e-6, reserved=0, strides=(0,) * 7):
    return clp._binding.GrpoNormDesc(n, d, dtype, wdtype, kind, eps, reserved, *strides)


def _fwd(clp, desc, **kw):
    a = Buf().a
    p = dict(x=a, res=None, w=a, b=None, mask=None, y=a, z=None, mean=None, rstd=a, ckpt=None)
    p.update(kw)
    return clp.lib.grpo_norm_fwd(*p.values(), ctypes.byref(desc) if desc else None, None)


def _bwd(clp, desc, ws=1 << 30, **kw):
    a = Buf().a
    p = dict(dy=a, x=a, ckpt=None, w=a, mean=None, rstd=a, mask=None, dres=None, dx=a, dw=a,
             db=None, add_dw=None, add_db=None)
    p.update(kw)
    wsp = p.pop("wsp", a)
    return clp.lib.grpo_norm_bwd(*p.values(), ctypes.byref(desc) if desc else None, wsp, ws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), -1), (dict(d=0), -1), (dict(dtype=3), -1), (dict(dtype=-1), -1),
    (dict(wdtype=1), -1),               # fp16 weight beside bf16 rows
    (dict(kind=2), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(reserved=1), -1), (dict(strides=(15, 0, 0, 0, 0, 0, 0)), -1),
    (dict(strides=(0, 0, 0, 0, 0, 0, 8)), -1), (dict(n=(1 << 30) + 1), -3),
    (dict(d=(1 << 27) + 1), -3),
])
def test_bad_descriptions_are_refused(clp, kw, want):
    d = _desc(clp, **kw)
    assert _fwd(clp, d) == want
    assert _bwd(clp, d) == want
    out = ctypes.c_size_t()
    assert clp.lib.grpo_norm_workspace_size(ctypes.byref(d), ctypes.byref(out)) == want


def test_norm_forward_refuses_bad_pointers(clp):
    a = Buf().a
    d = _desc(clp)
    assert _fwd(clp, None) == -1
    assert _fwd(clp, d, x=None) == -1
    assert _fwd(clp, d, y=None) == -1
    assert _fwd(clp, d, z=a) == -1            # z without a residual
    assert _fwd(clp, d, mean=a) == -1         # RMS norm has no mean
    assert _fwd(clp, d, x=a + 1) == -2
    assert _fwd(clp, d, w=a + 1) == -2
    assert _fwd(clp, d, rstd=a + 2) == -2
    assert _fwd(clp, d, ckpt=a + 128) == -2


def test_norm_backward_refuses_bad_pointers(clp):
    a = Buf().a
    d = _desc(clp)
    assert _bwd(clp, None) == -1
    for name in ("dy", "dx", "rstd", "x"):
        assert _bwd(clp, d, **{name: None}) == -1
    assert _bwd(clp, d, ckpt=a) == -1         # x and its checkpoint
    assert _bwd(clp, d, mean=a) == -1
    assert _bwd(clp, _desc(clp, kind=0)) == -1  # layer norm without its mean
    assert _bwd(clp, d, dw=None, add_dw=a) == -1
    assert _bwd(clp, d, add_db=a) == -1
    assert _bwd(clp, d, wsp=None) == -1
    assert _bwd(clp, d, dy=a + 1) == -2
    assert _bwd(clp, d, dw=a + 2) == -2
    assert _bwd(clp, d, wsp=a + 16) == -2
    assert _bwd(clp, d, ws=64) == -4


def test_checkpoint_calls_refuse_bad_arguments(clp):
    a, lib = Buf().a, clp.lib
    assert lib.grpo_ckpt_pack(None, None, a, 4, 16, 0, 0, None) == -1
    assert lib.grpo_ckpt_pack(a, None, None, 4, 16, 0, 0, None) == -1
    assert lib.grpo_ckpt_pack(a, None, a, 4, 16, 3, 0, None) == -1
    assert lib.grpo_ckpt_pack(a, None, a, 4, 16, 0, 15, None) == -1
    assert lib.grpo_ckpt_pack(a, None, a, -1, 16, 0, 0, None) == -1
    assert lib.grpo_ckpt_pack(a + 1, None, a, 4, 16, 0, 0, None) == -2
    assert lib.grpo_ckpt_pack(a, None, a + 16, 4, 16, 0, 0, None) == -2
    assert lib.grpo_ckpt_pack(a, None, a, 4, (1 << 27) + 1, 0, 0, None) == -3
    assert lib.grpo_ckpt_unpack(a, None, 4, 16, 0, 0, None) == -1
    assert lib.grpo_ckpt_unpack(a, a + 2, 4, 16, 2, 0, None) == -2
    assert lib.grpo_ckpt_size(4, 0, ctypes.byref(ctypes.c_size_t())) == -1
    assert lib.grpo_ckpt_size(4, 16, None) == -1
    assert lib.grpo_ckpt_layout(4, 16, None, None, None) == -1


def test_wgrad_refuses_bad_arguments(clp):
    a, f = Buf().a, clp.lib.grpo_ckpt_wgrad
    big = 1 << 40
    ok = [a, a, None, a, 4, 16, 24, 0, a, big, None]

    def call(**kw):
        names = ["dy", "ckpt", "add", "dW", "n", "out", "inn", "stride", "ws", "bytes", "stream"]
        v = dict(zip(names, ok))
        v.update(kw)
        return f(*v.values())

    for name in ("dy", "ckpt", "dW", "ws"):
        assert call(**{name: None}) == -1
    assert call(n=-1) == -1 and call(out=0) == -1 and call(inn=0) == -1
    assert call(stride=8) == -1
    assert call(out=12) == -3 and call(inn=12) == -3 and call(stride=20) == -3
    assert call(inn=(1 << 20) + 8) == -3
    assert call(dy=a + 8) == -2 and call(dW=a + 8) == -2 and call(add=a + 4) == -2
    assert call(ckpt=a + 16) == -2 and call(ws=a + 64) == -2
    assert call(bytes=16) == -4
    assert clp.lib.grpo_ckpt_wgrad_workspace_size(4, 16, 12, ctypes.byref(ctypes.c_size_t())) == -3


@pytest.mark.parametrize("n,d", [(0, 5), (1, 1), (3, 32), (7, 33), (5, 2880), (2, 16385)])
def test_checkpoint_layout(clp, n, d):
    c = clp.alloc_ckpt(n, d)
    ldq, off, lde = c._layout()
    assert ldq == -(-d // 16) * 16 and lde == -(-(-(-d // 32)) // 16) * 16
    assert off % 256 == 0 and n * ldq <= off < n * ldq + 256
    assert c.data.numel() == clp.grpo_ckpt_size(n, d)
    assert off + n * lde <= c.data.numel() < off + n * lde + 256
    assert c.q.shape == (n, d) and c.exponents.shape == (n, -(-d // 32))
    assert c.data.numel() <= n * (1.04 * d + 32) + 512  # 1.03 bytes a value and padding


def test_checkpoint_views_point_into_the_buffer(clp):
    c = clp.alloc_ckpt(3, 40)
    c.data.copy_(torch.arange(c.data.numel(), dtype=torch.int64).to(torch.uint8))
    ldq, off, lde = c._layout()
    assert c.q.view(torch.uint8)[2, 5] == (2 * ldq + 5) % 256
    assert c.exponents[1, 1] == (off + lde + 1) % 256


def test_norm_workspace_is_bounded(clp):
    # At most 608 rows of partial sums, whatever the number of tokens.
    for d in (1, 256, 2880, 8192, 8200, 16384):
        big = clp.grpo_norm_workspace_size(1 << 30, d)
        assert big == clp.grpo_norm_workspace_size(1 << 20, d) <= 608 * d * 8 + 256
        assert clp.grpo_norm_workspace_size(1, d) <= 2 * d * 4 + 256


BAD = [
    (lambda c: c.grpo_norm_fwd(torch.zeros(4)), ValueError),
    (lambda c: c.grpo_norm_fwd(torch.zeros(4, 8, dtype=torch.float64)), TypeError),
    (lambda c: c.grpo_norm_fwd(torch.zeros(4, 8), kind="batch"), ValueError),
    (lambda c: c.grpo_norm_fwd(torch.zeros(4, 8), torch.zeros(7)), ValueError),
    (lambda c: c.grpo_norm_fwd(torch.zeros(4, 8), torch.zeros(8).half()), TypeError),
    (lambda c: c.grpo_norm_fwd(torch.zeros(4, 8).half(), torch.zeros(8).half(), torch.zeros(8)),
     TypeError),
    (lambda c: c.grpo_norm_fwd(torch.zeros(8, 4).t()), ValueError),
    (lambda c: c.grpo_norm_fwd(torch.zeros(1, 8).expand(4, 8)), ValueError),  # rows overlap
    (lambda c: c.grpo_norm_fwd(torch.zeros(4, 8), residual=torch.zeros(4, 9)), ValueError),
    (lambda c: c.grpo_norm_fwd(torch.zeros(4, 8), z=torch.zeros(4, 8)), ValueError),
    (lambda c: c.grpo_norm_fwd(torch.zeros(4, 8), mask=torch.zeros(4)), TypeError),
    (lambda c: c.grpo_norm_fwd(torch.zeros(4, 8), mean=torch.zeros(4)), ValueError),
    (lambda c: c.grpo_norm_fwd(torch.zeros(4, 8), ckpt=c.alloc_ckpt(4, 9)), ValueError),
    (lambda c: c.grpo_norm_fwd(torch.zeros(4, 8)), ValueError),  # not on a CUDA device
    (lambda c: c.grpo_norm_bwd(torch.zeros(4, 8), torch.zeros(4, 8).half(), None, None,
                               torch.zeros(4)), TypeError),
    (lambda c: c.grpo_norm_bwd(torch.zeros(4, 8), torch.zeros(4, 8), None, torch.zeros(4),
                               torch.zeros(4)), ValueError),
    (lambda c: c.grpo_norm_bwd(torch.zeros(4, 8), torch.zeros(4, 8), None, None, torch.zeros(4),
                               kind="layer"), ValueError),
    (lambda c: c.grpo_norm_bwd(torch.zeros(4, 8), c.alloc_ckpt(3, 8), None, None,
                               torch.zeros(4)), ValueError),
    (lambda c: c.grpo_norm_bwd(torch.zeros(4, 8), torch.zeros(4, 8), None, None, torch.zeros(4)),
     ValueError),
    (lambda c: c.grpo_ckpt_pack(torch.zeros(4, 8, 2)), ValueError),
    (lambda c: c.grpo_ckpt_pack(torch.zeros(4, 8)), ValueError),
    (lambda c: c.grpo_ckpt_unpack(c.alloc_ckpt(4, 8), torch.int8), TypeError),
    (lambda c: c.grpo_ckpt_unpack(c.alloc_ckpt(4, 8)), ValueError),
    (lambda c: c.grpo_ckpt_unpack(c.Checkpoint8(torch.zeros(8, dtype=torch.uint8), 4, 8)),
     ValueError),
    (lambda c: c.grpo_ckpt_wgrad(torch.zeros(4, 8), c.alloc_ckpt(4, 8)), TypeError),
    (lambda c: c.grpo_ckpt_wgrad(torch.zeros(4, 8).bfloat16(), torch.zeros(4, 8)), TypeError),
    (lambda c: c.grpo_ckpt_wgrad(torch.zeros(4, 8).bfloat16(), c.alloc_ckpt(5, 8)), ValueError),
    (lambda c: c.grpo_ckpt_wgrad(torch.zeros(4, 8).bfloat16(), c.alloc_ckpt(4, 8),
                                 dW=torch.zeros(8, 9)), ValueError),
    (lambda c: c.grpo_ckpt_wgrad(torch.zeros(4, 8).bfloat16(), c.alloc_ckpt(4, 8)), ValueError),
]


@pytest.mark.parametrize("case", range(len(BAD)))
def test_python_calls_refuse(clp, case):
    call, error = BAD[case]
    with pytest.raises(error):
        call(clp)
