"""What an AdamW step hands to the library, on host tensors with the call recorded: the
addresses that it reads and writes through are those of the tensors as they are now."""

import pytest
import torch

import __graft_entry__

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3 = torch.float8_e4m3fn


@pytest.fixture
def adamw(monkeypatch):
    """(AdamW on host tensors, the list of recorded steps' tables)."""
    __graft_entry__.build()
    import chunked_log_prob_gb300._adamw as m

    steps = []

    def record(device, fn, table, count, params):
        assert fn is m.lib.grpo_adamw_step and device.type == "cpu"
        steps.append([{name: getattr(e, name) for name, _ in e._fields_} for e in table])
        return 0

    monkeypatch.setattr(m, "call_on", record)
    monkeypatch.setattr(m, "_cuda_device", lambda t: t.device)
    return m.AdamW, steps


def _made(adamw, bits=8, ct=BF, n=3):
    params = [torch.randn(130 + i, 4) for i in range(n)]
    copies = [p.to(ct) if i != 1 else None for i, p in enumerate(params)]
    opt = adamw(params, lr=1e-3, state_bits=bits, copies=copies)
    return opt, params, copies, [torch.zeros_like(p) for p in params]


def _as_described(opt, entry, i):
    s, c = opt.states[i], opt.copies[i]
    assert entry["param"] == opt.params[i].data_ptr()
    assert entry["numel"] == opt.params[i].numel()
    assert entry["m"] == s.m.data_ptr() and entry["v"] == s.v.data_ptr()
    if s.m_scale is not None:
        assert entry["m_scale"] == s.m_scale.data_ptr()
        assert entry["v_scale"] == s.v_scale.data_ptr()
    assert entry["copy"] == (None if c is None else c.data_ptr())
    if c is not None:
        assert entry["copy_dtype"] == {BF: 0, HF: 1}[c.dtype]


@pytest.mark.parametrize("bits,part", [(32, "m"), (32, "v"), (8, "m"), (8, "v"), (8, "m_scale"),
                                       (8, "v_scale"), (8, "param"), (32, "copy")])
def test_exchanged_storage_is_followed(adamw, bits, part):
    opt, params, copies, grads = _made(adamw[0], bits)
    opt.step(grads)
    kept = []  # so that no new storage lies where an old one did
    for i in (0, 2):
        t = {"param": params[i], "copy": copies[i]}.get(part)
        t = getattr(opt.states[i], part) if t is None else t
        kept.append(t.data)
        t.data = t.data.clone()
    opt.step(grads)
    for i in range(3):
        _as_described(opt, adamw[1][-1][i], i)
    opt.step(grads)
    assert adamw[1][-1] == adamw[1][-2] and opt.steps_done == 3


def test_a_copy_of_another_type_in_the_same_place(adamw):
    opt, _, copies, grads = _made(adamw[0])
    opt.step(grads)
    copies[2].data = copies[2].data.view(HF)
    opt.step(grads)
    _as_described(opt, adamw[1][-1][2], 2)


def test_fewer_values_in_the_same_place_are_refused(adamw):
    opt, params, copies, grads = _made(adamw[0], 32)
    opt.step(grads)
    # A gradient of the shape that the parameter had.
    keep, params[1].data = params[1].data, params[1].data[:7]
    for _ in range(2):  # and again: what was refused is not taken for described
        with pytest.raises(ValueError, match=r"states m\[1\]"):
            opt.step(grads)
    params[1].data = keep
    opt.step(grads)
    keep, copies[0].data = copies[0].data, copies[0].data[:1]
    with pytest.raises(ValueError, match=r"copies\[0\]"):
        opt.step(grads)
    copies[0].data = keep
    opt.step(grads)
    assert opt.steps_done == 3 and len(adamw[1]) == 3


def test_what_was_read_before_a_refusal_is_read_again(adamw):
    # One tensor lies elsewhere, a later one is refused; then both are back as they were.
    opt, params, copies, grads = _made(adamw[0])
    opt.step(grads)
    there, copy = params[0].data, copies[2].data
    params[0].data, copies[2].data = there.clone(), copy.double()
    with pytest.raises(TypeError, match=r"copies\[2\]"):
        opt.step(grads)
    params[0].data, copies[2].data = there, copy
    opt.step(grads)
    for i in range(3):
        _as_described(opt, adamw[1][-1][i], i)


def test_a_copy_of_no_type_that_is_taken(adamw):
    opt, _, copies, grads = _made(adamw[0])
    opt.step(grads)
    copies[0].data = copies[0].data.double()
    with pytest.raises(TypeError, match=r"copies\[0\]"):
        opt.step(grads)
    assert len(adamw[1]) == 1


def test_tensors_that_share_values_are_refused(adamw):
    cls = adamw[0]
    p, q = torch.randn(40), torch.randn(40)
    s = [torch.zeros(40) for _ in range(4)]
    both = torch.zeros(60, dtype=BF)
    for kw, what in (
            (dict(states=[(s[0], s[1]), (s[0], s[2])]), r"states m\[0\] and states m\[1\]"),
            (dict(states=[(s[0], s[0]), (s[1], s[2])]), r"states m\[0\] and states v\[0\]"),
            (dict(states=[(p, s[1]), (s[2], s[3])]), r"params\[0\] and states m\[0\]"),
            (dict(copies=[both[:40], both[20:]]), r"copies\[0\] and copies\[1\]"),
            (dict(copies=[both[:40], both[:40]]), r"copies\[0\] and copies\[1\]")):
        with pytest.raises(ValueError, match=what + " overlap"):
            cls([p, q], lr=1e-3, **kw)
    scale = torch.zeros(2)
    e = [torch.zeros(40, dtype=torch.uint8).view(E4M3) for _ in range(4)]
    with pytest.raises(ValueError, match=r"states m_scale\[0\] and states m_scale\[1\] overlap"):
        cls([p, q], lr=1e-3, states=[(e[0], e[1], scale[:1], scale[1:]),
                                     (e[2], e[3], scale[:1], torch.zeros(1))])
    # Neighbours in one buffer are not.
    flat = torch.zeros(6, 40)
    cls([flat[0], flat[1]], lr=1e-3, states=[(flat[2], flat[3]), (flat[4], flat[5])])
