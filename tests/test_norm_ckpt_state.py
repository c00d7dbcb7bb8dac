"""Host-side checks of the norm and checkpoint calls' bookkeeping (CPU)."""

import contextlib

import pytest
import torch

import __graft_entry__


@pytest.fixture(scope="module")
def clp():
    __graft_entry__.build()
    import chunked_log_prob_gb300 as m

    return m


def test_lose_copy_refuses_what_is_no_index(clp):
    for bad in (-2, 1 << 30, 1 << 40):
        with pytest.raises(clp.GrpoError) as e:
            clp.grpo_selftest_lose_copy(bad)
        assert e.value.code == -1
    clp.grpo_selftest_lose_copy(5)
    clp.grpo_selftest_lose_copy(-1)  # takes it back


class FakeCuda:
    """One thread's current device, and streams numbered 1000 + device."""

    def __init__(self, clp, monkeypatch, current):
        self.current, self.calls = current, []
        monkeypatch.setattr(clp._binding, "_current_device", lambda: self.current)
        monkeypatch.setattr(clp._binding, "_raw_stream", lambda index: 1000 + index)
        monkeypatch.setattr(torch.cuda, "device", self.guard)

    @contextlib.contextmanager
    def guard(self, device):
        before, self.current = self.current, torch.device(device).index
        try:
            yield
        finally:
            self.current = before

    def fn(self, *args):
        self.calls.append((self.current, args))
        return -5


@pytest.mark.parametrize("current", [0, 1, 3])
def test_calls_run_on_the_tensors_device(clp, monkeypatch, current):
    fake = FakeCuda(clp, monkeypatch, current)
    assert clp._binding.call_on(torch.device("cuda", 1), fake.fn, 7, None) == -5
    assert fake.calls == [(1, (7, None, 1001))]
    assert fake.current == current  # the caller's device is back


def test_calls_leave_the_device_as_it_was_after_an_error(clp, monkeypatch):
    fake = FakeCuda(clp, monkeypatch, 0)

    def broken(*args):
        raise RuntimeError

    with pytest.raises(RuntimeError):
        clp._binding.call_on(torch.device("cuda", 2), broken)
    assert fake.current == 0


def test_calls_refuse_the_cpu(clp):
    with pytest.raises(ValueError):
        clp._binding.call_on(torch.device("cpu"), None)


def _every_call(clp):
    bf = torch.bfloat16
    h, w = torch.zeros(8, 256, dtype=bf), torch.zeros(512, 256, dtype=bf)
    ids, row = torch.zeros(8, dtype=torch.int32), torch.zeros(8)
    ws = torch.zeros(1 << 12, dtype=torch.uint8)
    c = clp.alloc_ckpt(8, 256)
    return {
        "grpo_logp_fwd": lambda: clp.grpo_logp_fwd(h, w, ids),
        "grpo_loss_fwd_bwd": lambda: clp.grpo_loss_fwd_bwd(h, w, ids, None, row, row, row, 1),
        "grpo_logp_fwd_noalloc": lambda: clp.grpo_logp_fwd_noalloc(h, w, ids, row),
        "grpo_read_device_status": lambda: clp.grpo_read_device_status(ws),
        "grpo_norm_fwd": lambda: clp.grpo_norm_fwd(h),
        "grpo_norm_bwd": lambda: clp.grpo_norm_bwd(h, h, None, None, row),
        "grpo_ckpt_pack": lambda: clp.grpo_ckpt_pack(h),
        "grpo_ckpt_unpack": lambda: clp.grpo_ckpt_unpack(c),
        "grpo_ckpt_wgrad": lambda: clp.grpo_ckpt_wgrad(h, c),
    }


def test_every_launching_call_goes_to_the_tensors_device(clp, monkeypatch):
    # The library launches where it finds itself: no call may reach it otherwise.
    seen = []

    def record(device, fn, *args):
        seen.append((device.type, fn.__name__))
        return 0

    monkeypatch.setattr(clp._binding, "call_on", record)
    monkeypatch.setattr(clp._norm_ckpt, "call_on", record)
    for name, call in _every_call(clp).items():
        call()
        assert seen.pop() == ("cpu", name)
        assert not seen
