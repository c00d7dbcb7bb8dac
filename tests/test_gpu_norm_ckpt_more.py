"""GPU: the norms and checkpoints where tests/test_gpu_norm_ckpt.py does not go."""

import importlib.util
import os
import sys
import threading

import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def clp():
    import __graft_entry__

    __graft_entry__.build()
    import chunked_log_prob_gb300 as m

    return m


def _example():
    spec = importlib.util.spec_from_file_location(
        "tail_step", os.path.join(ROOT, "examples", "tail_step.py"))
    m = importlib.util.module_from_spec(spec)
    sys.modules["tail_step"] = m
    spec.loader.exec_module(m)
    return m


def test_example_counts_what_it_says(clp, capsys):
    m, p = _example(), synth.make_problem("tiny", seed=0)
    n, d, f = p.n_tokens, p.hidden_size, 512
    g = torch.Generator().manual_seed(0)
    bf = torch.bfloat16
    tail = m.Tail(torch.randn(d, f, generator=g).to(DEV, bf), torch.ones(d, dtype=bf, device=DEV),
                  p.weight.to(DEV))
    x, a = torch.randn(n, d, generator=g).to(DEV, bf), torch.randn(n, f, generator=g).to(DEV, bf)
    old = torch.full((n,), -8.0, device=DEV)
    r = m.tail_step(tail, x, a, p.ids.to(DEV), p.mask.to(DEV), old, old, p.adv.to(DEV), p.seq_len)
    assert r.kept_bytes == clp.grpo_ckpt_size(n, d) + clp.grpo_ckpt_size(n, f) + 4 * n
    m.main()
    assert "z and a kept in" in capsys.readouterr().out


def _rows(g, n, d, t):
    return torch.randn(n, d, generator=g).to(DEV, t)


# Rows that leave registers: beyond 16384 columns; unaligned ones beyond 8192
# (forward); fp32 with residual, weight and bias that shared memory has no room for.
LONG = [(16392, torch.bfloat16), (20001, torch.bfloat16), (9001, torch.float16),
        (16384, torch.float32), (17000, torch.float32)]


@pytest.mark.parametrize("d,t", LONG)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_long_rows_in_place(clp, d, t, kind):
    g = torch.Generator().manual_seed(d)
    n = 37
    x, r, dy = (_rows(g, n, d, t) for _ in range(3))
    w, b = (1 + 0.1 * torch.randn(d, generator=g).to(DEV, t) for _ in range(2))
    mask = (torch.rand(n, generator=g) < 0.7).to(torch.uint8).to(DEV)
    kw = dict(kind=kind, mask=mask)
    want = clp.grpo_norm_fwd(x, w, b, residual=r, want_ckpt=True, **kw)
    xi, ri = x.clone(), r.clone()
    got = clp.grpo_norm_fwd(xi, w, b, residual=ri, y=xi, z=ri, want_ckpt=True, **kw)
    assert got.y.data_ptr() == xi.data_ptr() and got.z.data_ptr() == ri.data_ptr()
    assert torch.equal(got.y, want.y) and torch.equal(got.z, want.z)
    assert torch.equal(got.rstd, want.rstd)
    assert torch.equal(got.ckpt.q.view(torch.uint8), want.ckpt.q.view(torch.uint8))
    for src in ("x", "ckpt"):
        z = want.z if src == "x" else want.ckpt
        args = (w, want.mean, want.rstd)
        ref = clp.grpo_norm_bwd(dy, z, *args, dres=r, want_dbias=True, **kw)
        for place in ("dy", "dres") + (("x",) if src == "x" else ()):
            own = {"dy": dy.clone(), "dres": r.clone(), "x": want.z.clone()}
            zi = own["x"] if src == "x" else z
            out = clp.grpo_norm_bwd(own["dy"], zi, *args, dres=own["dres"], want_dbias=True,
                                    dx=own[place], **kw)
            assert all(torch.equal(a, c) for a, c in zip(out, ref)), place


@pytest.mark.parametrize("d", [64, 512, 2880, 4096, 12288])
@pytest.mark.parametrize("wt", [torch.bfloat16, torch.float32])
def test_weights_off_16_bytes(clp, d, wt):
    # Rows are aligned, weight and bias start one element into their buffers.
    g = torch.Generator().manual_seed(d)
    n = 50
    x, dy = (_rows(g, n, d, torch.bfloat16) for _ in range(2))
    w, b = (torch.randn(d, generator=g).to(DEV, wt) for _ in range(2))
    wo, bo = (torch.cat([v[:1], v])[1:] for v in (w, b))
    assert wo.data_ptr() % 16 == wt.itemsize
    want = clp.grpo_norm_fwd(x, w, b, kind="layer")
    got = clp.grpo_norm_fwd(x, wo, bo, kind="layer")
    assert torch.equal(got.y, want.y)
    ref = clp.grpo_norm_bwd(dy, x, w, want.mean, want.rstd, kind="layer", want_dbias=True)
    out = clp.grpo_norm_bwd(dy, x, wo, want.mean, want.rstd, kind="layer", want_dbias=True)
    assert all(torch.equal(a, c) for a, c in zip(out, ref))


def test_two_host_threads(clp):
    # Shapes that share a kernel but not its launch, each thread on its own stream.
    g = torch.Generator().manual_seed(0)
    sets = []
    for d in (256, 512, 1024, 4096):
        x, r, dy = (_rows(g, 300, d, torch.bfloat16) for _ in range(3))
        w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
        sets.append((x, r, dy, w))

    def step(x, r, dy, w):
        f = clp.grpo_norm_fwd(x, w, residual=r, want_ckpt=True)
        b = clp.grpo_norm_bwd(dy, f.ckpt, w, None, f.rstd, dres=r)
        return [f.y, f.z, b.dx, b.dweight, clp.grpo_ckpt_wgrad(b.dx, f.ckpt)]

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    errors = []

    def work(first):
        try:
            stream = torch.cuda.Stream(DEV)
            with torch.cuda.stream(stream):
                for i in range(60):
                    k = (first + i) % len(sets)
                    got = step(*sets[k])
                    stream.synchronize()
                    assert all(torch.equal(a, c) for a, c in zip(got, want[k]))
        except BaseException as e:  # noqa: BLE001 (handed to the test's thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
