"""GPU: the decoder tail's training step (examples/tail_step.py), which runs the
norm, the head loss, the norm's backward pass from an 8-bit checkpoint and the
weight gradient from another, against the fp64 oracles in a row."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
import synth
from oracle import norm_ckpt_oracle as o

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import __graft_entry__

    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location(
        "tail_step", os.path.join(ROOT, "examples", "tail_step.py"))
    m = importlib.util.module_from_spec(spec)
    import sys

    sys.modules["tail_step"] = m
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def rel(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


def _setup(f):
    p = synth.make_problem("tiny", seed=3)
    n, d = p.n_tokens, p.hidden_size
    g = torch.Generator().manual_seed(5)
    bf = torch.bfloat16
    proj = (torch.randn(d, f, generator=g) / f ** 0.5).to(bf)
    norm = (1 + 0.2 * torch.randn(d, generator=g)).to(bf)
    x, a = torch.randn(n, d, generator=g).to(bf), torch.randn(n, f, generator=g).to(bf)
    mask = torch.ones(n, dtype=torch.uint8)
    mask[n - 40:] = 0
    x[n - 40:], a[n - 40:] = 0, 0
    return p, proj, norm, x, a, mask


def test_tail_step_against_the_oracles(example):
    p, proj, norm, x, a, mask = _setup(512)
    n, d = p.n_tokens, p.hidden_size
    tail = example.Tail(proj.to(DEV), norm.to(DEV), p.weight.to(DEV))
    r = (a.to(DEV) @ proj.to(DEV).t()).cpu()  # the product as the library rounds it
    z = (x.float() + r.float()).to(torch.bfloat16)
    h, _, rstd = o.norm_fwd(f64(z), f64(norm), None, "rms", 1e-6, mask=mask.numpy())
    hb = torch.from_numpy(h).to(torch.bfloat16)
    base, _ = oracle.selective_logp(hb, p.weight, p.ids.numpy())
    old, ref = p.old_ref(torch.from_numpy(base))
    got = example.tail_step(tail, x.to(DEV), a.to(DEV), p.ids.to(DEV), mask.to(DEV), old.to(DEV),
                            ref.to(DEV), p.adv.to(DEV), p.seq_len)
    torch.cuda.synchronize()
    want = oracle.loss_fwd_bwd(hb, p.weight, p.ids.numpy(), mask.numpy(), old, ref, p.adv,
                               p.seq_len, p.eps_low, p.eps_high, p.beta)
    assert abs(got.loss.item() - want["L"]) <= 1e-3 * abs(want["L"])  # the loss tests' bound
    top = float(torch.finfo(torch.bfloat16).max)
    qz = o.ckpt_expand(*o.ckpt_pack(f64(z), top, mask=mask.numpy()))
    qa = o.ckpt_expand(*o.ckpt_pack(f64(a), top, mask=mask.numpy()))
    dx, dw, _ = o.norm_bwd(want["dH"], qz, f64(norm), None, rstd, "rms", mask=mask.numpy())
    # dH is within 2e-2 (the loss tests' bound); dx adds bf16's half step 2^-8,
    # the products of it no more than their inputs have.
    tol = 2e-2 + 2.0 ** -8
    assert rel(f64(got.dx), dx) <= tol
    assert rel(f64(got.dnorm), dw) <= tol
    assert rel(f64(got.dproj), dx.T @ qa) <= tol + 2.0 ** -8
    assert rel(f64(got.da), dx @ f64(proj)) <= tol + 2.0 ** -8
    assert (got.dx[n - 40:] == 0).all()
    # 1.03 bytes a value and a rstd a row, against 2.
    assert got.kept_bytes < 0.56 * 2 * n * (d + 512)


def test_tail_step_from_checkpoints_is_close_to_the_exact_gradient(example):
    # An e4m3 is off by at most 2^-4 of a value, at random: a weight gradient
    # summed over 216 tokens of independent values is off by less than 2^-4.
    p, proj, norm, x, a, mask = _setup(256)
    tail = example.Tail(proj.to(DEV), norm.to(DEV), p.weight.to(DEV))
    old = torch.full((p.n_tokens,), -8.0, device=DEV)
    got = example.tail_step(tail, x.to(DEV), a.to(DEV), p.ids.to(DEV), mask.to(DEV), old, old,
                            p.adv.to(DEV), p.seq_len)
    exact = f64(got.dx).T @ f64(a)
    assert rel(f64(got.dproj), exact) <= 2.0 ** -4


def test_tail_step_accumulates(example):
    p, proj, norm, x, a, mask = _setup(256)
    tail = example.Tail(proj.to(DEV), norm.to(DEV), p.weight.to(DEV))
    old = torch.full((p.n_tokens,), -8.0, device=DEV)
    args = (tail, x.to(DEV), a.to(DEV), p.ids.to(DEV), mask.to(DEV), old, old, p.adv.to(DEV),
            p.seq_len)
    one = example.tail_step(*args)
    dproj, dnorm = one.dproj.clone(), one.dnorm.clone()
    two = example.tail_step(*args, dproj=dproj, dnorm=dnorm)
    assert two.dproj.data_ptr() == dproj.data_ptr()
    # Two equal sums: exactly twice each, but for the order of dproj's rounding.
    assert torch.equal(dnorm, 2 * one.dnorm)
    assert rel(f64(dproj), 2 * f64(one.dproj)) <= 2.0 ** -22


def test_example_runs(example, capsys):
    example.main()
    assert "loss" in capsys.readouterr().out
