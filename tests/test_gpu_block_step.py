"""GPU: the feed-forward block's whole training step (examples/block_step.py): its
gradients against the formulas in fp64, and what the optimizer makes of them."""

import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

import oracle
import synth
from oracle import block_oracle as bo
from oracle import norm_ckpt_oracle as no

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    __import__("__graft_entry__").build()
    spec = importlib.util.spec_from_file_location(
        "block_step", os.path.join(ROOT, "examples", "block_step.py"))
    m = importlib.util.module_from_spec(spec)
    sys.modules["block_step"] = m
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.detach().cpu().double().numpy()


def rel(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


def _setup(example, f, **kw):
    p = synth.make_problem("tiny", seed=0)
    n, d = p.n_tokens, p.hidden_size
    g = torch.Generator().manual_seed(1)
    w = example.random_weights(d, f, p.weight, g)
    w["norm1"] = 1 + 0.1 * torch.randn(d, generator=g)
    w["norm2"] = 1 + 0.1 * torch.randn(d, generator=g)
    block = example.Block({k: v.to(DEV) for k, v in w.items()}, **kw)
    x = torch.randn(n, d, generator=g).to(torch.bfloat16)
    mask = p.mask.clone()
    mask[n - 40:] = 0
    return p, block, x, mask


def test_gradients_of_the_whole_step(example):
    p, block, x, mask = _setup(example, 512)
    n = p.n_tokens
    w = {k: f64(v) for k, v in block.w.items()}
    m = mask.numpy()
    bf = torch.bfloat16

    def round16(z):
        return torch.from_numpy(z).to(bf)

    # The formulas, rounded where the step stores its tensors.
    y1, _, r1 = no.norm_fwd(f64(x), w["norm1"], None, "rms", 1e-6, mask=m)
    y1 = f64(round16(y1))
    a, _, _ = bo.glu_fwd(y1, w["gate"], w["up"], "silu", m)
    a = f64(round16(a))
    z = f64(round16(f64(x) + f64(round16(a @ w["down"].T)))) * (m != 0)[:, None]
    h, _, r2 = no.norm_fwd(z, w["norm2"], None, "rms", 1e-6, mask=m)
    hb = round16(h)
    base, _ = oracle.selective_logp(hb, block.w["head"].cpu(), p.ids.numpy())
    old, ref = p.old_ref(torch.from_numpy(base))
    want = oracle.loss_fwd_bwd(hb, block.w["head"].cpu(), p.ids.numpy(), m, old, ref, p.adv,
                               p.seq_len, p.eps_low, p.eps_high, p.beta)
    top = float(torch.finfo(bf).max)
    qz = no.ckpt_expand(*no.ckpt_pack(z, top, mask=m))
    qa = no.ckpt_expand(*no.ckpt_pack(a, top, mask=m))
    dz, dw2, _ = no.norm_bwd(want["dH"], qz, w["norm2"], None, r2, "rms", mask=m)
    g, u = y1 @ w["gate"].T, y1 @ w["up"].T
    dg, du, _ = bo.glu_bwd(dz @ w["down"], g, u, "silu", m)
    dy = dg @ w["gate"] + du @ w["up"]
    dx, dw1, _ = no.norm_bwd(dy, f64(x), w["norm1"], None, r1, "rms", mask=m)
    dx = (dx + dz) * (m != 0)[:, None]

    got = block.grads(x.to(DEV), p.ids.to(DEV), mask.to(DEV), old.to(DEV), ref.to(DEV),
                      p.adv.to(DEV), p.seq_len)
    assert abs(got.loss.item() - want["L"]) <= 1e-3 * abs(want["L"])  # the loss tests' bound
    # dH is within 2e-2 (the loss tests' bound); each tensor on the way that is stored in
    # bf16 adds its half step, 2^-8: dz; dz Wd; dgate and dup; dx.
    tol, half = 2e-2 + 2.0 ** -8, 2.0 ** -8
    gw = {k: f64(v) for k, v in got.weights.items()}
    assert rel(gw["norm2"], dw2) <= tol
    assert rel(gw["down"], dz.T @ qa) <= tol + half
    assert rel(gw["gate"], dg.T @ y1) <= tol + 3 * half
    assert rel(gw["up"], du.T @ y1) <= tol + 3 * half
    assert rel(gw["norm1"], dw1) <= tol + 4 * half
    assert rel(f64(got.dx), dx) <= tol + 4 * half
    assert (got.dx[n - 40:] == 0).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_the_step_that_follows(example, bits):
    p, block, x, mask = _setup(example, 256, lr=1e-3, state_bits=bits, max_norm=0.01)
    old = torch.full((p.n_tokens,), -8.0, device=DEV)
    args = (x.to(DEV), p.ids.to(DEV), mask.to(DEV), old, old, p.adv.to(DEV), p.seq_len)
    before = {k: f64(v) for k, v in block.master.items()}
    r = block.grads(*args)
    norm = block.update(r).item()
    grads = {k: f64(v) for k, v in r.weights.items()}
    want = np.sqrt(sum((g ** 2).sum() for g in grads.values()))
    assert abs(norm - want) <= 20 * 2.0 ** -24 * want and norm > 0.01
    scale = 0.01 / (want + 1e-6)
    for k, p0 in before.items():
        zero = np.zeros_like(p0)
        decay = 0.0 if k.startswith("norm") else 0.01
        new, _, _ = bo.adamw(p0, grads[k], zero, zero, 1, 1e-3, decay=decay, scale=scale)
        got = f64(block.master[k])
        # The first step is lr g / (|g| + eps): where the scaled gradient is about eps,
        # the scale's own 1e-6 shows; else a few units of the parameter and of the step.
        assert (np.abs(got - new) <= 4 * 2.0 ** -24 * np.abs(p0) + 1e-3 * 1e-5).all(), k
        assert torch.equal(block.w[k], block.master[k].to(torch.bfloat16))
    again = block.grads(*args)
    assert torch.isfinite(again.loss).all() and again.loss.item() != r.loss.item()
    block.update(again)
    assert block.opt.steps_done == 2


def test_a_step_captured_with_its_gradients(example):
    # Forward, backward, clipping and update in one graph; an eager twin beside it.
    import chunked_log_prob_gb300 as clp

    made = []
    for _ in range(2):
        p, block, x, mask = _setup(example, 256, lr=1e-3)
        made.append(block)
    old = torch.full((p.n_tokens,), -8.0, device=DEV)
    args = (x.to(DEV), p.ids.to(DEV), mask.to(DEV), old, old, p.adv.to(DEV), p.seq_len)
    eager, held = made
    count = torch.zeros(1, dtype=torch.int64, device=DEV)
    names = example.NAMES
    held.opt = clp.AdamW([held.master[k] for k in names], lr=1e-3, state_bits=8,
                         weight_decay=eager.opt.weight_decay, step_tensor=count,
                         copies=[held.w[k] for k in names])
    eager.grads(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        count.add_(1)
        loss = held.grads(*args)
        held.update(loss)
    for _ in range(3):
        graph.replay()
        r = eager.grads(*args)
        eager.update(r)
        torch.cuda.synchronize()
        assert abs(r.loss.item() - loss.loss.item()) <= 1e-3 * abs(r.loss.item()) + 1e-6
    assert count.item() == 3
    for k in names:
        # The bias corrections of the two differ by some units of fp32.
        assert (eager.master[k] - held.master[k]).abs().max() <= 3 * 1e-3


def test_example_runs(example, capsys):
    example.main()
    assert "step 2: loss" in capsys.readouterr().out
