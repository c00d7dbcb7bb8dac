"""GPU: the feed-forward block's training step, captured, is the eager one bit for bit."""

import importlib.util
import os
import sys

import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    __import__("__graft_entry__").build()
    spec = importlib.util.spec_from_file_location(
        "block_step_more", os.path.join(ROOT, "examples", "block_step.py"))
    m = importlib.util.module_from_spec(spec)
    sys.modules["block_step_more"] = m
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_steps_are_the_eager_ones(example, bits):
    # Both count their steps on the device, so both work out the same corrections.
    import chunked_log_prob_gb300 as clp

    p = synth.make_problem("tiny", seed=0)
    n, d = p.n_tokens, p.hidden_size
    g = torch.Generator().manual_seed(1)
    w = example.random_weights(d, 256, p.weight, g)
    x = torch.randn(n, d, generator=g).to(DEV, torch.bfloat16)
    mask = p.mask.clone()
    mask[n - 40:] = 0
    old = torch.full((n,), -8.0, device=DEV)
    args = (x, p.ids.to(DEV), mask.to(DEV), old, old, p.adv.to(DEV), p.seq_len)
    names = example.NAMES
    blocks, counts = [], []
    for _ in range(2):
        b = example.Block({k: v.to(DEV) for k, v in w.items()}, lr=1e-3)
        counts.append(torch.zeros(1, dtype=torch.int64, device=DEV))
        b.opt = clp.AdamW([b.master[k] for k in names], lr=1e-3, state_bits=bits, seed=3,
                          weight_decay=b.opt.weight_decay, step_tensor=counts[-1],
                          copies=[b.w[k] for k in names])
        blocks.append(b)
    eager, held = blocks

    def step(i):
        counts[i].add_(1)
        r = blocks[i].grads(*args)
        return r, blocks[i].update(r)

    eager.grads(*args)  # the device's first calls are not captured
    clp.grpo_grad_norm([old])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept, norm = step(1)
    assert torch.equal(held.master["gate"], eager.master["gate"])  # captured, not run
    for _ in range(3):
        graph.replay()
        want, size = step(0)
        torch.cuda.synchronize()
        assert torch.equal(kept.loss, want.loss) and torch.equal(norm, size)
        assert torch.equal(kept.dx, want.dx)
        for k in names:
            assert torch.equal(kept.weights[k], want.weights[k]), k
            assert torch.equal(held.master[k], eager.master[k]), k
            assert torch.equal(held.w[k], eager.w[k]), k
    for a, b in zip(eager.opt.states, held.opt.states):
        for y, z in zip(a, b):
            assert y is None and z is None or torch.equal(y.view(torch.uint8), z.view(torch.uint8))
