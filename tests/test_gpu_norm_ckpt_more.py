"""GPU: the norms and checkpoints where tests/test_gpu_norm_ckpt.py does not go."""

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
