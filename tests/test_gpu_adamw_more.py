"""GPU: what an AdamW step and the gradients' norm hold to beyond their formulas."""

import numpy as np
import pytest
import torch

from oracle import block_oracle as o

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def clp():
    __import__("__graft_entry__").build()
    import chunked_log_prob_gb300 as m

    return m


def f64(t):
    return t.detach().cpu().double().numpy().reshape(-1)


@pytest.mark.parametrize("bits", [8, 32])
def test_copies_and_moments_that_were_moved_away_and_back(clp, bits):
    # As a program does that makes room between steps: what comes back lies elsewhere.
    g = torch.Generator().manual_seed(1)
    made = []
    for _ in range(2):
        p = torch.randn(3000, generator=g.manual_seed(2)).to(DEV)
        c = p.to(BF)
        made.append((p, c, clp.AdamW([p], lr=1e-2, state_bits=bits, copies=[c], seed=4)))
    (p, c, opt), (q, d, stays) = made
    grads = [torch.randn(3000, generator=g).to(DEV) for _ in range(3)]
    for gr in grads:
        stays.step([gr])
        opt.step([gr])
        held = [t for t in (c, *opt.states[0]) if t is not None]
        kept = [t.data for t in held]  # so that the addresses are not used again
        for t in held:
            t.data = t.data.cpu()
        with pytest.raises(ValueError, match="expected device"):
            opt.step([gr])
        for t in held:
            t.data = t.data.to(DEV)
        assert all(t.data_ptr() != k.data_ptr() for t, k in zip(held, kept))
        for k in kept:
            k.view(torch.uint8).fill_(0xEE)
        assert torch.equal(c, d) and torch.equal(c, p.to(BF))
    for a, b in zip((p, *opt.states[0].moments()), (q, *stays.states[0].moments())):
        assert torch.equal(a, b)
    for k in kept:
        assert (k.view(torch.uint8) == 0xEE).all()
