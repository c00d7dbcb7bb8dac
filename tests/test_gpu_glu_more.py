"""GPU: what the gated feed-forward block's calls hold to beyond their formulas."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def clp():
    __import__("__graft_entry__").build()
    import chunked_log_prob_gb300 as m

    return m


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, t=BF, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device=DEV)).to(t)


@pytest.mark.parametrize("box", [0, 3, 6, 7])
def test_a_tile_is_nan_as_a_whole_where_what_is_added_does_not_come(clp, box):
    # More tiles than pairs: tiles are whole. Boxes before the lost one are on their way
    # out as its wait runs out.
    g = _gen(3)
    n, d, f = 1000, 2560, 2560
    x, dg, du = _randn(g, n, d), _randn(g, n, f), _randn(g, n, f)
    add = torch.randn(f, d, generator=g, device=DEV)
    ws = torch.empty(clp.grpo_glu_wgrad_workspace_size(n, f, d), dtype=torch.uint8, device=DEV)
    want = clp.grpo_glu_wgrad(dg, du, x, add_gate=add, add_up=add, workspace=ws)
    clp.grpo_selftest_lose_copy((1 << 29) + box)
    got = clp.grpo_glu_wgrad(dg, du, x, add_gate=add, add_up=add, workspace=ws)
    assert clp.grpo_read_device_status(ws) == -7
    assert torch.isnan(got[0][:32, :128]).all()  # the warp's part of its tile
    for p, q in zip(got, want):
        bad = torch.isnan(p)
        assert torch.equal(p[~bad], q[~bad])
        # Each warp's part of a tile, 32 x 128, is whole or NaN.
        parts = bad.reshape(f // 32, 32, d // 128, 128)
        assert torch.equal(parts.any(1).any(2), parts.all(1).all(2))
    for p, q in zip(clp.grpo_glu_wgrad(dg, du, x, add_gate=add, add_up=add, workspace=ws), want):
        assert torch.equal(p, q)
