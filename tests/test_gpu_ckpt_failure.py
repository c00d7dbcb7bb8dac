"""GPU: what the norms and the weight gradient do when a copy never arrives.

``grpo_selftest_lose_copy`` has the next call leave one copy out. The wait for it
runs out after about a second; the kernel lets what is in flight land and
returns. Nothing faults, and the context stays usable.
"""

import time

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TIMEOUT = -7  # GRPO_ERR_DEVICE_TIMEOUT


@pytest.fixture(scope="module")
def clp():
    import __graft_entry__

    __graft_entry__.build()
    import chunked_log_prob_gb300 as m

    return m


def _wgrad_case(clp, n, out, d):
    g = torch.Generator().manual_seed(n)
    dy = torch.randn(n, out, generator=g).to(DEV, torch.bfloat16)
    c = clp.grpo_ckpt_pack(torch.randn(n, d, generator=g).to(DEV, torch.bfloat16))
    ws = torch.empty(clp.grpo_ckpt_wgrad_workspace_size(n, out, d), dtype=torch.uint8, device=DEV)
    return dy, c, ws


# One tile; one tile cut into pieces; more tiles than pairs, the last ones cut.
WGRAD = [(512, 256, 256), (4096, 256, 256), (4096, 4096, 4096)]


@pytest.mark.parametrize("n,out,d", WGRAD)
@pytest.mark.parametrize("stage", [2, 7])
def test_wgrad_ends_and_reports(clp, n, out, d, stage):
    dy, c, ws = _wgrad_case(clp, n, out, d)
    want = clp.grpo_ckpt_wgrad(dy, c, workspace=ws)
    assert clp.grpo_read_device_status(ws) == 0
    t0 = time.perf_counter()
    clp.grpo_selftest_lose_copy(stage)
    clp.grpo_ckpt_wgrad(dy, c, workspace=ws)
    # The status call waits for the stream. A second for the wait, and one more
    # for each copy in flight whose barrier waits for a role that gave up.
    assert clp.grpo_read_device_status(ws) == TIMEOUT
    assert 0.3 < time.perf_counter() - t0 < 20.0
    again = clp.grpo_ckpt_wgrad(dy, c, workspace=ws)
    assert clp.grpo_read_device_status(ws) == 0
    assert torch.equal(again, want)
