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


def _tiles(t):
    o, i = t.shape
    return t.reshape(o // 256, 256, i // 256, 256).transpose(1, 2).reshape(-1, 256 * 256)


# Tiles that the pair of the lost copy had not yet written. 4096 x 4096 outputs:
# pair 0 of 76 has three of the 228 whole tiles of 64 stages each, then 24 stages
# of the first of the 28 cut ones.
@pytest.mark.parametrize("n,out,d,stage,lost,add", [
    (512, 256, 256, 2, 1, "none"), (4096, 256, 256, 7, 1, "same"), (4096, 4096, 4096, 2, 4, "none"),
    (4096, 4096, 4096, 2, 4, "same"), (4096, 4096, 4096, 70, 3, "other"),
    (4096, 4096, 4096, 200, 1, "same")])
def test_wgrad_leaves_nan_and_nothing_stale(clp, n, out, d, stage, lost, add):
    dy, c, ws = _wgrad_case(clp, n, out, d)
    grad = None if add == "none" else torch.ones(out, d, device=DEV)
    want = _tiles(clp.grpo_ckpt_wgrad(dy, c, add=grad, workspace=ws))
    dW = grad if add == "same" else torch.full((out, d), 7.0, device=DEV)
    ws.zero_()  # the pieces of cut tiles would be plausible ones
    clp.grpo_selftest_lose_copy(stage)
    got = _tiles(clp.grpo_ckpt_wgrad(dy, c, add=grad, dW=dW, workspace=ws))
    assert clp.grpo_read_device_status(ws) == TIMEOUT
    nan = torch.isnan(got)
    assert torch.equal(nan.any(1), nan.all(1))  # a tile is whole or NaN
    assert int(nan.all(1).sum()) == lost
    keep = ~nan.any(1)
    assert torch.equal(got[keep], want[keep])


def _rows_or_nan(got, want, lost):
    """Every row is `want`'s or NaN throughout, row `lost` NaN; which are NaN."""
    got, want = got.float().reshape(len(got), -1), want.float().reshape(len(want), -1)
    nan = torch.isnan(got)
    assert torch.equal(nan.any(1), nan.all(1))
    keep = ~nan.all(1)
    assert torch.equal(got[keep], want[keep])
    assert not keep[lost]
    return nan.all(1)


# Several rows a CTA, one row a CTA, and rows that do not start on 16 bytes.
@pytest.mark.parametrize("d", [512, 1001, 4096, 8200, 16384])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_forward_leaves_nan(clp, d, kind):
    n, lost = 2000, 5
    g = torch.Generator().manual_seed(d)
    x, r = (torch.randn(n, d, generator=g).to(DEV, torch.bfloat16) for _ in range(2))
    w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    want = clp.grpo_norm_fwd(x, w, residual=r, kind=kind, want_ckpt=True)
    z = torch.full_like(x, 7.0)
    ckpt = clp.Checkpoint8(torch.zeros_like(want.ckpt.data), n, d)
    clp.grpo_selftest_lose_copy(lost)
    got = clp.grpo_norm_fwd(x, w, residual=r, kind=kind, z=z, ckpt=ckpt)
    torch.cuda.synchronize()
    nan = _rows_or_nan(got.y, want.y, lost)
    assert int(nan.sum()) < n // 20  # one CTA's rows
    for a, b in ((got.z, want.z), (got.rstd, want.rstd), (ckpt.q.float(), want.ckpt.q.float())):
        assert torch.equal(_rows_or_nan(a, b, lost), nan)
    if kind == "layer":
        assert torch.equal(_rows_or_nan(got.mean, want.mean, lost), nan)
    again = clp.grpo_norm_fwd(x, w, residual=r, kind=kind)
    assert torch.equal(again.y, want.y) and torch.equal(again.z, want.z)


# Beyond 8192 columns two CTAs share a row, at column 6144 of 12001, and only the
# first of them loses its copy: the other still owes it the row's sums.
@pytest.mark.parametrize("d", [512, 1001, 4096, 12001])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("source", ["x", "ckpt"])
def test_norm_backward_leaves_nan(clp, d, kind, source):
    n, lost = 2000, 5
    g = torch.Generator().manual_seed(d)
    x, dy, dr = (torch.randn(n, d, generator=g).to(DEV, torch.bfloat16) for _ in range(3))
    w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    f = clp.grpo_norm_fwd(x, w, kind=kind, want_ckpt=True)
    src = x if source == "x" else f.ckpt
    args = (dy, src, w, f.mean, f.rstd)
    kw = dict(dres=dr, kind=kind, want_dbias=True)
    want = clp.grpo_norm_bwd(*args, **kw)
    dx = torch.full_like(dy, 7.0)
    t0 = time.perf_counter()
    clp.grpo_selftest_lose_copy(lost)
    got = clp.grpo_norm_bwd(*args, dx=dx, **kw)
    torch.cuda.synchronize()
    assert 0.3 < time.perf_counter() - t0 < 10.0
    nan = _rows_or_nan(got.dx, want.dx, lost)
    assert int(nan.sum()) < n // 20  # one CTA's rows
    mine = 6144 if d > 8192 else d
    for a, b in ((got.dweight, want.dweight), (got.dbias, want.dbias)):
        assert torch.isnan(a[:mine]).all()
        assert torch.equal(a[mine:], b[mine:])
    again = clp.grpo_norm_bwd(*args, **kw)
    assert all(torch.equal(a, b) for a, b in zip(again, want))
