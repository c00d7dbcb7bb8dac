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


def _even(g, *shape, t, scale):
    """Values of one sign and size: what a sum cuts off adds up, and nothing cancels."""
    return (scale * (0.5 + 0.5 * torch.rand(*shape, generator=g, device=DEV))).to(t)


def _whole(got, want, t, products, terms=1):
    """Each value is within half a step, of its own binade, of one whose fp32 sums are whole:
    a sum of at most 2048 products may be cut off by one unit of 2^-23 of itself per 16
    products and at four joins, and such sums are added with roundings of 2^-24 of what is
    there by then, half of the whole on average. (The roundings to 16 bits do not cancel in
    a mean: long sums of one sign all lie within one step.)"""
    err = terms * ((2048 / 16 + 4) * 2.0 ** -23 + (products / 1024 / 2 + 2) * 2.0 ** -24)
    half = torch.exp2(torch.floor(torch.log2(want * (1 + err)))) * (torch.finfo(t).eps / 2)
    over = ((got.double() - want).abs() - half) / want
    assert over.max().item() <= err, f"{over.max().item():.2e} beyond half a step, not {err:.2e}"


@pytest.mark.parametrize("t,n,d", [(HF, 300, 1 << 17), (HF, 300, 1 << 20), (HF, 3, 1 << 20),
                                   (BF, 300, 1 << 20), (BF, 8, 1 << 20), (HF, 300, 5000)])
def test_long_sums_of_the_forward_pass_are_not_cut_short(clp, t, n, d):
    g = _gen(1)
    f, s = 64, (14.0 / d) ** 0.5
    x, wg, wu = _even(g, n, d, t=t, scale=s), _even(g, f, d, t=t, scale=s), _even(g, f, d, t=t, scale=s)
    gate, up = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    r = clp.grpo_glu_fwd(x, wg, wu, act="relu", want_gates=True)
    _whole(r.gate, gate, t, d)
    _whole(r.up, up, t, d)
    _whole(r.h, gate * up, t, d, 2)
    if n <= 8:
        return
    dh = _even(g, n, f, t=t, scale=0.1)
    b = clp.grpo_glu_bwd(dh, x, wg, wu, act="relu", want_h=True, want_dx=False)
    _whole(b.dgate, dh.double() * up, t, d)
    _whole(b.dup, dh.double() * gate, t, d)
    _whole(b.h, gate * up, t, d, 2)


@pytest.mark.parametrize("t,n,f", [(HF, 300, 1 << 17), (HF, 200, 14336), (BF, 64, 1 << 19),
                                   (HF, 2000, 3000), (HF, 9, 1 << 20)])
@pytest.mark.parametrize("cut", [True, False])
def test_long_sums_of_dx_are_not_cut_short(clp, t, n, f, cut):
    g = _gen(2)
    d, s = 64, (7.0 / f) ** 0.5
    wg, wu, dh = (_even(g, m, k, t=t, scale=s) for m, k in ((f, d), (f, d), (n, f)))
    ones = torch.ones(n, f, device=DEV, dtype=t)
    ws = None if cut else torch.empty(0, device=DEV)
    r = clp.grpo_glu_bwd(dh, None, wg, wu, gate=ones, up=ones, act="relu", workspace=ws)
    assert torch.equal(r.dgate, dh) and torch.equal(r.dup, dh)
    want = dh.double() @ (wg.double() + wu.double())
    _whole(r.dx, want, t, 2 * f)


@pytest.mark.parametrize("t,d,f", [(HF, 1024, 328), (HF, 1032, 328), (BF, 1032, 520),
                                   (BF, 2112, 200), (HF, 4160, 200), (HF, 6200, 1368),
                                   (BF, 32776, 136)])
@pytest.mark.parametrize("n", [33, 300])
def test_sums_about_the_longest(clp, t, d, f, n):
    # Against fp64, tile widths and masks as they come; a tile's sum is one, two or more.
    g = _gen(d)
    x, wg, wu = (_randn(g, m, k, t=t, scale=c) for m, k, c in
                 ((n, d, 1.0), (f, d, d ** -0.5), (f, d, d ** -0.5)))
    dh = _randn(g, n, f, t=t)
    m = (torch.rand(n, generator=g, device=DEV) < 0.7).to(torch.uint8)
    m[0] = 1
    live = m != 0
    gate, up = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    half = torch.finfo(t).eps / 2
    # One unit of 2^-23 of the partial sum per 16 products and at joins.
    err = (d / 16 + 8) * 2.0 ** -23 * (x.double().abs() @ wg.double().abs().t())
    plain = clp.grpo_glu_fwd(x, wg, wu, act="relu", want_gates=True, want_ckpt=True)
    assert ((plain.gate.double() - gate).abs() <= err + half * (gate.abs() + err) + 2.0 ** -25).all()
    x[~live], dh[~live] = float("nan"), float("nan")
    r = clp.grpo_glu_fwd(x, wg, wu, act="relu", mask=m, want_gates=True)
    for p, q in zip(r[:3], plain[:3]):
        assert torch.equal(p[live], q[live]) and not p[~live].any()
    b = clp.grpo_glu_bwd(dh, x, wg, wu, act="silu", mask=m, want_h=True)
    both = torch.cat([b.dgate, b.dup], 1).double()
    w2 = torch.cat([wg, wu]).double()
    want = both @ w2
    err = (2 * f / 16 + 8) * 2.0 ** -23 * (both.abs() @ w2.abs())
    assert ((b.dx.double() - want).abs() <= err + half * (want.abs() + err) + 2.0 ** -25)[live].all()
    s = torch.sigmoid(gate)
    want = dh.double() * gate * s
    # |silu'| <= 1.1; __expf and the quick division are off by 2 + 1.2 |g| and 2 units.
    err = dh.double().abs() * (1.1 * (d / 16 + 8) * 2.0 ** -23 * 4 * d ** 0.5
                               + 32 * 2.0 ** -23 * (1 + gate.abs()))
    assert ((b.dup.double() - want).abs() <= err + half * (want.abs() + err) + 2.0 ** -25)[live].all()


@pytest.mark.parametrize("call", ["fwd", "again", "dx"])
@pytest.mark.parametrize("stage", [5, 40, 70])
def test_a_lost_copy_of_a_long_sum(clp, call, stage):
    # Five sums a tile: the copy is lost in the first, the third or the last.
    g = _gen(7)
    n, d, f = (700, 72 * 64, 1024) if call != "dx" else (2600, 1024, 36 * 64)
    x, wg, wu, dh = (_randn(g, a, b, t=HF, scale=c) for a, b, c in
                     ((n, d, 1.0), (f, d, d ** -0.5), (f, d, d ** -0.5), (n, f, 1.0)))
    none = torch.empty(0, device=DEV)

    def run():
        if call == "fwd":
            return list(clp.grpo_glu_fwd(x, wg, wu, want_gates=True)[:3])
        if call == "again":
            return list(clp.grpo_glu_bwd(dh, x, wg, wu, want_dx=False)[:2])
        return [clp.grpo_glu_bwd(dh, None, wg, wu, gate=dh, up=dh, workspace=none).dx]

    want = run()
    clp.grpo_selftest_lose_copy(stage)
    got = run()
    for p, q in zip(got, want):
        fine = ~torch.isnan(p)
        assert not fine.all() and torch.equal(p[fine], q[fine])
    for p, q in zip(run(), want):
        assert torch.equal(p, q)


@pytest.mark.parametrize("n", [1, 8, 12, 400])
def test_all_that_a_captured_forward_pass_writes(clp, n):
    g = _gen(n)
    d, f = 136, 520
    x, wg, wu = _randn(g, n, d), _randn(g, f, d, scale=d ** -0.5), _randn(g, f, d, scale=d ** -0.5)
    m = (torch.rand(n, generator=g, device=DEV) < 0.6).to(torch.uint8)
    m[0] = 1
    clp.grpo_glu_fwd(x, wg, wu, mask=m, want_gates=True, want_ckpt=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = clp.grpo_glu_fwd(x, wg, wu, mask=m, want_gates=True, want_ckpt=True)
    for seed in (1, 2):
        x.copy_(_randn(_gen(seed), n, d))
        want = clp.grpo_glu_fwd(x, wg, wu, mask=m, want_gates=True, want_ckpt=True)
        for z in (held.h, held.gate, held.up, held.ckpt.data):
            z.fill_(1)
        graph.replay()
        for p, q in zip((held.h, held.gate, held.up), (want.h, want.gate, want.up)):
            assert torch.equal(p, q)
        assert torch.equal(held.ckpt.q.view(torch.uint8), want.ckpt.q.view(torch.uint8))
        assert torch.equal(held.ckpt.exponents, want.ckpt.exponents)
