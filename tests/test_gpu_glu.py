"""GPU: the gated feed-forward block against its formulas in fp64."""

import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16
ACTS = ["silu", "gelu", "gelu_tanh", "relu"]


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


def _weights(g, f, d, t):
    return _randn(g, f, d, t=t, scale=d ** -0.5), _randn(g, f, d, t=t, scale=d ** -0.5)


def _act64(name, g):
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        phi = 0.5 * torch.erfc(-g * 0.5 ** 0.5)
        return g * phi, phi + g * torch.exp(-g * g / 2) / (2 * torch.pi) ** 0.5
    if name == "gelu_tanh":
        c = (2 / torch.pi) ** 0.5
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 0.134145 * g * g)
    return g.clamp(min=0), (g > 0).double()


# Units of fp32 that an activation or its slope, both of size O(1 + |g|), may be off:
# __expf and the quick division are off by 2 + 1.2 |g| and 2, erfc by a few; |g| < 9 in
# these tests.
ACT_ULP = 32 * 2.0 ** -23


def _sum_error(a, b):
    """How far the tensor core's fp32 sum over k of a_ik b_jk may be: it cuts off, one
    unit of 2^-23 of the partial sum per 16 products and at the join."""
    return (a.shape[1] / 16 + 4) * 2.0 ** -23 * (a.abs() @ b.abs().t())


def _check(got, want, err, t):
    """|got - want| within the error before the rounding and half a step of it; fp16
    below its normal range rounds by 2^-25."""
    half = torch.finfo(t).eps / 2
    tol = half * (want.abs() + err) + err + (2.0 ** -25 if t is HF else 0.0)
    over = (got.double() - want).abs() - tol
    assert not torch.isnan(over).any()
    assert over.max().item() <= 0, f"beyond its bound by {over.max().item():.3e}"


SIZES = [(1, 8, 8), (7, 64, 128), (128, 72, 136), (129, 520, 264), (257, 1000, 1368),
         (300, 64, 2048), (3, 2048, 40), (1000, 256, 128), (17, 4104, 200), (16, 1536, 264),
         (64, 136, 1160), (33, 8, 256)]


@pytest.mark.parametrize("n,d,f", SIZES)
@pytest.mark.parametrize("t", [BF, HF])
def test_forward(clp, n, d, f, t):
    g = _gen(n + d + f)
    x, (wg, wu) = _randn(g, n, d, t=t), _weights(g, f, d, t)
    x64, g64, u64 = x.double(), wg.double(), wu.double()
    gp, up = x64 @ g64.t(), x64 @ u64.t()
    eg, eu = _sum_error(x64, g64), _sum_error(x64, u64)
    for act in ACTS:
        r = clp.grpo_glu_fwd(x, wg, wu, act=act, want_gates=True, want_ckpt=True)
        a, s = _act64(act, gp)
        # |act'| <= 1.13
        ea = 1.13 * eg + ACT_ULP * (1 + gp.abs())
        _check(r.h, a * up, ea * (up.abs() + eu) + a.abs() * eu + 2.0 ** -23 * (a * up).abs(), t)
        _check(r.gate, gp, eg, t)
        _check(r.up, up, eu, t)
        c = clp.grpo_ckpt_pack(r.h)
        assert torch.equal(r.ckpt.q.view(torch.uint8), c.q.view(torch.uint8))
        assert torch.equal(r.ckpt.exponents, c.exponents)
        assert torch.equal(clp.grpo_glu_fwd(x, wg, wu, act=act).h, r.h)


@pytest.mark.parametrize("n,d,f", SIZES)
@pytest.mark.parametrize("t", [BF, HF])
def test_backward(clp, n, d, f, t):
    g = _gen(n + d + f + 1)
    x, (wg, wu), dh = _randn(g, n, d, t=t), _weights(g, f, d, t), _randn(g, n, f, t=t, scale=0.1)
    x64, g64, u64, dh64 = (z.double() for z in (x, wg, wu, dh))
    gp, up = x64 @ g64.t(), x64 @ u64.t()
    gate, up16 = gp.to(t), up.to(t)
    for act in ACTS:
        for kept in (True, False):
            if kept:
                r = clp.grpo_glu_bwd(dh, None, wg, wu, gate=gate, up=up16, act=act, want_h=True)
                ga, ua, eg, eu = gate.double(), up16.double(), 0.0, 0.0
            else:
                r = clp.grpo_glu_bwd(dh, x, wg, wu, act=act, want_h=True)
                ga, ua, eg, eu = gp, up, _sum_error(x64, g64), _sum_error(x64, u64)
            a, s = _act64(act, ga)
            if act == "relu" and not kept:  # its slope jumps where the sign is in doubt
                clear = (ga.abs() > eg).double()
                a, s, dhc = a, s, dh64 * clear
                got = [r.dgate.double() * clear, r.dup]
            else:
                dhc, got = dh64, [r.dgate, r.dup]
            ea = 1.13 * eg + ACT_ULP * (1 + ga.abs())
            es = 1.2 * eg + ACT_ULP * (1 + ga.abs())  # |act''| <= 1.2
            _check(got[0], dhc * ua * s,
                   dhc.abs() * (es * (ua.abs() + eu) + s.abs() * eu) + 2.0 ** -22 * (dhc * ua * s).abs(), t)
            _check(got[1], dh64 * a, dh64.abs() * ea + 2.0 ** -23 * (dh64 * a).abs(), t)
            _check(r.h, a * ua, ea * (ua.abs() + eu) + a.abs() * eu + 2.0 ** -23 * (a * ua).abs(), t)
            dg, du = r.dgate.double(), r.dup.double()
            err = _sum_error(torch.cat([dg, du], 1), torch.cat([g64, u64]).reshape(2 * f, d).t())
            _check(r.dx, dg @ g64 + du @ u64, err, t)


def test_gradients_are_the_differences(clp):
    # L = sum h dh, a step of 2^-6 along a direction in x and in the weights: the
    # central difference is off by e^2 / 6 of the third derivative (under 1e-3 here),
    # the gradients by their 16-bit roundings, 2^-11 each, of independent sign.
    g = _gen(5)
    n, d, f = 24, 64, 96
    x, (wg, wu), dh = _randn(g, n, d, t=HF), _weights(g, f, d, HF), _randn(g, n, f, t=HF)
    r = clp.grpo_glu_bwd(dh, x, wg, wu, act="gelu_tanh")
    dwg, dwu = clp.grpo_glu_wgrad(r.dgate, r.dup, x)

    def loss(x, wg, wu):
        a, _ = _act64("gelu_tanh", x @ wg.t())
        return (a * (x @ wu.t()) * dh.double()).sum()

    at = [z.double() for z in (x, wg, wu)]
    for i, grad in enumerate((r.dx, dwg, dwu)):
        v = torch.randn(at[i].shape, generator=g, device=DEV).double()
        v /= v.norm()
        e = 2.0 ** -6
        lo, hi = [list(at) for _ in range(2)]
        lo[i], hi[i] = at[i] - e * v, at[i] + e * v
        diff = (loss(*hi) - loss(*lo)) / (2 * e)
        assert abs((grad.double() * v).sum() - diff) <= 3e-3 * grad.double().norm()


MASKS = ["some", "none", "one", "tail", "blocks"]


def _mask(kind, n, g):
    m = torch.zeros(n, dtype=torch.uint8, device=DEV)
    if kind == "some":
        m = (torch.rand(n, generator=g, device=DEV) < 0.5).to(torch.uint8)
    elif kind == "one":
        m[n // 2] = 1
    elif kind == "tail":
        m[:n // 3] = 1
    elif kind == "blocks":  # completions of 96 slots
        m = ((torch.arange(n, device=DEV) % 96) < 40).to(torch.uint8) * 255
    return m


@pytest.mark.parametrize("kind", MASKS)
@pytest.mark.parametrize("n", [1, 37, 700])
def test_masked_rows_do_not_exist(clp, kind, n):
    g = _gen(n)
    d, f = 136, 264
    x, (wg, wu), dh = _randn(g, n, d), _weights(g, f, d, BF), _randn(g, n, f)
    gate, up = _randn(g, n, f), _randn(g, n, f)
    m = _mask(kind, n, g)
    off = m == 0
    want = [clp.grpo_glu_fwd(x, wg, wu, want_gates=True),
            clp.grpo_glu_bwd(dh, x, wg, wu, want_h=True),
            clp.grpo_glu_bwd(dh, x, wg, wu, gate=gate, up=up, want_h=True)]
    for z in (x, dh, gate, up):
        z[off] = float("nan")
    r = clp.grpo_glu_fwd(x, wg, wu, mask=m, want_gates=True, want_ckpt=True)
    got = [r, clp.grpo_glu_bwd(dh, x, wg, wu, mask=m, want_h=True),
           clp.grpo_glu_bwd(dh, x, wg, wu, gate=gate, up=up, mask=m, want_h=True)]
    for a, b in zip(got, want):
        for p, q in zip(a, b):
            if p is None or q is None:
                continue
            assert (p[off] == 0).all()
            assert torch.equal(p[~off], q[~off])
    c = clp.grpo_ckpt_pack(r.h, mask=m)
    assert torch.equal(r.ckpt.q.view(torch.uint8), c.q.view(torch.uint8))
    assert torch.equal(r.ckpt.exponents, c.exponents)


def _wide(t, rows, cols, g, fill=7.0):
    """A tensor of [rows, cols] inside a wider one, and the wider one."""
    wide = torch.full((rows + 2, cols + 24), fill, dtype=t, device=DEV)
    return wide[1:-1, 8:-16], wide


@pytest.mark.parametrize("n", [5, 20, 200])
def test_rows_apart_and_nothing_beyond_them(clp, n):
    g = _gen(n)
    d, f = 200, 328
    x, xw = _wide(BF, n, d, g)
    x.copy_(_randn(g, n, d))
    w = _randn(g, 2 * f, d, scale=d ** -0.5)  # both weights in one
    wg, wu = w[:f], w[f:]
    dh, _ = _wide(BF, n, f, g)
    dh.copy_(_randn(g, n, f))
    outs, wide = zip(*[_wide(BF, n, f, g) for _ in range(6)])
    dx, dxw = _wide(BF, n, d, g)
    want = clp.grpo_glu_fwd(x.contiguous(), wg.clone(), wu.clone(), want_gates=True)
    got = clp.grpo_glu_fwd(x, wg, wu, h=outs[0], gate=outs[1], up=outs[2])
    for p, q in zip(got[:3], want[:3]):
        assert torch.equal(p, q)
    wb = clp.grpo_glu_bwd(dh.contiguous(), x.contiguous(), wg.clone(), wu.clone(), want_h=True)
    gb = clp.grpo_glu_bwd(dh, x, wg, wu, dgate=outs[3], dup=outs[4], h=outs[5], dx=dx)
    for p, q in zip(gb, wb):
        assert torch.equal(p, q)
    dw = clp.grpo_glu_wgrad(gb.dgate, gb.dup, x)
    for p, q in zip(dw, clp.grpo_glu_wgrad(wb.dgate, wb.dup, x.contiguous())):
        assert torch.equal(p, q)
    kb = clp.grpo_glu_bwd(dh, None, wg, wu, gate=outs[1], up=outs[2], dgate=outs[3], dup=outs[4])
    kw = clp.grpo_glu_bwd(dh.contiguous(), None, wg, wu, gate=want.gate, up=want.up)
    for p, q in zip(kb[:3], kw[:3]):
        assert torch.equal(p, q)
    for big in (*wide, dxw):
        edge = big.clone()
        edge[1:-1, 8:-16] = 7.0
        assert (edge == 7.0).all()


@pytest.mark.parametrize("n", [9, 300])
def test_gradients_in_place(clp, n):
    g = _gen(3)
    d, f = 72, 264
    x, (wg, wu), dh = _randn(g, n, d), _weights(g, f, d, BF), _randn(g, n, f)
    fwd = clp.grpo_glu_fwd(x, wg, wu, want_gates=True)
    for kept in (False, True):
        kw = dict(gate=fwd.gate, up=fwd.up) if kept else {}
        want = clp.grpo_glu_bwd(dh, x, wg, wu, want_h=True, **kw)
        dh2 = dh.clone()
        if kept:
            gate, up = fwd.gate.clone(), fwd.up.clone()
            got = clp.grpo_glu_bwd(dh2, x, wg, wu, gate=gate, up=up, dgate=gate, dup=up, h=dh2)
        else:
            got = clp.grpo_glu_bwd(dh2, x, wg, wu, dgate=dh2, want_h=True)
        for p, q in zip(got, want):
            assert torch.equal(p, q)


# Tokens, inner, hidden: one stage, odd counts, one tile cut into pieces, more tiles
# than pairs, a hidden size of half a tile, and a long sum.
WGRAD = [(1, 8, 8), (5, 24, 136), (63, 264, 72), (64, 128, 128), (65, 520, 264), (1500, 256, 256),
         (5541, 264, 136), (20000, 128, 128), (700, 3000, 2560), (2049, 1368, 520)]


@pytest.mark.parametrize("n,f,d", WGRAD)
@pytest.mark.parametrize("t", [BF, HF])
def test_weight_gradients(clp, n, f, d, t):
    g = _gen(n)
    # All of one sign: the tensor core's cutting off adds up, and no sum cancels.
    dg, du = _randn(g, n, f, t=t).abs(), _randn(g, n, f, t=t)
    x = _randn(g, n, d, t=t).abs()
    add = [torch.randn(f, d, generator=g, device=DEV) for _ in range(2)]
    want = [z.double().t() @ x.double() for z in (dg, du)]
    size = [z.double().abs().t() @ x.double() for z in (dg, du)]
    got = clp.grpo_glu_wgrad(dg, du, x)
    # Within 512 tokens a unit of 2^-23 of the partial sum per 16 products; then a
    # rounding per 512 tokens and per piece.
    tol = (512 / 16 + 4 + (n / 512 + 76) / 2) * 2.0 ** -23
    for p, q, s in zip(got, want, size):
        assert p.dtype is torch.float32
        assert ((p.double() - q).abs() <= tol * s).all()
        assert (p.double() - q).norm() <= 2e-6 * q.norm() + 1e-30
    both = clp.grpo_glu_wgrad(dg, du, x, add_gate=add[0], add_up=add[1])
    for p, q, a in zip(both, got, add):
        # one rounding more
        assert ((p.double() - q.double() - a.double()).abs() <= 2.0 ** -24 * p.double().abs() + 1e-30).all()
    ws = torch.empty(clp.grpo_glu_wgrad_workspace_size(n, f, d), dtype=torch.uint8, device=DEV)
    same = clp.grpo_glu_wgrad(dg, du, x, add_gate=add[0], add_up=add[1], dw_gate=add[0],
                              dw_up=add[1], workspace=ws)
    assert same[0] is add[0] and clp.grpo_read_device_status(ws) == 0
    for p, q in zip(same, both):
        assert torch.equal(p, q)


def test_no_tokens(clp):
    g = _gen(0)
    d, f = 64, 96
    wg, wu = _weights(g, f, d, BF)
    x, dh = _randn(g, 0, d), _randn(g, 0, f)
    assert clp.grpo_glu_fwd(x, wg, wu, want_ckpt=True).h.shape == (0, f)
    r = clp.grpo_glu_bwd(dh, x, wg, wu)
    assert r.dx.shape == (0, d)
    add = torch.ones(f, d, device=DEV)
    dg, du = clp.grpo_glu_wgrad(r.dgate, r.dup, x, add_gate=add)
    assert torch.equal(dg, add) and not du.any()


@pytest.mark.parametrize("n", [2, 40, 300])
def test_infinities_and_nan_stay_where_they_are(clp, n):
    g = _gen(9)
    d, f = 64, 136
    x, (wg, wu), dh = _randn(g, n, d), _weights(g, f, d, BF), _randn(g, n, f)
    want = clp.grpo_glu_fwd(x, wg, wu)
    back = clp.grpo_glu_bwd(dh, x, wg, wu)
    x[1, 3], dh[0, 5] = float("inf"), float("nan")
    got = clp.grpo_glu_fwd(x, wg, wu, want_ckpt=True)
    c = clp.grpo_ckpt_pack(got.h)
    assert torch.equal(got.ckpt.q.view(torch.uint8), c.q.view(torch.uint8))
    assert torch.equal(got.ckpt.exponents, c.exponents)
    keep = torch.arange(n, device=DEV) != 1
    assert torch.equal(got.h[keep], want.h[keep]) and not torch.isfinite(got.h[1]).all()
    gb = clp.grpo_glu_bwd(dh, x, wg, wu)
    keep[0] = False
    assert torch.equal(gb.dx[keep], back.dx[keep])
    assert torch.isnan(gb.dgate[0, 5]) and torch.isfinite(gb.dgate[0, :5]).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("t", [BF, HF])
def test_projections_far_out(clp, act, t):
    # Where e^-g overflows or vanishes: act(g) = g or 0, its slope 1 or 0 (gelu's and
    # silu's are below the least 16-bit number there), without a NaN.
    big = 3e4 if t is HF else 1e30
    vals = torch.tensor([-big, -200.0, -100.0, 0.0, 100.0, 200.0, big, 30.0], device=DEV).to(t)
    gate = vals.repeat(2, 1)
    up, dh = torch.ones_like(gate), torch.full_like(gate, 0.5)
    w = torch.zeros(8, 8, dtype=t, device=DEV)
    r = clp.grpo_glu_bwd(dh, None, w, w, gate=gate, up=up, act=act, want_h=True, want_dx=False)
    assert r.dx is None
    pos = vals > 0
    for row in range(2):
        assert torch.equal(r.h[row][pos], vals[pos])
        assert (r.h[row][~pos] == 0).all()
        assert (r.dgate[row][pos] == 0.5).all()
        assert torch.equal(r.dup[row][pos], vals[pos] / 2)
    at0 = {"silu": 0.25, "gelu": 0.25, "gelu_tanh": 0.25, "relu": 0.0}[act]
    assert r.dgate[0, 3].item() == at0 and (r.dgate[0, :3] == 0).all()


@pytest.mark.parametrize("n", [1, 12, 400])
def test_captured_and_replayed_beside_other_calls(clp, n):
    g = _gen(n)
    d, f = 136, 520
    x, (wg, wu), dh = _randn(g, n, d), _weights(g, f, d, BF), _randn(g, n, f)
    m = _mask("some", n, g)
    ws = torch.empty(clp.grpo_glu_wgrad_workspace_size(n, f, d), dtype=torch.uint8, device=DEV)

    def run():
        a = clp.grpo_glu_fwd(x, wg, wu, mask=m, want_gates=True, want_ckpt=True)
        b = clp.grpo_glu_bwd(dh, x, wg, wu, mask=m, want_h=True)
        c = clp.grpo_glu_bwd(dh, x, wg, wu, gate=a.gate, up=a.up, mask=m)
        return [a.h, a.ckpt.data[:0], *b, *c[:3], *clp.grpo_glu_wgrad(b.dgate, b.dup, x, workspace=ws)]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    x.copy_(_randn(g, n, d))
    dh.copy_(_randn(g, n, f))
    want = [z.clone() for z in run()]
    side = torch.cuda.Stream()
    for _ in range(3):
        for z in out:
            z.fill_(1)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        clp.grpo_glu_fwd(x, wg, wu)  # another call meanwhile
        torch.cuda.current_stream().wait_stream(side)
        for p, q in zip(out, want):
            assert torch.equal(p, q)


@pytest.mark.parametrize("t", [BF, HF])
def test_checkpoints_of_any_size_of_value(clp, t):
    # Blocks from the type's least to its largest numbers, and beyond it.
    g = _gen(31)
    n, d, f = 300, 64, 320
    x, (wg, wu) = _randn(g, n, d, t=t), _weights(g, f, d, t)
    span = torch.linspace(-24, 16 if t is HF else 60, n, device=DEV)
    x = (x.double() * (2.0 ** span.double())[:, None]).to(t)
    r = clp.grpo_glu_fwd(x, wg, wu, act="relu", want_ckpt=True)
    c = clp.grpo_ckpt_pack(r.h)
    assert torch.equal(r.ckpt.q.view(torch.uint8), c.q.view(torch.uint8))
    assert torch.equal(r.ckpt.exponents, c.exponents)


def test_two_host_threads(clp):
    g = _gen(4)
    n, d, f = 260, 136, 264
    jobs = [(_randn(g, n, d), *_weights(g, f, d, BF)) for _ in range(2)]
    want = [clp.grpo_glu_fwd(*j).h for j in jobs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                h = clp.grpo_glu_fwd(*jobs[i]).h
            torch.cuda.current_stream().synchronize()
            if not torch.equal(h, want[i]):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for z in threads:
        z.start()
    for z in threads:
        z.join()
    assert not bad


def test_rows_are_independent_of_their_neighbours(clp):
    # A row's h is that of the row alone: few rows, many rows, whatever the form.
    g = _gen(8)
    d, f = 520, 264
    x, (wg, wu) = _randn(g, 600, d), _weights(g, f, d, BF)
    all_rows = clp.grpo_glu_fwd(x, wg, wu).h.double()
    for n in (1, 2, 3, 5, 8, 9, 16, 17, 31, 32, 33, 64, 65, 128):
        part = clp.grpo_glu_fwd(x[:n], wg, wu).h.double()
        # Two fp32 sums in different orders, before their rounding: a step at most.
        assert ((part - all_rows[:n]).abs() <= 2.0 ** -7 * all_rows[:n].abs() + 1e-6).all()
        assert (part - all_rows[:n]).norm() <= 2.0 ** -8 * all_rows[:n].norm()


@pytest.mark.parametrize("call", ["fwd", "again", "kept"])
def test_a_lost_copy_leaves_nan_and_the_context(clp, call):
    g = _gen(2)
    n, d, f = 700, 1024, 2048
    x, (wg, wu), dh = _randn(g, n, d), _weights(g, f, d, BF), _randn(g, n, f)
    gates = clp.grpo_glu_fwd(x, wg, wu, want_gates=True)

    def run():
        if call == "fwd":
            return [clp.grpo_glu_fwd(x, wg, wu).h]
        if call == "again":
            return list(clp.grpo_glu_bwd(dh, x, wg, wu)[:3])
        return list(clp.grpo_glu_bwd(dh, x, wg, wu, gate=gates.gate, up=gates.up)[2:3])

    want = run()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    clp.grpo_selftest_lose_copy(5)
    got = run()
    torch.cuda.synchronize()
    assert 0.3 < time.perf_counter() - t0 < 30.0
    for p, q in zip(got, want):
        assert torch.isnan(p).any()
    p, q = got[0], want[0]  # what is not NaN is right
    fine = ~torch.isnan(p)
    assert torch.equal(p[fine], q[fine])
    for p, q in zip(run(), want):
        assert torch.equal(p, q)


def test_a_lost_copy_of_the_weight_gradient_is_reported(clp):
    g = _gen(2)
    n, d, f = 4096, 256, 256
    x, dg, du = _randn(g, n, d), _randn(g, n, f), _randn(g, n, f)
    ws = torch.empty(clp.grpo_glu_wgrad_workspace_size(n, f, d), dtype=torch.uint8, device=DEV)
    want = clp.grpo_glu_wgrad(dg, du, x, workspace=ws)
    clp.grpo_selftest_lose_copy(7)
    got = clp.grpo_glu_wgrad(dg, du, x, workspace=ws)
    assert clp.grpo_read_device_status(ws) == -7
    assert torch.isnan(got[0]).any() or torch.isnan(got[1]).any()
    for p, q in zip(got, want):
        fine = ~torch.isnan(p)
        assert torch.equal(p[fine], q[fine])
    for p, q in zip(clp.grpo_glu_wgrad(dg, du, x, workspace=ws), want):
        assert torch.equal(p, q)


def test_a_lost_copy_with_something_to_add(clp):
    # More tiles than pairs, so that tiles are whole and their boxes in flight.
    g = _gen(3)
    n, d, f = 1000, 2560, 2560
    x, dg, du = _randn(g, n, d), _randn(g, n, f), _randn(g, n, f)
    add = torch.randn(f, d, generator=g, device=DEV)
    ws = torch.empty(clp.grpo_glu_wgrad_workspace_size(n, f, d), dtype=torch.uint8, device=DEV)
    want = clp.grpo_glu_wgrad(dg, du, x, add_gate=add, add_up=add, workspace=ws)
    for stage in (0, 20):
        clp.grpo_selftest_lose_copy(stage)
        got = clp.grpo_glu_wgrad(dg, du, x, add_gate=add, add_up=add, workspace=ws)
        assert clp.grpo_read_device_status(ws) == -7
        assert torch.isnan(got[0]).any() or torch.isnan(got[1]).any()
        for p, q in zip(got, want):
            fine = ~torch.isnan(p)
            assert torch.equal(p[fine], q[fine])
    for p, q in zip(clp.grpo_glu_wgrad(dg, du, x, add_gate=add, add_up=add, workspace=ws), want):
        assert torch.equal(p, q)


def test_more_masked_rows_than_are_listed(clp):
    # Beyond 131072 rows the tiles are of consecutive rows, masked ones among them.
    g = _gen(12)
    n, d, f = 131_100, 16, 24
    x, (wg, wu), dh = _randn(g, n, d), _weights(g, f, d, BF), _randn(g, n, f)
    m = _mask("some", n, g)
    m[1000:3000] = 0
    off = m == 0
    want = clp.grpo_glu_fwd(x, wg, wu), clp.grpo_glu_bwd(dh, x, wg, wu, want_h=True)
    x[off], dh[off] = float("nan"), float("nan")
    got = (clp.grpo_glu_fwd(x, wg, wu, mask=m),
           clp.grpo_glu_bwd(dh, x, wg, wu, mask=m, want_h=True))
    for a, b in zip(got, want):
        for p, q in zip(a, b):
            if p is not None:
                assert (p[off] == 0).all() and torch.equal(p[~off], q[~off])


@pytest.mark.parametrize("n", [16 * 8192, 16 * 8192 - 5])
def test_as_many_masked_rows_as_are_listed(clp, n):
    g = _gen(13)
    d, f = 8, 16
    x, (wg, wu) = _randn(g, n, d), _weights(g, f, d, BF)
    m = torch.zeros(n + 3, dtype=torch.uint8, device=DEV)[3:]  # off 16 bytes
    m[-1] = m[77] = 1
    h = clp.grpo_glu_fwd(x, wg, wu, mask=m).h
    want = clp.grpo_glu_fwd(x, wg, wu).h
    assert torch.equal(h[m != 0], want[m != 0]) and not h[m == 0].any()


@pytest.mark.parametrize("n", [112, 368, 240, 256, 111, 113])
def test_segments_apart_in_the_last_tile(clp, n):
    # Every second segment of a tile whose rows end 112 behind its first: the places
    # that hold none must not look like the eighth of eight in a row.
    g = _gen(n)
    d, f = 72, 136
    x, (wg, wu), dh = _randn(g, n, d), _weights(g, f, d, BF), _randn(g, n, f)
    want = clp.grpo_glu_fwd(x, wg, wu), clp.grpo_glu_bwd(dh, x, wg, wu, want_h=True)
    at = torch.arange(n, device=DEV) // 16
    for keep in (at % 2 == 0, at % 3 == 0, at >= at.max() - 1, at != at.max() // 2):
        m = keep.to(torch.uint8)
        got = (clp.grpo_glu_fwd(x, wg, wu, mask=m),
               clp.grpo_glu_bwd(dh, x, wg, wu, mask=m, want_h=True))
        for a, b in zip(got, want):
            for p, q in zip(a, b):
                if p is not None:
                    assert torch.equal(p[keep], q[keep]) and not p[~keep].any()


# Rows, hidden, inner: one tile in 50 pieces; a tile to a few pairs each; whole rounds
# and a cut one (80 tiles on 76 pairs); columns and rows that end inside tiles.
CUT = [(3, 48, 12800), (64, 2048, 4096), (35, 496, 6976), (600, 776, 4096), (2500, 2048, 4096),
       (300, 264, 4096)]


@pytest.mark.parametrize("n,d,f", CUT)
@pytest.mark.parametrize("t", [BF, HF])
def test_dx_in_pieces(clp, n, d, f, t):
    g = _gen(n)
    (wg, wu), dh = _weights(g, f, d, t), _randn(g, n, f, t=t, scale=0.1)
    gate, up = _randn(g, n, f, t=t), _randn(g, n, f, t=t)
    need = clp.grpo_glu_bwd_workspace_size(n, f, d)
    assert need > 0
    ws = torch.full((need // 4,), float("nan"), device=DEV)
    none = torch.empty(0, device=DEV)
    m = _mask("blocks", n, g)
    m[0] = 1
    off = m == 0
    big = torch.cat([wg.double(), wu.double()])
    for mask in (None, m):
        if mask is not None:
            dh[off] = float("nan")
        kw = dict(gate=gate, up=up, mask=mask)
        r = clp.grpo_glu_bwd(dh, None, wg, wu, workspace=ws, **kw)
        both = torch.cat([r.dgate.double(), r.dup.double()], 1)
        want, err = both @ big, _sum_error(both, big.t())
        _check(r.dx, want, err, t)
        _check(clp.grpo_glu_bwd(dh, None, wg, wu, workspace=none, **kw).dx, want, err, t)
        again = clp.grpo_glu_bwd(dh, None, wg, wu, **kw)
        assert torch.equal(again.dx, r.dx)
        if mask is not None:
            assert not r.dx[off].any()
    dx, wide = _wide(t, n, d, g)
    assert torch.equal(clp.grpo_glu_bwd(dh, None, wg, wu, gate=gate, up=up, mask=m, dx=dx).dx, r.dx)
    wide[1:-1, 8:-16] = 7.0
    assert (wide == 7.0).all()


def test_a_lost_copy_of_dx_in_pieces(clp):
    g = _gen(21)
    n, d, f = 64, 512, 8192
    (wg, wu), dh = _weights(g, f, d, BF), _randn(g, n, f)
    gate, up = _randn(g, n, f), _randn(g, n, f)
    want = clp.grpo_glu_bwd(dh, None, wg, wu, gate=gate, up=up).dx
    clp.grpo_selftest_lose_copy(3)
    got = clp.grpo_glu_bwd(dh, None, wg, wu, gate=gate, up=up).dx
    fine = ~torch.isnan(got)
    assert not fine.all() and torch.equal(got[fine], want[fine])
    assert torch.equal(clp.grpo_glu_bwd(dh, None, wg, wu, gate=gate, up=up).dx, want)


def test_offsets_beyond_32_bits(clp):
    # 2.3e9 values of h: the last rows are what they are on their own.
    g = _gen(30)
    n, d, f = 140_000, 64, 16384
    x, (wg, wu) = _randn(g, n, d), _weights(g, f, d, BF)
    last = slice(n - 200, n)
    r = clp.grpo_glu_fwd(x, wg, wu)
    want = clp.grpo_glu_fwd(x[last], wg, wu)
    assert torch.equal(r.h[last], want.h)
    dg = r.h  # any gradient will do, in place
    b = clp.grpo_glu_bwd(dg, x, wg, wu, dgate=dg, workspace=torch.empty(0, device=DEV))
    wb = clp.grpo_glu_bwd(want.h, x[last], wg, wu, workspace=torch.empty(0, device=DEV))
    for p, q in zip(b[:3], wb[:3]):
        assert torch.equal(p[last], q)
    k = clp.grpo_glu_bwd(b.dup, None, wg, wu, gate=b.dgate, up=b.dup, dgate=b.dgate, want_dx=False)
    kw = clp.grpo_glu_bwd(wb.dup, None, wg, wu, gate=wb.dgate, up=wb.dup, want_dx=False)
    assert torch.equal(k.dgate[last], kw.dgate) and torch.equal(k.dup[last], kw.dup)
