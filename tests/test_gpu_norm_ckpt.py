"""GPU: norms and 8-bit checkpoints against the fp64 oracle.

Tolerances count roundings. E = 2^-24 is fp32's half step, R = eps / 2 the half
step of the tensors' type (bf16 2^-8, fp16 2^-11, fp32 2^-24).

- z = x + r: one fp32 addition, exact in fp64, rounded once: bit for bit.
- mean: a thread's 16 values, 5 shuffles, up to 16 warps in 5 more, a division:
  at most 30 roundings of mean |z|; two more walks' values a thread beyond 8192
  columns (32 at 16384): 50 covers both.
- rstd: as many for the sum of squares (each square 2 more), halved by the root.
- y: h = (z - mean) rstd and two more roundings, then R |y|.
- dx: sums over columns like the mean's; 60 E of the terms' magnitudes, then R |dx|.
- dw, db: one rounding per row a thread adds (at most n), per partial sum (at
  most 608 / 8 + 8) and 4 for a term; of the sum of magnitudes.
- checkpoints and what is packed: exact.
- wgrad: products are exact; at most n additions of 2 E each (the tensor core
  may cut off instead of rounding), and one for `add`.
"""

import numpy as np
import pytest
import torch

from oracle import norm_ckpt_oracle as o

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# every path: one warp (8 and 16 values a thread), several rows a CTA, one row
# a CTA, rows longer than registers; odd sizes take the one-by-one path.
WIDTHS = [1, 7, 31, 32, 33, 64, 100, 256, 257, 264, 512, 520, 1000, 1001, 1536, 2047, 2880, 4096,
          8192, 8193, 8200, 12001, 16384, 16385, 16392, 20000]


@pytest.fixture(scope="module")
def clp():
    import __graft_entry__

    __graft_entry__.build()
    import chunked_log_prob_gb300 as m

    return m


def half_step(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return float(torch.finfo(t).smallest_normal) * torch.finfo(t).eps  # a subnormal step


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def rand(g, n, d, t, scale=1.0, offset=0.0):
    x = torch.randn(n, d, generator=g) * torch.exp(0.5 * torch.randn(n, 1, generator=g))
    x = x * scale + offset
    if d > 2:
        x[:, d // 2] *= 20
    return x.to(t)


def masks(kind, n, g):
    if kind == "none":
        return None
    if kind == "all":
        return torch.zeros(n, dtype=torch.uint8)
    m = (torch.rand(n, generator=g) < 0.6).to(torch.uint8)
    return m * 3  # any nonzero byte counts


def strided(x, extra, shift):
    """The same values in rows `extra` elements further apart, `shift` elements in."""
    n, d = x.shape
    big = torch.full((n, d + extra), 99.0, dtype=x.dtype, device=x.device)
    v = big[:, shift:shift + d]
    v.copy_(x)
    return v


def check(name, got, want, tol):
    got = f64(got)
    assert got.shape == want.shape, name
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = np.argwhere(bad)[0]
        raise AssertionError(f"{name}{tuple(i)}: {got[tuple(i)]!r} against {want[tuple(i)]!r}, "
                             f"tolerance {np.broadcast_to(tol, want.shape)[tuple(i)]:.3g}; "
                             f"{bad.sum()} of {bad.size}")


def fwd_tol(z, w, y, mean, rstd, t):
    a = np.abs(z)
    mean_err = 50 * E * a.mean(1, keepdims=True)
    h = np.abs(z - mean[:, None]) * rstd[:, None]
    r = rstd[:, None]
    # rstd: centring error of the mean enters squared; 30 roundings of the sum.
    rstd_rel = 30 * E + (mean_err * r) ** 2
    return (half_step(t) * np.abs(y) + tiny(t) +
            np.abs(w) * (h * (rstd_rel + 4 * E) + mean_err * r) + 4 * E * np.abs(y)), \
        mean_err[:, 0], rstd[:, None][:, 0] * (rstd_rel[:, 0] + 2 * E)


def run_fwd(clp, n, d, dtype, wdtype, kind, residual, bias, mask, ckpt, seed, layout="packed",
            want_stats=True, poison=False):
    g = torch.Generator().manual_seed(seed)
    t, wt = DT[dtype], DT[wdtype]
    x = rand(g, n, d, t, offset=0.5)
    r = rand(g, n, d, t) if residual else None
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(wt)
    b = torch.randn(d, generator=g).to(wt) if bias else None
    m = masks(mask, n, g)
    if poison and m is not None:
        for v in (x, r):
            if v is not None:
                v[m == 0] = float("nan")
    put = (lambda v: None if v is None else v.to(DEV))
    xs, rs = put(x), put(r)
    y = z = None
    if layout != "packed":
        extra, shift = {"aligned": (24, 8), "odd": (5, 1)}[layout]
        xs = strided(xs, extra, shift)
        y = strided(torch.zeros_like(xs), extra, shift)
        if residual:
            rs = strided(rs, extra + 8, shift)
            z = strided(torch.zeros_like(xs), extra, shift)
    eps = 1e-5
    out = clp.grpo_norm_fwd(xs, put(w), put(b), residual=rs, kind=kind, eps=eps, mask=put(m),
                            want_stats=want_stats, want_ckpt=ckpt, y=y, z=z)
    torch.cuda.synchronize()
    zz = x.double() if r is None else (x.float() + r.float()).to(t).double()
    zz = zz.numpy().copy()
    live = np.ones(n, bool) if m is None else m.numpy() != 0
    zz[~live] = 0
    if residual:
        check("z", out.z, zz, 0.0)
    wy, wm, wr = o.norm_fwd(zz, f64(w), f64(b), kind, eps, mask=live)
    tol, mean_tol, rstd_tol = fwd_tol(zz, f64(w), wy, wm, wr, t)
    check("y", out.y, wy, tol * live[:, None])
    if want_stats:
        if kind == "layer":
            check("mean", out.mean, wm, mean_tol)
        check("rstd", out.rstd, wr, rstd_tol)
    if ckpt:
        q, ex = o.ckpt_pack(zz, float(torch.finfo(t).max))
        np.testing.assert_array_equal(out.ckpt.exponents.cpu().numpy(), ex)
        np.testing.assert_array_equal(f64(out.ckpt.q.float()), q)
    if layout != "packed":
        for v in (y, z):
            if v is not None:  # what lies between the rows stays
                base = v._base
                keep = torch.ones_like(base, dtype=torch.bool)
                keep[:, v.storage_offset():v.storage_offset() + d] = False
                assert (base[keep] == 99.0).all()
    return out


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_forward_widths(clp, d, dtype, kind):
    run_fwd(clp, 19, d, dtype, dtype, kind, residual=True, bias=kind == "layer", mask="some",
            ckpt=True, seed=d, poison=True)
    run_fwd(clp, 3, d, dtype, "fp32", kind, residual=False, bias=False, mask="none", ckpt=False,
            seed=d + 1)


@pytest.mark.parametrize("n", [1, 2, 7, 1216, 5000])
@pytest.mark.parametrize("d", [24, 300, 1536, 4096])
def test_norm_forward_rows(clp, n, d):
    run_fwd(clp, n, d, "bf16", "bf16", "rms", residual=True, bias=True, mask="none", ckpt=True,
            seed=n)


@pytest.mark.parametrize("layout", ["aligned", "odd"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [40, 999, 1536, 8200])
def test_norm_forward_strides(clp, layout, dtype, d):
    run_fwd(clp, 33, d, dtype, "fp32", "layer", residual=True, bias=True, mask="some", ckpt=True,
            seed=4, layout=layout)


@pytest.mark.parametrize("d", [64, 2880, 8200])
def test_norm_forward_every_row_masked(clp, d):
    out = run_fwd(clp, 40, d, "bf16", "bf16", "layer", residual=True, bias=True, mask="all",
                  ckpt=True, seed=1, poison=True)
    for v in (out.y, out.z, out.mean, out.rstd):
        assert (v == 0).all()


def test_norm_forward_without_stats_weight_or_rows(clp):
    run_fwd(clp, 5, 96, "bf16", "bf16", "rms", False, False, "none", False, 0, want_stats=False)
    x = rand(torch.Generator().manual_seed(0), 4, 72, torch.float32).to(DEV)
    out = clp.grpo_norm_fwd(x, kind="layer", eps=0.0)
    assert out.z is x
    wy, wm, wr = o.norm_fwd(f64(x), None, None, "layer", 0.0)
    check("y", out.y, wy, fwd_tol(f64(x), np.ones(72), wy, wm, wr, torch.float32)[0])
    empty = clp.grpo_norm_fwd(x[:0], want_ckpt=True)
    assert empty.y.shape == (0, 72) and empty.ckpt.q.shape == (0, 72)


def test_norm_forward_cancellation(clp):
    # Values around 1000 with spread 1: the variance is not a difference of squares.
    g = torch.Generator().manual_seed(3)
    x = (1000 + torch.randn(8, 2880, generator=g))
    out = clp.grpo_norm_fwd(x.to(DEV), kind="layer", eps=0.0)
    wy, wm, wr = o.norm_fwd(x.double().numpy(), None, None, "layer", 0.0)
    tol, _, rtol = fwd_tol(x.double().numpy(), np.ones(2880), wy, wm, wr, torch.float32)
    check("y", out.y, wy, tol)
    check("rstd", out.rstd, wr, rtol)


def test_norm_forward_nan_and_inf_stay_in_their_row(clp):
    x = rand(torch.Generator().manual_seed(0), 6, 512, torch.bfloat16).to(DEV)
    x[1, 3], x[4, 7] = float("nan"), float("inf")
    out = clp.grpo_norm_fwd(x, want_ckpt=True)
    finite = torch.isfinite(out.y.float()).all(1).cpu().tolist()
    assert finite == [True, False, True, True, False, True]
    q = out.ckpt.q.float()
    assert torch.isnan(q[1, 3]) and torch.isnan(q[4, 7]) and torch.isnan(q).sum() == 2


def test_norm_forward_in_place(clp):
    g = torch.Generator().manual_seed(9)
    for d in (512, 4096, 8200, 1001):
        x, r = (rand(g, 21, d, torch.bfloat16).to(DEV) for _ in range(2))
        w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
        want = clp.grpo_norm_fwd(x, w, residual=r)
        xi, ri = x.clone(), r.clone()
        got = clp.grpo_norm_fwd(xi, w, residual=ri, y=xi, z=ri)
        assert torch.equal(got.y, want.y) and torch.equal(got.z, want.z)
        assert got.y.data_ptr() == xi.data_ptr()


# ---------------------------------------------------------------- backward ----


def run_bwd(clp, n, d, dtype, wdtype, kind, source, dres, bias, mask, add, seed, layout="packed",
            poison=False):
    g = torch.Generator().manual_seed(seed)
    t, wt = DT[dtype], DT[wdtype]
    x = rand(g, n, d, t, offset=0.5)
    dy = rand(g, n, d, t, scale=0.1)
    dr = rand(g, n, d, t, scale=0.1) if dres else None
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(wt)
    m = masks(mask, n, g)
    live = np.ones(n, bool) if m is None else m.numpy() != 0
    _, wm, wr = o.norm_fwd(f64(x), None, None, kind, 1e-5, mask=live)
    mean = torch.from_numpy(wm).float() if kind == "layer" else None
    rstd = torch.from_numpy(wr).float()
    adds = [torch.randn(d, generator=g) if add else None for _ in range(2)]
    put = (lambda v: None if v is None else v.to(DEV))
    if source == "ckpt":
        src = clp.grpo_ckpt_pack(put(x), mask=put(m))
        q, ex = o.ckpt_pack(f64(x), float(torch.finfo(t).max), mask=live)
        z = o.ckpt_expand(q, ex)
    else:
        z = f64(x)
    if poison and m is not None:
        for v in (x, dy, dr):
            if v is not None:
                v[m == 0] = float("nan")
    if source != "ckpt":
        src = put(x)
    dyd, drd, dxd = put(dy), put(dr), None
    if layout != "packed":
        extra, shift = {"aligned": (24, 8), "odd": (5, 1)}[layout]
        dyd = strided(dyd, extra, shift)
        dxd = strided(torch.zeros_like(dyd), extra, shift)
        drd = strided(drd, extra, shift) if dres else None
        if source != "ckpt":
            src = strided(src, extra + 8, shift)
    out = clp.grpo_norm_bwd(dyd, src, put(w), put(mean), put(rstd), dres=drd, kind=kind,
                            mask=put(m), want_dbias=bias, add_dweight=put(adds[0]),
                            add_dbias=put(adds[1]) if bias else None, dx=dxd)
    torch.cuda.synchronize()
    dy64 = np.where(live[:, None], f64(dy), 0.0)
    z64 = np.where(live[:, None], z, 0.0)
    r64 = None if dr is None else np.where(live[:, None], f64(dr), 0.0)
    mean64, rstd64 = f64(mean), f64(rstd)
    dx, dw, db = o.norm_bwd(dy64, z64, f64(w), mean64, rstd64, kind, dres=r64, mask=live)
    rs = (rstd64 * live)[:, None]
    # h = (z - mean) rstd: 2 roundings of |z| + |mean| (the difference is of its
    # own size exactly rounded, so 2 of |h|).
    h = np.abs(z64 - (0 if mean64 is None else mean64[:, None])) * rs
    u = np.abs(dy64 * f64(w))
    mag = rs * (u + u.mean(1, keepdims=True) + h * (u * h).mean(1, keepdims=True))
    mag = mag + (0 if r64 is None else np.abs(r64))
    check("dx", out.dx, dx, half_step(t) * np.abs(dx) + (tiny(t) + 60 * E * mag) * live[:, None])
    k = n + 608 / 8 + 8 + 4
    a0 = 0 if adds[0] is None else adds[0].double().numpy()
    a1 = 0 if adds[1] is None else adds[1].double().numpy()
    check("dweight", out.dweight, dw + a0, k * E * (np.abs(dy64) * h).sum(0) + E * np.abs(dw + a0))
    if bias:
        check("dbias", out.dbias, db + a1, k * E * np.abs(dy64).sum(0) + E * np.abs(db + a1))
    if dxd is not None:
        base = dxd._base
        keep = torch.ones_like(base, dtype=torch.bool)
        keep[:, dxd.storage_offset():dxd.storage_offset() + d] = False
        assert (base[keep] == 99.0).all()
    return out


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("source", ["x", "ckpt"])
def test_norm_backward_widths(clp, d, dtype, source):
    run_bwd(clp, 21, d, dtype, dtype, "layer", source, dres=True, bias=True, mask="some", add=True,
            seed=d, poison=True)
    run_bwd(clp, 3, d, dtype, "fp32", "rms", source, dres=False, bias=False, mask="none",
            add=False, seed=d + 1)


@pytest.mark.parametrize("n", [1, 2, 9, 1216, 5000])
@pytest.mark.parametrize("d", [24, 300, 1536, 4096])
def test_norm_backward_rows(clp, n, d):
    run_bwd(clp, n, d, "bf16", "bf16", "rms", "ckpt", dres=True, bias=True, mask="none", add=False,
            seed=n)


@pytest.mark.parametrize("layout", ["aligned", "odd"])
@pytest.mark.parametrize("source", ["x", "ckpt"])
@pytest.mark.parametrize("d", [40, 999, 1536, 8200])
def test_norm_backward_strides(clp, layout, source, d):
    run_bwd(clp, 33, d, "bf16", "fp32", "layer", source, dres=True, bias=True, mask="some",
            add=True, seed=4, layout=layout)


@pytest.mark.parametrize("d", [64, 2880, 8200])
@pytest.mark.parametrize("source", ["x", "ckpt"])
def test_norm_backward_every_row_masked(clp, d, source):
    out = run_bwd(clp, 40, d, "bf16", "bf16", "layer", source, dres=True, bias=True, mask="all",
                  add=False, seed=1, poison=True)
    for v in out:
        assert (v == 0).all()


def test_norm_backward_no_rows_and_no_gradients(clp):
    dy = torch.zeros(0, 96, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(0, device=DEV)
    w = torch.ones(96, device=DEV)
    add = torch.arange(96, dtype=torch.float32, device=DEV)
    out = clp.grpo_norm_bwd(dy, dy, w, st, st, kind="layer", want_dbias=True, add_dweight=add)
    assert torch.equal(out.dweight, add) and (out.dbias == 0).all() and out.dx.shape == (0, 96)
    x = rand(torch.Generator().manual_seed(0), 5, 96, torch.bfloat16).to(DEV)
    r = clp.grpo_norm_fwd(x).rstd
    out = clp.grpo_norm_bwd(x, x, None, None, r)
    assert out.dweight is None and out.dbias is None
    want = o.norm_bwd(f64(x), f64(x), None, None, f64(r), "rms")[0]
    h = np.abs(f64(x)) * f64(r)[:, None]
    u = np.abs(f64(x))
    check("dx", out.dx, want, half_step(torch.bfloat16) * np.abs(want) + tiny(torch.bfloat16) +
          60 * E * f64(r)[:, None] * (u + h * (u * h).mean(1, keepdims=True)))


def test_norm_backward_in_place_and_repeatable(clp):
    g = torch.Generator().manual_seed(9)
    for d in (512, 4096, 8200, 1001):
        x, dy, dr = (rand(g, 700, d, torch.bfloat16).to(DEV) for _ in range(3))
        w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
        r = clp.grpo_norm_fwd(x, w).rstd
        want = clp.grpo_norm_bwd(dy, x, w, None, r, dres=dr)
        again = clp.grpo_norm_bwd(dy, x, w, None, r, dres=dr)
        assert torch.equal(want.dx, again.dx) and torch.equal(want.dweight, again.dweight)
        acc = want.dweight.clone()
        dyi = dy.clone()
        got = clp.grpo_norm_bwd(dyi, x, w, None, r, dres=dr, dx=dyi, dweight=acc, add_dweight=acc)
        assert torch.equal(got.dx, want.dx) and torch.equal(acc, 2 * want.dweight)
        dri = dr.clone()
        got = clp.grpo_norm_bwd(dy, x, w, None, r, dres=dri, dx=dri)
        assert torch.equal(got.dx, want.dx)


def test_norm_backward_against_differences(clp):
    # The kernels' own forward, differenced in fp32: f = sum(y dy) by fp64 sums
    # on the host. Step 2^-6: the difference's rounding is 40 E |y| |dy| per
    # value over the step, its curvature step^2 / 6 times f''' (about |h|^3).
    g = torch.Generator().manual_seed(0)
    n, d, step = 2, 48, 2.0 ** -6
    x, dy = torch.randn(n, d, generator=g), torch.randn(n, d, generator=g)
    w, b = torch.randn(d, generator=g), torch.randn(d, generator=g)
    for kind in ("layer", "rms"):
        out = clp.grpo_norm_fwd(x.to(DEV), w.to(DEV), b.to(DEV), kind=kind)
        grad = clp.grpo_norm_bwd(dy.to(DEV), x.to(DEV), w.to(DEV), out.mean, out.rstd, kind=kind,
                                 want_dbias=True)
        probes = torch.cat([x[None].repeat(d, 1, 1) + s * step * torch.eye(d)[:, None, :]
                            for s in (1, -1)])
        y = clp.grpo_norm_fwd(probes.reshape(-1, d).to(DEV), w.to(DEV), b.to(DEV), kind=kind).y
        f = (f64(y).reshape(2, d, n, d) * f64(dy)).sum(-1)
        num = (f[0] - f[1]).T / (2 * step)
        size = np.abs(f64(dy) * f64(w)).sum(1, keepdims=True)
        tol = size * (40 * E * 4 / step + step ** 2 / 6 * 8)
        check("dx", grad.dx, num, tol)


# -------------------------------------------------------------- checkpoints ----


def special_rows(t):
    top, small = float(torch.finfo(t).max), float(torch.finfo(t).smallest_normal)
    x = torch.zeros(12, 97, dtype=torch.float64)
    x[0] = top
    x[1] = torch.linspace(-top, top, 97, dtype=torch.float64)
    x[2], x[3] = small, small * 2.0 ** -5
    x[4, ::3], x[5, 64] = float("nan"), float("inf")
    x[5, 0], x[6] = 7.0, -0.0
    x[7, 32:64] = 448.0
    x[8] = torch.linspace(0, 448, 97, dtype=torch.float64)
    x[9] = torch.linspace(-1, 1, 97, dtype=torch.float64) * 2.0 ** -9
    x[9, 5] = 1.0
    x[10] = top * 0.876
    x[11, 96] = -float("inf")
    return x.to(t)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [97, 96])
def test_ckpt_special_values(clp, dtype, d):
    x = special_rows(DT[dtype])[:, :d].contiguous()
    c = clp.grpo_ckpt_pack(x.to(DEV))
    q, ex = o.ckpt_pack(f64(x), float(torch.finfo(x.dtype).max))
    np.testing.assert_array_equal(c.exponents.cpu().numpy(), ex)
    np.testing.assert_array_equal(f64(c.q.float()), q)
    back = clp.grpo_ckpt_unpack(c, x.dtype)
    want = torch.from_numpy(o.ckpt_expand(q, ex)).to(x.dtype)
    np.testing.assert_array_equal(f64(back), f64(want))
    assert torch.isfinite(back[:4].float()).all()  # the largest values stay finite


@pytest.mark.parametrize("d", [1, 8, 31, 40, 256, 257, 1535, 4096, 16392])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_ckpt_pack_and_unpack(clp, d, dtype):
    g = torch.Generator().manual_seed(d)
    n = 37
    x = rand(g, n, d, DT[dtype])
    m = masks("some", n, g)
    xp = x.clone()
    xp[m == 0] = float("nan")
    q, ex = o.ckpt_pack(f64(x), float(torch.finfo(x.dtype).max), mask=m.numpy())
    for layout in ("packed", "aligned", "odd"):
        xd = xp.to(DEV)
        if layout != "packed":
            xd = strided(xd, *{"aligned": (24, 8), "odd": (5, 1)}[layout])
        c = clp.grpo_ckpt_pack(xd, mask=m.to(DEV))
        np.testing.assert_array_equal(c.exponents.cpu().numpy(), ex)
        np.testing.assert_array_equal(f64(c.q.float()), q)
        for to in DT.values():
            out = None
            if layout != "packed":
                out = strided(torch.zeros(n, d, dtype=to, device=DEV),
                              *{"aligned": (24, 8), "odd": (5, 1)}[layout])
            back = clp.grpo_ckpt_unpack(c, to, out=out)
            want = torch.from_numpy(o.ckpt_expand(q, ex)).to(to)
            np.testing.assert_array_equal(f64(back), f64(want))
            if out is not None:
                base = out._base
                keep = torch.ones_like(base, dtype=torch.bool)
                keep[:, out.storage_offset():out.storage_offset() + d] = False
                assert (base[keep] == 99.0).all()


def test_ckpt_pack_is_the_norms(clp):
    x = rand(torch.Generator().manual_seed(1), 9, 2880, torch.bfloat16).to(DEV)
    a, b = clp.grpo_norm_fwd(x, want_ckpt=True).ckpt, clp.grpo_ckpt_pack(x)
    assert torch.equal(a.q.view(torch.uint8), b.q.view(torch.uint8))
    assert torch.equal(a.exponents, b.exponents)


# -------------------------------------------------------------------- wgrad ----


def run_wgrad(clp, n, out, d, add, seed, mask="none", stride=0):
    g = torch.Generator().manual_seed(seed)
    x = rand(g, n, d, torch.bfloat16)
    dy = rand(g, n, out, torch.bfloat16, scale=0.01)
    m = masks(mask, n, g)
    if m is not None:
        dy[m == 0] = 0
        x[m == 0] = float("nan")
    a = torch.randn(out, d, generator=g) if add else None
    c = clp.grpo_ckpt_pack(x.to(DEV), mask=None if m is None else m.to(DEV))
    dyd = dy.to(DEV)
    if stride:
        dyd = strided(dyd, stride, 8)
    ws = torch.empty(clp.grpo_ckpt_wgrad_workspace_size(n, out, d), dtype=torch.uint8, device=DEV)
    got = clp.grpo_ckpt_wgrad(dyd, c, add=None if a is None else a.to(DEV), workspace=ws)
    assert clp.grpo_read_device_status(ws) == 0
    q, ex = o.ckpt_pack(np.nan_to_num(f64(x)), float(torch.finfo(torch.bfloat16).max),
                        mask=None if m is None else m.numpy())
    x64, dy64 = o.ckpt_expand(q, ex), f64(dy)
    mag = np.abs(dy64).T @ np.abs(x64)
    want = o.wgrad(dy64, x64, f64(a))
    check("dW", got, want, (n + 1) * 2 * E * mag + E * np.abs(want))
    # Against the whole: far below what a lost tile or token would show.
    rel = np.linalg.norm(f64(got) - want) / max(np.linalg.norm(want), 1e-300)
    assert rel <= 1e-5, rel
    return got, c, dyd


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 200, 1000])
@pytest.mark.parametrize("out,d", [(8, 8), (64, 40), (136, 264), (256, 256)])
def test_wgrad_small(clp, n, out, d):
    run_wgrad(clp, n, out, d, add=n % 2 == 0, seed=n)


@pytest.mark.parametrize("n,out,d", [(4096, 256, 256), (5541, 264, 1536), (2049, 2880, 520),
                                     (300, 4096, 1000), (8200, 72, 72), (64, 1280, 2880),
                                     (20000, 16, 256)])
def test_wgrad_sizes(clp, n, out, d):
    run_wgrad(clp, n, out, d, add=True, seed=n)
    run_wgrad(clp, n, out, d, add=False, seed=n + 1, mask="some", stride=24)


def test_wgrad_no_tokens(clp):
    c = clp.grpo_ckpt_pack(torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV))
    dy = torch.zeros(0, 40, dtype=torch.bfloat16, device=DEV)
    assert (clp.grpo_ckpt_wgrad(dy, c) == 0).all()
    a = torch.randn(40, 64, device=DEV)
    assert torch.equal(clp.grpo_ckpt_wgrad(dy, c, add=a), a)
    b = a.clone()
    assert torch.equal(clp.grpo_ckpt_wgrad(dy, c, add=b, dW=b), a)


def test_wgrad_in_place_and_repeatable(clp):
    for n, out, d in ((3000, 264, 520), (700, 1024, 1536)):
        got, c, dy = run_wgrad(clp, n, out, d, add=False, seed=7)
        again = clp.grpo_ckpt_wgrad(dy, c)
        assert torch.equal(got, again)
        acc = torch.ones_like(got)
        want = clp.grpo_ckpt_wgrad(dy, c, add=torch.ones_like(got))
        clp.grpo_ckpt_wgrad(dy, c, add=acc, dW=acc)
        assert torch.equal(acc, want)


def test_wgrad_exponents_of_every_size(clp):
    # Blocks from 2^-100 to 2^100: each of them is widened exactly, whichever
    # way its exponent takes on chip, with blocks of zeros among them.
    g = torch.Generator().manual_seed(3)
    n, out, d = 130, 24, 1024
    size = torch.randint(-100, 101, (n, d // 32), generator=g).double()
    size[5], size[:, 7] = -130, -140  # below the smallest exponent: zeros
    x = (torch.randn(n, d, generator=g).double() * torch.exp2(size).repeat_interleave(32, 1)).bfloat16()
    dy = torch.zeros(n, out, dtype=torch.bfloat16)
    dy[torch.arange(n), torch.arange(n) % out] = 1.0  # few terms in each sum
    c = clp.grpo_ckpt_pack(x.to(DEV))
    got = clp.grpo_ckpt_wgrad(dy.to(DEV), c)
    q, ex = o.ckpt_pack(f64(x), float(torch.finfo(torch.bfloat16).max))
    x64 = o.ckpt_expand(q, ex)
    mag = np.abs(f64(dy)).T @ np.abs(x64)
    check("dW", got, f64(dy).T @ x64, 8 * 2 * E * mag)  # 6 terms


def test_wgrad_repeats_on_cold_inputs(clp):
    # 28 of the 256 tiles are cut, and their tokens come from memory late and out
    # of step: every launch gives the same bits.
    g = torch.Generator(device=DEV).manual_seed(11)
    x = torch.randn(16384, 4096, device=DEV, generator=g).bfloat16()
    dy = torch.randn(16384, 4096, device=DEV, generator=g).bfloat16()
    c = clp.grpo_ckpt_pack(x)
    cold = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    first = clp.grpo_ckpt_wgrad(dy, c)
    for _ in range(200):
        cold.zero_()
        assert torch.equal(clp.grpo_ckpt_wgrad(dy, c), first)


def test_wgrad_nan_reaches_only_its_columns(clp):
    x = rand(torch.Generator().manual_seed(0), 100, 64, torch.bfloat16).to(DEV)
    x[50, 9] = float("nan")
    dy = rand(torch.Generator().manual_seed(1), 100, 40, torch.bfloat16).to(DEV)
    dw = clp.grpo_ckpt_wgrad(dy, clp.grpo_ckpt_pack(x))
    assert torch.isnan(dw[:, 9]).all() and torch.isnan(dw).sum() == 40


# ----------------------------------------------------- streams, graphs, size ----


def _step(clp, x, r, w, dy):
    f = clp.grpo_norm_fwd(x, w, residual=r, want_ckpt=True)
    b = clp.grpo_norm_bwd(dy, f.ckpt, w, None, f.rstd, dres=dy)
    c = clp.grpo_ckpt_pack(f.y)
    dw = clp.grpo_ckpt_wgrad(b.dx, c)
    return [f.y, f.z, b.dx, b.dweight, dw, clp.grpo_ckpt_unpack(c)]


def test_side_stream_and_graph_give_the_same(clp):
    g = torch.Generator().manual_seed(2)
    x, r, dy = (rand(g, 300, 520, torch.bfloat16).to(DEV) for _ in range(3))
    w = torch.ones(520, dtype=torch.bfloat16, device=DEV)
    want = [t.clone() for t in _step(clp, x, r, w, dy)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _step(clp, x, r, w, dy)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _step(clp, x, r, w, dy)
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_offsets_beyond_32_bits(clp):
    # 2.2e9 values: the last rows lie past 2^31 elements and 2^32 bytes.
    n, d = 540_000, 4096
    x = torch.zeros(n, d, dtype=torch.bfloat16, device=DEV)
    tail = rand(torch.Generator().manual_seed(0), 64, d, torch.bfloat16).to(DEV)
    x[-64:] = tail
    w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    few = clp.grpo_norm_fwd(tail, w, residual=tail, want_ckpt=True)
    out = clp.grpo_norm_fwd(x, w, residual=x, want_ckpt=True)
    assert torch.equal(out.y[-64:], few.y) and torch.equal(out.z[-64:], few.z)
    assert torch.equal(out.ckpt.q[-64:].view(torch.uint8), few.ckpt.q.view(torch.uint8))
    assert torch.equal(out.ckpt.exponents[-64:], few.ckpt.exponents)
    grad = clp.grpo_norm_bwd(x, out.ckpt, w, None, out.rstd, dres=x, dx=out.y)
    gfew = clp.grpo_norm_bwd(tail, few.ckpt, w, None, few.rstd, dres=tail)
    assert torch.equal(grad.dx[-64:], gfew.dx)
    # rows of zeros add nothing, in whatever order the others are added
    np.testing.assert_allclose(f64(grad.dweight), f64(gfew.dweight), rtol=1e-4, atol=1e-4)
    back = clp.grpo_ckpt_unpack(out.ckpt, out=out.z)
    assert torch.equal(back[-64:], clp.grpo_ckpt_unpack(few.ckpt))
    dy = torch.zeros(n, 8, dtype=torch.bfloat16, device=DEV)
    dy[-64:] = 0.5
    got = clp.grpo_ckpt_wgrad(dy, out.ckpt)
    want = 0.5 * clp.grpo_ckpt_unpack(few.ckpt, torch.float32).double().sum(0)
    mag = 0.5 * clp.grpo_ckpt_unpack(few.ckpt, torch.float32).double().abs().sum(0)
    check("dW", got, f64(want)[None].repeat(8, 0), (64 + 1) * 2 * E * f64(mag)[None].repeat(8, 0))


def test_launches_are_timed(clp):
    x = torch.ones(4, 64, dtype=torch.bfloat16, device=DEV)
    clp.grpo_launch_timing_enable(True)
    _step(clp, x, x, torch.ones(64, dtype=torch.bfloat16, device=DEV), x)
    clp.grpo_launch_timing_enable(False)
    names = {k["name"] for k in clp.grpo_launch_timing_read()}
    assert {"norm_fwd_kernel", "norm_bwd_kernel", "norm_bwd_finish_kernel", "ckpt_pack_kernel",
            "ckpt_unpack_kernel"} <= names
    assert any(k.startswith("ckpt_wgrad") for k in names)
