"""CPU pins of the fp64 oracle of the norms and the 8-bit checkpoint."""

import math

import numpy as np
import pytest
import torch

from oracle import norm_ckpt_oracle as o

ALL_E4M3 = np.array([(-1) ** s * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
                     for s in (0, 1) for e in range(16) for m in range(8)
                     if not (e == 15 and m == 7)])


def test_e4m3_keeps_its_own_values():
    np.testing.assert_array_equal(o.e4m3(ALL_E4M3), ALL_E4M3)


def test_e4m3_is_the_nearest_value_with_ties_to_even():
    pos = np.sort(ALL_E4M3[:127])
    mid = (pos[1:] + pos[:-1]) / 2
    got = o.e4m3(mid)
    want = np.where(np.arange(len(mid)) % 2 == 0, pos[:-1], pos[1:])  # even bit patterns
    np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(o.e4m3(np.nextafter(mid, 0)), pos[:-1])
    np.testing.assert_array_equal(o.e4m3(np.nextafter(mid, 1e9)), pos[1:])


def test_e4m3_agrees_with_torch():
    v = np.random.default_rng(0).normal(size=20000).astype(np.float32) * 40
    v = np.clip(v, -448, 448)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(o.e4m3(v), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_ckpt_error_and_range(dtype):
    g = torch.Generator().manual_seed(1)
    top = float(torch.finfo(dtype).max)
    x = torch.randn(64, 70, generator=g) * torch.exp(6 * torch.randn(64, 1, generator=g))
    x = x.clamp(-top, top).to(dtype)  # finite in every type
    x[0, 0], x[1, 40], x[2, 69] = top, -top, torch.finfo(dtype).tiny
    x[3] = 0
    xd = x.double().numpy()
    q, ex = o.ckpt_pack(xd, top)
    assert np.abs(q).max() <= 448 and ex.min() >= 10 and ex.max() <= 247
    back = o.ckpt_expand(q, ex)
    assert np.abs(back).max() <= top
    unit = np.ldexp(1.0, np.repeat(ex - 127, 32, axis=1)[:, :70])
    bound = np.maximum(np.abs(xd) * 2.0 ** -4, unit * 2.0 ** -10)
    held = np.abs(back) == 240 * unit  # values that would have left the type
    ok = np.abs(back - xd) <= bound
    assert np.all(ok | (held & (np.abs(xd) > 248 * unit)))
    # every value is a normal bf16 (or zero)
    b = torch.from_numpy(back).to(torch.bfloat16)
    np.testing.assert_array_equal(b.double().numpy(), back)
    nz = np.abs(back[back != 0])
    assert nz.min() >= 2.0 ** -126


def test_ckpt_largest_value_is_kept_within_half_a_step():
    # 1.75 2^e sits exactly on 448; the next value needs the larger unit.
    for a, k in ((448.0, 0), (np.nextafter(448.0, 500), 1), (1.0, -8), (1.75, -8), (1.751, -7)):
        _, ex = o.ckpt_pack(np.array([[a, 0.0]]), 3e38)
        assert ex[0, 0] - 127 == k, (a, ex)


def test_ckpt_special_values_and_mask():
    x = np.array([[1.0, np.inf, np.nan, -np.inf, 0.5] + [0.25] * 30])
    q, ex = o.ckpt_pack(x, 3e38)
    assert np.isnan(q[0, 1:4]).all() and q[0, 0] == 256 and ex[0, 0] == 127 - 8
    q, ex = o.ckpt_pack(x, 3e38, mask=[0])
    assert (q == 0).all() and (ex == 10).all()


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_forward_by_hand(kind):
    z = np.array([[1.0, 2.0, 4.0, -3.0]])
    y, mean, rstd = o.norm_fwd(z, [1, 2, 1, 1], [0, 0, 1, 0], kind, 0.5)
    mu = 1.0 if kind == "layer" else 0.0
    var = math.fsum((v - mu) ** 2 for v in z[0]) / 4
    r = 1 / math.sqrt(var + 0.5)
    want = [(1 - mu) * r, (2 - mu) * r * 2, (4 - mu) * r + 1, (-3 - mu) * r]
    np.testing.assert_allclose(y[0], want, rtol=1e-15)
    assert mean[0] == mu and abs(rstd[0] - r) < 1e-15


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("d", [1, 2, 7, 33])
def test_norm_backward_against_differences(kind, d):
    rng = np.random.default_rng(d)
    n, eps = 3, 1e-3
    z, dy = rng.normal(size=(n, d)), rng.normal(size=(n, d))
    w, b = 1 + 0.3 * rng.normal(size=d), rng.normal(size=d)
    dres = rng.normal(size=(n, d))

    def value(z, w, b):
        y, _, _ = o.norm_fwd(z, w, b, kind, eps)
        return float((y * dy).sum() + (z * dres).sum())

    _, mean, rstd = o.norm_fwd(z, w, b, kind, eps)
    dx, dw, db = o.norm_bwd(dy, z, w, mean, rstd, kind, dres=dres)
    # Central differences: cancellation 2^-52 |value| / step (about 1e-9), and
    # step^2 f''' / 6, f''' up to about (1 / sd)^3 |dy| <= 1e4 at d = 2.
    step, tol = 1e-5, 1e-6
    for i in range(n):
        for j in range(d):
            p, m = z.copy(), z.copy()
            p[i, j] += step
            m[i, j] -= step
            num = (value(p, w, b) - value(m, w, b)) / (2 * step)
            assert abs(num - dx[i, j]) <= tol
    for j in range(d):
        e = np.zeros(d)
        e[j] = step
        assert abs((value(z, w + e, b) - value(z, w - e, b)) / (2 * step) - dw[j]) <= tol
        assert abs((value(z, w, b + e) - value(z, w, b - e)) / (2 * step) - db[j]) <= tol


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_backward_against_autograd(kind):
    rng = np.random.default_rng(5)
    z = torch.from_numpy(rng.normal(size=(4, 19))).requires_grad_()
    w = torch.from_numpy(rng.normal(size=19)).requires_grad_()
    b = torch.from_numpy(rng.normal(size=19)).requires_grad_()
    dy = torch.from_numpy(rng.normal(size=(4, 19)))
    if kind == "layer":
        y = torch.nn.functional.layer_norm(z, (19,), w, b, 1e-5)
    else:
        y = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + 1e-5) * w + b
    y.backward(dy)
    _, mean, rstd = o.norm_fwd(z.detach().numpy(), None, None, kind, 1e-5)
    dx, dw, db = o.norm_bwd(dy.numpy(), z.detach().numpy(), w.detach().numpy(), mean, rstd, kind)
    np.testing.assert_allclose(dx, z.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(dw, w.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(db, b.grad.numpy(), rtol=1e-10, atol=1e-12)


def test_masked_rows_are_not_read():
    z = np.random.default_rng(0).normal(size=(3, 5))
    z[1] = np.nan
    y, mean, rstd = o.norm_fwd(z, None, None, "layer", 1e-5, mask=[1, 0, 1])
    assert np.isfinite(y).all() and (y[1] == 0).all() and rstd[1] == 0
    dx, dw, _ = o.norm_bwd(z, z, None, mean, rstd, "layer", mask=[1, 0, 1])
    assert np.isfinite(dx).all() and (dx[1] == 0).all() and np.isfinite(dw).all()


def test_a_planted_mistake_shows():
    # A backward that forgets the mean(u h) term is not the gradient.
    rng = np.random.default_rng(2)
    z, dy = rng.normal(size=(2, 9)), rng.normal(size=(2, 9))
    _, mean, rstd = o.norm_fwd(z, None, None, "rms", 1e-5)
    dx, _, _ = o.norm_bwd(dy, z, None, None, rstd, "rms")
    assert np.abs(dx - dy * rstd[:, None]).max() > 1e-2


def test_wgrad_is_the_sum_over_tokens():
    rng = np.random.default_rng(3)
    dy, x, add = rng.normal(size=(5, 2)), rng.normal(size=(5, 3)), rng.normal(size=(2, 3))
    want = [[add[i, j] + math.fsum(dy[t, i] * x[t, j] for t in range(5)) for j in range(3)]
            for i in range(2)]
    np.testing.assert_allclose(o.wgrad(dy, x, add), want, rtol=1e-14)
