"""CPU pins of the fp64 oracle of the gated block and the optimizer."""

import math

import numpy as np
import pytest
import torch

from oracle import block_oracle as o

ACTS = ["silu", "gelu", "gelu_tanh", "relu"]


@pytest.mark.parametrize("name", ACTS)
def test_activation_is_torchs_and_its_slope_the_difference_quotient(name):
    g = np.linspace(-9, 9, 181) + 0.0123
    f = {"silu": torch.nn.functional.silu, "relu": torch.nn.functional.relu,
         "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda x: torch.nn.functional.gelu(x, approximate="tanh")}[name]
    a, s = o.act(name, g)
    assert np.abs(a - f(torch.from_numpy(g)).numpy()).max() < 1e-14
    e = 1e-6  # central difference: e^2 / 6 of the third derivative, and 1e-16 / e
    d = (o.act(name, g + e)[0] - o.act(name, g - e)[0]) / (2 * e)
    assert np.abs(s - d).max() < 1e-8


@pytest.mark.parametrize("name", ACTS)
def test_block_gradients_are_autograds(name):
    r = np.random.default_rng(0)
    x, wg, wu = r.standard_normal((5, 8)), r.standard_normal((12, 8)), r.standard_normal((12, 8))
    dh = r.standard_normal((5, 12))
    t = [torch.from_numpy(z).requires_grad_() for z in (x, wg, wu)]
    f = {"silu": torch.nn.functional.silu, "relu": torch.nn.functional.relu,
         "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[name]
    h = f(t[0] @ t[1].T) * (t[0] @ t[2].T)
    h.backward(torch.from_numpy(dh))
    oh, g, u = o.glu_fwd(x, wg, wu, name)
    dg, du, h2 = o.glu_bwd(dh, g, u, name)
    for got, want in ((oh, h.detach()), (h2, h.detach()), (dg @ wg + du @ wu, t[0].grad),
                      (dg.T @ x, t[1].grad), (du.T @ x, t[2].grad)):
        assert np.abs(got - want.numpy()).max() < 1e-12


def test_adamw_is_torchs():
    r = np.random.default_rng(1)
    p = torch.from_numpy(r.standard_normal(50)).requires_grad_()
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = r.standard_normal(50)
        p.grad = torch.from_numpy(g)
        opt.step()
        q, m, v = o.adamw(q, g, m, v, t, 1e-2, (0.8, 0.95), 1e-6, 0.1)
        assert np.abs(q - p.detach().numpy()).max() < 1e-14


def test_e4m3_table_is_torchs():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(o.e4m3_values(), codes.double().numpy())


def test_random_bits_are_even_and_unrelated():
    # 2^20 places: the mean of 16 uniform bits is off by 65536 / sqrt(12 n) = 18.5 at
    # one sigma, a correlation by 1e-3; six sigma of each.
    n = 1 << 20
    at = np.arange(n)
    words = [w for seed, step in ((0, 1), (0, 2), (1, 1), (1 << 40, 1), (0, 1 << 33))
             for w in o.random_bits(at, seed, step)]
    words += [o.random_bits(at + far, 0, 1)[0] for far in (1 << 32, 1 << 33, 5 << 32)]
    for w in words:
        assert abs(w.mean() - 32767.5) < 6 * 18.5
        assert w.min() < 16 and w.max() > 65519
        assert abs(np.corrcoef(w[:-1], w[1:])[0, 1]) < 6e-3
        counts = np.bincount((w / 256).astype(int), minlength=256)  # 4096 each, sigma 64
        assert np.abs(counts - 4096).max() < 6 * 64
    c = np.corrcoef(words)
    assert np.abs(c - np.eye(len(words))).max() < 6e-3


def test_rounding_at_random_is_right_in_the_mean():
    # A value between neighbours a sixteenth apart, over 2^16 u's: exactly the share.
    u = np.arange(65536.0)
    grid = o.e4m3_values()
    for x in (300.0, 1.03, 0.007, 0.0009):
        y = np.full(65536, x)
        y[0] = TOP = 448.0  # keeps the scale at 1
        for power in (1, 2):
            code, _, _, s = o.to_8(np.where(np.arange(65536) % 128 == 0, TOP, x), power, u)
            live = np.arange(65536) % 128 != 0
            assert np.all(s == 1.0)
            mean = (grid[code[live] & 0x7F] ** power).mean()
            # Only every 128th u is left out, and the smallest v is held at 2^-9.
            if power == 1 or x > 2 ** -9:
                assert abs(mean / x ** power - 1) < 2e-3
    assert math.isclose(grid[126], 448.0)
