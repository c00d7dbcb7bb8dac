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


# lr decay = 1.5 2^-24, which 1 - lr decay as an fp32 takes for 2^-24 or 2^-23.
FADE_LR, FADE = 1e-5, 1.5e5 * 2.0 ** -24


def _faded(p0):
    """The values after a step without gradients, in fp64."""
    return p0 * (1 - float(np.float32(FADE_LR)) * float(np.float32(FADE)))


@pytest.mark.parametrize("bits", [8, 32])
def test_a_small_decay_is_the_one_that_was_asked(clp, bits):
    # p in [1, 2) is faded by 0.75 to 1.5 of its spacing; with no step beside it, the sum
    # is rounded once: half a spacing, 2^-24. lr decay itself is off by 2^-24 of itself,
    # and its product with p: 4 2^-24 of 3 2^-24.
    n = 100_000
    p = 1 + torch.rand(n, generator=torch.Generator().manual_seed(3))
    p0 = f64(p)
    p = p.to(DEV)
    opt = clp.AdamW([p], lr=FADE_LR, weight_decay=FADE, state_bits=bits)
    opt.step([torch.zeros(n, device=DEV)])
    assert (np.abs(f64(p) - _faded(p0)) <= 2.0 ** -24 * (1 + 12 * 2.0 ** -24)).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_a_small_decay_beside_a_step(clp, bits):
    # Steps of every size below lr: the sums' roundings are even over a spacing, so their
    # mean over n values is 2^-23 / sqrt(12 n) at one sigma; six of them are 6e-10. The
    # step's own error, 16 2^-24 of at most 4e-5 and of either sign, is far below. The decay
    # taken for 2^-24 or 2^-23 would move the mean by 4e-8.
    n = 1 << 17
    g = torch.Generator().manual_seed(5)
    p = (1 + torch.rand(n, generator=g)).to(DEV)
    m, v = torch.randn(n, generator=g), 0.1 + torch.rand(n, generator=g)
    gr = torch.randn(n, generator=g)
    if bits == 8:
        state = clp.alloc_adam_state(p, 8)
        state.m.copy_((100 * m).to(state.m.dtype))
        state.v.copy_((100 * v).to(state.v.dtype))
        for z in (state.m_scale, state.v_scale):
            z.fill_(0.01)
    else:
        state = clp.AdamState(m.to(DEV), v.to(DEV))
    p0, m0, v0 = f64(p), *map(f64, state.moments())
    opt = clp.AdamW([p], lr=FADE_LR, weight_decay=FADE, states=[state], steps_done=4)
    opt.step([gr.to(DEV)])
    want, _, _ = o.adamw(p0, f64(gr), m0, v0, 5, float(np.float32(FADE_LR)),
                         decay=float(np.float32(FADE)))
    off = f64(p) - want
    assert np.abs(off).max() <= 2.0 ** -24 + 16 * 2.0 ** -24 * 4e-4
    assert abs(off.mean()) <= 6e-10


@pytest.mark.parametrize("bits", [8, 32])
def test_a_small_decay_of_bf16_parameters(clp, bits):
    # 127 values in (1, 2), each of which has one nearest fp32 for its faded value (none
    # is within 2^-20 of a spacing of the middle between two, 12 2^-24 would do); of that
    # the 16 random bits make a bf16.
    n = 1 << 24
    p = (1 + torch.rand(n, generator=torch.Generator().manual_seed(7))).clamp(1.01, 1.99).to(BF)
    want = _faded(f64(p))
    p = p.to(DEV)
    opt = clp.AdamW([p], lr=FADE_LR, weight_decay=FADE, state_bits=bits, seed=21)
    opt.step([torch.zeros(n, dtype=BF, device=DEV)])
    part = want * 2.0 ** 23 % 1.0
    assert want.min() > 1 and (np.abs(part - 0.5) > 2.0 ** -20).all()
    _, _, u = o.random_bits(np.arange(n), 21, 1)
    raised = want.astype(np.float32).view(np.uint32) + u.astype(np.uint32)
    want = (raised & np.uint32(0xFFFF0000)).view(np.float32)
    assert (p.float().cpu().numpy() == want).all()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("t", [F32, BF])
def test_infinite_parameters_stay_and_their_neighbours_step(clp, bits, t):
    g = torch.Generator().manual_seed(9)
    p = torch.randn(1000, generator=g).to(DEV, t)
    gr = torch.randn(1000, generator=g).to(DEV)
    q = p.clone()
    at = torch.tensor([3, 8, 700], device=DEV)
    bad = torch.tensor([float("inf"), float("-inf"), float("nan")], dtype=t, device=DEV)
    q[at] = bad
    for x in (p, q):
        opt = clp.AdamW([x], lr=1e-3, state_bits=bits, weight_decay=0.1, seed=2)
        for _ in range(2):
            opt.step([gr])
    assert torch.equal(q[at][:2], bad[:2]) and torch.isnan(q[700])
    p[at] = q[at] = 0
    assert torch.equal(p, q)


def _norm64(grads):
    return torch.stack([x.double().square().sum() for x in grads]).sum().sqrt().item()


# A rounding to fp32, 2^-24, and a last bit more for what is before it: the parts that the
# sums leave (2^-24 of them is lost of each of some 2^9 squares a thread) and fp64 sums.
LAST_BIT = 1.01 * 2.0 ** -24


@pytest.mark.parametrize("t", [F32, BF, HF])
@pytest.mark.parametrize("kind", ["even", "random"])
def test_the_norm_of_long_tensors_to_the_last_bit(clp, t, kind):
    # Several chunks of 16384 values for each of the 1216 CTAs: 512 squares a thread, whose
    # plain fp32 sums of values of one size would be off by some 2^-24 each time.
    n = 8 * 1216 * 16384 + 12345
    x = torch.full((n,), 0.37, device=DEV, dtype=t)
    if kind == "random":
        x.mul_(torch.rand(n, generator=torch.Generator(DEV).manual_seed(1), device=DEV))
    want = _norm64([x])
    got = clp.grpo_grad_norm([x]).norm.item()
    assert abs(got - want) <= LAST_BIT * want


@pytest.mark.parametrize("t", [F32, BF])
@pytest.mark.parametrize("size", [1e-44, 1e-38, 1e-30, 1e-24, 1e-22, 1e-19, 1e-16, 1e-15, 1e-14,
                                  1e14, 2e15, 1e18, 1.7e19])
def test_the_norm_of_very_small_and_very_large_gradients(clp, t, size):
    g = torch.Generator(DEV).manual_seed(2)
    for n in (1, 1001, 16384, 400_003):
        x = (size * (0.5 + 0.5 * torch.rand(n, generator=g, device=DEV, dtype=torch.float64))).to(t)
        y = torch.randn(n, generator=g, device=DEV).to(t)  # beside usual ones
        for grads in ([x], [x, y], [torch.cat([x, y])], [torch.stack([x, y], 1).reshape(-1)]):
            want = _norm64(grads)
            got = clp.grpo_grad_norm(grads).norm.item()
            if want < 2.0 ** -126:  # subnormals are 2^-149 apart
                assert abs(got - want) <= 1.01 * 2.0 ** -150
            else:
                assert abs(got - want) <= LAST_BIT * want
            r = clp.grpo_grad_norm(grads, max_norm=0.1)
            assert abs(r.scale.item() - min(1.0, 0.1 / (want + 1e-6))) <= LAST_BIT * r.scale.item()


def test_the_norm_of_zeros_and_of_what_is_not_finite(clp):
    for t in (F32, BF, HF):
        x = torch.zeros(100_000, device=DEV, dtype=t)
        assert clp.grpo_grad_norm([x]).norm.item() == 0.0
        for bad, is_nan in ((float("inf"), False), (float("-inf"), False), (float("nan"), True)):
            for at in (0, 99_999):
                x.fill_(0.25)
                x[at] = bad
                r = clp.grpo_grad_norm([x], max_norm=1.0)
                assert torch.isnan(r.norm) if is_nan else r.norm.item() == float("inf")
                assert torch.isnan(r.scale)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("eps", [1e-300, 1e-45, 1e-40, 1e-38])
def test_an_eps_above_zero_however_small(clp, bits, eps):
    # Values without a gradient so far have no step: 0 / eps. The others' is lr.
    p = torch.ones(300, device=DEV)
    gr = torch.zeros(300, device=DEV)
    gr[::3] = 0.5
    opt = clp.AdamW([p], lr=0.25, eps=eps, weight_decay=0.0, state_bits=bits)
    opt.step([gr])
    assert (p[gr == 0] == 1).all()
    assert ((p[::3] - 0.75).abs() <= 8 * 2.0 ** -24).all()


@pytest.mark.parametrize("gt", [F32, BF, HF])
@pytest.mark.parametrize("off", [0, 1])
def test_bf16_parameters_with_moments_in_32_bits(clp, gt, off):
    # Moments against fp64 as for fp32 parameters; the parameter goes where its 16 random
    # bits send the fp32 sum, which is within a few units of 2^-24 of the exact one.
    sizes = [1, 7, 128, 129, 255, 257, 1000, 4096, 4097, 40_003]
    g = torch.Generator().manual_seed(11)

    def made(t, scale=1.0):
        out = []
        for n in sizes:
            big = (scale * torch.randn(n + off, generator=g)).to(t).to(DEV)
            out.append(big[off:])
        return out

    lr, decay, seed = 3e-3, 0.1, 77
    params = made(BF)
    states = [clp.AdamState(m, v.abs()) for m, v in zip(made(F32, 0.1), made(F32, 0.02))]
    opt = clp.AdamW(params, lr=lr, weight_decay=decay, states=states, steps_done=3, seed=seed)
    lr = float(np.float32(lr))
    for t in (4, 5):
        grads = made(gt, 0.1)
        before = [(f64(p), f64(s.m), f64(s.v)) for p, s in zip(params, states)]
        opt.step(grads)
        at = 0
        for (p0, m0, v0), p, gr, s in zip(before, params, grads, states):
            q = f64(gr)
            p1, m1, v1 = o.adamw(p0, q, m0, v0, t, lr, decay=decay)
            # Two products and a sum each, beta's complements as fp32.
            dm, dv = 4 * 2.0 ** -24 * (np.abs(m0) + np.abs(q)), 4 * 2.0 ** -24 * (v0 + q ** 2)
            assert (np.abs(f64(s.m) - m1) <= dm).all()
            assert (np.abs(f64(s.v) - v1) <= dv + 1e-45).all()
            root = np.sqrt(v1 / (1 - 0.999 ** t)) + 1e-8
            scale = lr / (1 - 0.9 ** t) / root
            near = scale * dm + np.abs(scale * m1) * 16 * 2.0 ** -24 + 2.0 ** -23 * np.abs(p1)
            _, _, u = o.random_bits(np.arange(at, at + p0.size), seed, t)
            at += -(-p0.size // 128) * 128
            step = 2.0 ** (np.floor(np.log2(np.abs(p1))) - 7)
            raised = np.abs(p1) / step + u / 65536
            want = np.sign(p1) * np.floor(raised) * step
            clear = np.abs(raised - np.round(raised)) * step > near
            # The power of two above p1 may be the sum's own.
            clear &= np.abs(np.abs(p1) / step - 128) * step > near
            assert (f64(p) == want)[clear].all() and clear.mean() > 0.99 - 3 / p0.size
            assert (np.abs(f64(p) - p1) <= step + near).all()
