"""GPU: the AdamW step and the gradients' norm against their formulas in fp64."""

import numpy as np
import pytest
import torch

from oracle import block_oracle as o

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def clp():
    __import__("__graft_entry__").build()
    import chunked_log_prob_gb300 as m

    return m


def f64(t):
    return t.detach().cpu().double().numpy().reshape(-1)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# Sizes about the groups of 128 and 256, odd ones, one beyond a chunk.
SIZES = [1, 7, 127, 128, 129, 255, 256, 257, 1000, 2048, 2049, 16384, 40003]


def _tensors(g, sizes, t=F32, scale=1.0):
    return [(scale * torch.randn(n, generator=g)).to(t).to(DEV) for n in sizes]


def _places(sizes):
    at, out = 0, []
    for n in sizes:
        out.append(np.arange(at, at + n))
        at += -(-n // 128) * 128
    return out


LR, DECAY = 3e-3, 0.1


def _fp32_step(p0, g, m0, v0, t, decay, scale=1.0, betas=(0.9, 0.999), eps=1e-8, lr=LR):
    """fp64 values after the step, and how far an fp32 one may be from them: a few
    units of 2^-24 of each term."""
    p, m, v = o.adamw(p0, g, m0, v0, t, lr, betas, eps, decay, scale)
    dm = 4 * 2.0 ** -24 * (np.abs(m0) + np.abs(g * scale))
    dv = 4 * 2.0 ** -24 * (v0 + (g * scale) ** 2)
    # m's error over the root, v's half of its relative one, and some ten operations
    root = np.sqrt(v / (1 - betas[1] ** t)) + eps
    step = np.abs(lr * m / (1 - betas[0] ** t) / root)
    # 1 - lr decay is off by 2^-25, its product with p and the difference by 2^-24 of p
    # each: 2.5 2^-24 of p, and lr itself is an fp32.
    dp = lr * dm / (1 - betas[0] ** t) / root + step * 16 * 2.0 ** -24 + 3 * 2.0 ** -24 * np.abs(p0)
    return (p, m, v), (dp, dm, dv)


@pytest.mark.parametrize("gt", [F32, BF, HF])
@pytest.mark.parametrize("ct", [None, BF, HF])
def test_moments_in_32_bits(clp, gt, ct):
    g = _gen(0)
    params = _tensors(g, SIZES)
    copies = None if ct is None else [torch.zeros(n, dtype=ct, device=DEV) for n in SIZES]
    decay = [DECAY if i % 2 else 0.0 for i in range(len(SIZES))]
    opt = clp.AdamW(params, lr=LR, weight_decay=decay, copies=copies)
    want = [(f64(p), np.zeros(p.numel()), np.zeros(p.numel())) for p in params]
    for t in (1, 2, 3):
        grads = _tensors(g, SIZES, gt, 0.1)
        opt.step(grads)
        for i, (p, gr, s) in enumerate(zip(params, grads, opt.states)):
            new, tol = _fp32_step(want[i][0], f64(gr), want[i][1], want[i][2], t, decay[i])
            for got, w, d in zip((p, s.m, s.v), new, tol):
                assert (np.abs(f64(got) - w) <= d + 1e-45).all()
            want[i] = tuple(f64(z) for z in (p, s.m, s.v))  # on from the stored ones
            if copies is not None:
                assert torch.equal(copies[i], p.to(ct))
    assert opt.steps_done == 3


def _state_8(clp, g, sizes, scale=0.1):
    """Moments in 8 bits as an earlier step may have left them."""
    out = []
    for n in sizes:
        q = [(100 * torch.randn(n, generator=g)).to(E4M3).to(DEV),
             (20 + 100 * torch.rand(n, generator=g)).to(E4M3).to(DEV)]
        s = [(scale / 448 * (0.5 + torch.rand(-(-n // 128), generator=g))).to(DEV) for _ in range(2)]
        out.append(clp.AdamState(q[0], q[1], s[0], s[1]))
    return out


def _check_8(code, scale, y, power, u, err, slack=1e-4):
    """Codes of a moment y that the kernel knows to `err` of itself: the neighbour that
    u picks, or, with u that near the chance, either."""
    want, chance, lo, s = o.to_8(y, power, u)
    assert np.allclose(f64(scale), s, rtol=err + 1e-6, atol=1e-44)
    code = code.view(torch.uint8).cpu().numpy().reshape(-1).astype(int)
    near = np.abs(u / 65536 - chance) < slack
    # At a neighbour itself (chance 0 or 1) both sides' lower neighbours may differ.
    near |= (chance < slack) | (chance > 1 - slack)
    assert (code == want)[~near].all()
    assert (np.abs((code & 0x7F) - (want & 0x7F)) <= 1).all()
    sign = (code & 0x7F) != 0
    assert ((code & 0x80) == (want & 0x80))[sign].all()


@pytest.mark.parametrize("pt", [F32, BF])
@pytest.mark.parametrize("gt", [F32, BF, HF])
def test_moments_in_8_bits(clp, pt, gt):
    g = _gen(1)
    params, grads = _tensors(g, SIZES, pt), _tensors(g, SIZES, gt, 0.3)
    states = _state_8(clp, g, SIZES)
    before = [(f64(p), *map(f64, s.moments())) for p, s in zip(params, states)]
    seed, t = 0x123456789ABC, 7
    opt = clp.AdamW(params, lr=LR, weight_decay=DECAY, states=states, steps_done=t - 1, seed=seed)
    opt.step(grads)
    for (p0, m0, v0), p, gr, s, at in zip(before, params, grads, states, _places(SIZES)):
        (p1, m1, v1), (dp, _, _) = _fp32_step(p0, f64(gr), m0, v0, t, DECAY)
        um, uv, up = o.random_bits(at, seed, t)
        # m may cancel: known to units of its terms, not of itself.
        _check_8(s.m, s.m_scale, m1, 1, um, 1e-6, slack=2e-3)
        _check_8(s.v, s.v_scale, np.sqrt(v1), 2, uv, 1e-6)
        lost = np.isnan(p1)  # of moments that were NaN
        assert (np.isnan(f64(p)) == lost).all()
        if pt is F32:
            assert (np.abs(f64(p) - p1) <= dp + 1e-45)[~lost].all()
        else:
            step = 2.0 ** (np.floor(np.log2(np.abs(p1))) - 7)
            low = np.floor(np.abs(p1) / step) * step
            up_now = np.where(np.abs(p1) + up / 65536 * step >= low + step, low + step, low)
            want = np.sign(p1) * up_now
            near = np.abs((np.abs(p1) - low) / step + up / 65536 - 1) < 1e-3
            near |= (np.abs(p1) - low < 1e-3 * step) | (low + step - np.abs(p1) < 1e-3 * step)
            assert (f64(p) == want)[~near & ~lost].all()
            assert (np.abs(f64(p) - want) <= 1.001 * step)[~lost].all()


def test_values_off_16_bytes_are_the_same(clp):
    # The same tensors at addresses that no 16-byte load takes.
    g = _gen(2)
    sizes = [513, 4096, 1001]
    for bits, pt in ((32, F32), (8, F32), (8, BF)):
        base = _tensors(g, sizes, pt), _tensors(g, sizes, BF, 0.1)
        results = []
        for off in (0, 1):
            def moved(z):
                big = torch.zeros(z.numel() + 8, dtype=z.dtype, device=DEV)
                big[off:off + z.numel()] = z
                return big[off:off + z.numel()], big
            p, keep = zip(*[moved(z) for z in base[0]])
            gr = [moved(z)[0] for z in base[1]]
            opt = clp.AdamW(list(p), lr=LR, state_bits=bits, seed=5)
            for _ in range(3):
                opt.step(gr)
            results.append([z.clone() for z in p] + [m for s in opt.states for m in s.moments()])
            for z, n in zip(keep, sizes):
                rest = torch.cat([z[:off], z[off + n:]])
                assert not rest.any()  # nothing beyond the tensor
        for a, b in zip(*results):
            assert torch.equal(a, b)


def test_many_tensors_are_the_steps_of_each(clp):
    # Beyond one launch's table; empty ones and ones without a gradient among them.
    g = _gen(3)
    sizes = [int(n) for n in torch.randint(1, 700, (600,), generator=g)]
    sizes[5] = sizes[300] = 0
    params, grads = _tensors(g, sizes), _tensors(g, sizes, F32, 0.1)
    lrs = [1e-3 * (1 + i % 7) for i in range(600)]
    skip = {17, 256, 599}
    before = [p.clone() for p in params]
    opt = clp.AdamW(params, lr=lrs, weight_decay=0.0)
    opt.step([None if i in skip else q for i, q in enumerate(grads)])
    for i, (p, q, b) in enumerate(zip(params, grads, before)):
        if i in skip:
            assert torch.equal(p, b) and not opt.states[i].m.any()
        else:
            (w, _, _), (d, _, _) = _fp32_step(f64(b), f64(q), 0 * f64(b), 0 * f64(b), 1, 0.0,
                                              lr=float(np.float32(lrs[i])))
            assert (np.abs(f64(p) - w) <= d).all()


def test_random_rounding_does_not_lose_small_steps(clp):
    # bf16 weights of 1, whose neighbours are 2^-8 below and 2^-7 above; 64 steps of
    # -1e-4 (a fortieth of the spacing): the mean moves by 64e-4. Per weight the walk's
    # variance is at most 64 2^-8 1e-4, over 2^16 weights six sigma is 1.2e-4.
    n = 1 << 16
    p = torch.ones(n, dtype=BF, device=DEV)
    opt = clp.AdamW([p], lr=1e-4, betas=(0.0, 0.0), eps=0.0, weight_decay=0.0, state_bits=8)
    gr = torch.full((n,), 0.5, device=DEV)
    for _ in range(64):
        opt.step([gr])
    assert abs(p.double().mean().item() - (1 - 64e-4)) < 1.2e-4
    # The second moment in 8 bits: from v = 1 with gradients of 0.9 towards 0.81, beside
    # one value a block that keeps the scale. After 200 steps of a thousandth, v = 0.81
    # + 0.19 0.999^200 = 0.9656; steps of the format there are an eighth of v, so the
    # walk's variance is at most 200 1.9e-4 / 8 = 5e-3 and six sigma of the mean of 2^16
    # values 1.7e-3.
    q = clp.AdamState(torch.zeros(n, device=DEV).to(E4M3), torch.full((n,), 256.0, device=DEV).to(E4M3),
                      torch.zeros(n // 128, device=DEV), torch.full((n // 128,), 1 / 256, device=DEV))
    p = torch.zeros(n, device=DEV)
    opt = clp.AdamW([p], lr=0.0, states=[q], weight_decay=0.0)
    gr = torch.full((n,), 0.9, device=DEV)
    gr[::128] = 1.0
    for _ in range(200):
        opt.step([gr])
    live = torch.arange(n, device=DEV) % 128 != 0
    v = q.moments()[1].double()[live].mean().item()
    assert abs(v - (0.81 + 0.19 * 0.999 ** 200)) < 1.7e-3


def test_what_is_not_finite(clp):
    g = _gen(4)
    for bits in (32, 8):
        p, gr = torch.randn(300, generator=g).to(DEV), torch.randn(300, generator=g).to(DEV)
        opt = clp.AdamW([p], lr=LR, state_bits=bits)
        opt.step([gr])
        keep = [p.clone()] + [z.clone() for z in opt.states[0].moments()]
        # A scale that is not finite: nothing changes.
        for bad in (float("nan"), float("inf")):
            opt.step([gr], scale=torch.tensor(bad, device=DEV))
            for a, b in zip([p, *opt.states[0].moments()], keep):
                assert torch.equal(a, b)
        # One bad gradient: its own value is lost, its neighbours are not.
        gr[7] = float("nan")
        gr[200] = float("inf")
        opt.step([gr])
        ok = torch.ones(300, dtype=torch.bool, device=DEV)
        ok[7] = ok[200] = False
        assert torch.isnan(p[7]) and torch.isfinite(p[ok]).all()
        for z in opt.states[0].moments():
            assert not torch.isfinite(z[7]) and torch.isfinite(z[ok]).all()


def test_tiny_and_zero_gradients(clp):
    for bits in (32, 8):
        p = torch.ones(256, device=DEV)
        opt = clp.AdamW([p], lr=LR, state_bits=bits, weight_decay=0.0)
        opt.step([torch.zeros(256, device=DEV)])
        assert (p == 1).all() and not opt.states[0].moments()[0].any()
        # One large value beside 1e-12 of it: v stays above 0 for those that have one,
        # so no step is larger than a first step's.
        gr = torch.full((256,), 1e-9, device=DEV)
        gr[0], gr[5] = 1e3, 0.0
        for _ in range(20):
            opt.step([gr])
        assert torch.isfinite(p).all() and p[5] == 1
        assert (1 - p).abs().max() <= 20 * 1.01 * LR * 10
        if bits == 8:
            v = opt.states[0].v.view(torch.uint8)
            assert (v[:5] > 0).all() and v[5] == 0


def test_step_and_rate_on_the_device(clp):
    g = _gen(6)
    shape = (37, 21)
    p0, gr = torch.randn(*shape, generator=g).to(DEV), torch.randn(*shape, generator=g).to(DEV)
    for bits in (32, 8):
        a, b = p0.clone(), p0.clone()
        eager = clp.AdamW([a], lr=LR, state_bits=bits, seed=3)
        count = torch.zeros(1, dtype=torch.int64, device=DEV)
        held = clp.AdamW([b], lr=LR, state_bits=bits, seed=3, step_tensor=count)
        factor = torch.ones(1, device=DEV)
        ws = torch.empty(clp.grpo_grad_norm_workspace_size(1), dtype=torch.uint8, device=DEV)
        clp.grpo_grad_norm([gr])  # the device's first call is not captured

        def step():
            count.add_(1)
            held.step([gr], scale=clp.grpo_grad_norm([gr], max_norm=1.0, workspace=ws).scale,
                      lr_factor=factor)

        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            step()
        for t in range(5):
            factor.fill_(1.0 / (1 + t))
            graph.replay()
            eager.step([gr], scale=clp.grpo_grad_norm([gr], max_norm=1.0).scale, lr=LR / (1 + t))
            torch.cuda.synchronize()
            # The corrections come from expm1 in fp32 here, from doubles there: a step
            # differs by some 1e-6 of itself, its sum by a unit of |p| < 8.
            assert (a - b).abs().max() <= 5 * (1e-6 * 10 * LR + 2.0 ** -21)
        assert count.item() == 5
        for x, y in zip(eager.states[0].moments(), held.states[0].moments()):
            assert torch.equal(x, y)


def test_shapes_gradients_and_exchanged_storage(clp):
    g = _gen(7)
    p = torch.nn.Parameter(torch.randn(5, 33, generator=g).to(DEV))
    opt = clp.AdamW([p], lr=LR, weight_decay=0.0)
    with pytest.raises(ValueError, match="shape"):
        opt.step([torch.zeros(33, 5, device=DEV)])
    with pytest.raises(ValueError, match="contiguous"):
        opt.step([torch.zeros(33, 5, device=DEV).t()])
    with pytest.raises(TypeError, match=r"grads\[0\]"):
        opt.step([torch.zeros(5, 33, device=DEV).double()])
    with pytest.raises(ValueError, match="expected 1 of them"):
        opt.step([])
    with pytest.raises(ValueError, match="scale"):
        opt.step([torch.zeros(5, 33, device=DEV)], scale=torch.zeros(2, device=DEV))
    assert opt.steps_done == 0
    p.grad = torch.randn(5, 33, generator=g).to(DEV)
    before = p.detach().clone()
    p.data = p.data.clone()  # elsewhere now
    opt.step()
    (w, _, _), (d, _, _) = _fp32_step(f64(before), f64(p.grad), 0 * f64(before), 0 * f64(before), 1, 0.0)
    assert (np.abs(f64(p) - w) <= d).all()
    p.data = p.data[:3]  # same place, fewer values
    with pytest.raises(ValueError, match="states m"):
        opt.step([torch.zeros(3, 33, device=DEV)])
    q = torch.zeros(4, 8, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        clp.AdamW([q.t()], lr=LR)
    with pytest.raises(TypeError, match="params"):
        clp.AdamW([q.half()], lr=LR)
    with pytest.raises(TypeError, match="copies"):
        clp.AdamW([q.to(BF)], lr=LR, copies=[q.to(BF)])
    with pytest.raises(ValueError, match="copies"):
        clp.AdamW([q], lr=LR, copies=[q[:2].to(BF)])
    with pytest.raises(ValueError, match="states"):
        clp.AdamW([q], lr=LR, states=[])
    with pytest.raises(ValueError, match="lr"):
        clp.AdamW([q], lr=[1.0, 2.0])
    r = torch.zeros(20, device=DEV)
    with pytest.raises(ValueError, match="overlap"):
        clp.AdamW([q, r, q], lr=LR)
    with pytest.raises(ValueError, match="overlap"):
        clp.AdamW([r[4:12], q, r[11:]], lr=LR)
    clp.AdamW([r[:4], r[4:4], r[4:]], lr=LR)
    with pytest.raises(ValueError, match="step_tensor"):
        clp.AdamW([q], lr=LR, step_tensor=torch.zeros(1, device=DEV))


@pytest.mark.parametrize("t", [F32, BF, HF])
def test_gradient_norm(clp, t):
    g = _gen(8)
    for sizes in ([1], [7, 1000], SIZES, [200_001], [33] * 1500):
        grads = _tensors(g, sizes, t)
        want = np.sqrt(sum((f64(x) ** 2).sum() for x in grads))
        r = clp.grpo_grad_norm(grads + [None], max_norm=0.5)
        # fp32 squares and sums of 32: (1 + 31) 2^-24 / 2 of the norm, and its rounding.
        assert abs(r.norm.item() - want) <= 20 * 2.0 ** -24 * want
        assert abs(r.scale.item() - min(1.0, 0.5 / (want + 1e-6))) <= 24 * 2.0 ** -24 * r.scale.item()
        assert clp.grpo_grad_norm(grads).scale.item() == 1.0
        off = [torch.cat([x[:1], x])[1:] for x in grads]  # off 16 bytes
        again = clp.grpo_grad_norm(off)
        assert abs(again.norm.item() - want) <= 20 * 2.0 ** -24 * want
        assert torch.equal(clp.grpo_grad_norm(grads).norm, r.norm)


def test_gradient_norm_that_is_none_or_not_finite(clp):
    out = torch.empty(2, device=DEV)
    r = clp.grpo_grad_norm([None, None], max_norm=1.0, out=out)
    assert r.norm.item() == 0.0 and r.scale.item() == 1.0
    r = clp.grpo_grad_norm([torch.empty(0, device=DEV), torch.zeros(5, device=DEV)], max_norm=1.0)
    assert r.norm.item() == 0.0 and r.scale.item() == 1.0
    for bad in (float("nan"), float("inf"), 1e20):
        x = torch.zeros(5000, device=DEV)
        x[4321] = bad
        r = clp.grpo_grad_norm([x], max_norm=1.0)
        assert not torch.isfinite(r.norm) and torch.isnan(r.scale)


def test_results_repeat(clp):
    g = _gen(9)
    sizes = [100_003, 5, 70_000]
    runs = []
    base, grads = _tensors(g, sizes, BF), _tensors(g, sizes, BF, 0.1)
    for _ in range(2):
        p = [x.clone() for x in base]
        opt = clp.AdamW(p, lr=LR, state_bits=8, seed=11)
        for _ in range(3):
            opt.step(grads, scale=clp.grpo_grad_norm(grads, max_norm=0.1).scale)
        runs.append(p + [z for s in opt.states for z in s.moments()])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_going_on_from_kept_states_is_the_same(clp):
    g = _gen(10)
    sizes = [1000, 257]
    base = _tensors(g, sizes)
    grads = [_tensors(g, sizes, F32, 0.1) for _ in range(4)]
    a, b = [x.clone() for x in base], [x.clone() for x in base]
    one = clp.AdamW(a, lr=LR, state_bits=8, seed=3)
    two = clp.AdamW(b, lr=LR, state_bits=8, seed=3)
    for x in grads[:2]:
        one.step(x)
        two.step(x)
    kept = [clp.AdamState(*(z.clone() for z in s)) for s in two.states]
    two = clp.AdamW(b, lr=LR, states=kept, steps_done=two.steps_done, seed=3)
    for x in grads[2:]:
        one.step(x)
        two.step(x)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    for s, t in zip(one.states, two.states):
        for p, q in zip(s.moments(), t.moments()):
            assert torch.equal(p, q)


def test_on_another_stream(clp):
    g = _gen(11)
    p, gr = torch.randn(50_000, generator=g).to(DEV), torch.randn(50_000, generator=g).to(DEV)
    q = p.clone()
    one, two = clp.AdamW([p], lr=LR), clp.AdamW([q], lr=LR)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        one.step([gr], scale=clp.grpo_grad_norm([gr], max_norm=1.0).scale)
        with torch.cuda.stream(side):
            two.step([gr], scale=clp.grpo_grad_norm([gr], max_norm=1.0).scale)
    torch.cuda.synchronize()
    assert torch.equal(p, q)


def test_places_beyond_32_bits(clp):
    # One tensor of 2^32 + 1000 bf16 values, its moments in 8 bits: the last 1300 values,
    # on both sides of the border, as the formulas have them there.
    n, k = (1 << 32) + 1000, 1300
    first = n - k
    first -= first % 128  # whole blocks
    p = torch.zeros(n, dtype=BF, device=DEV)
    gr = torch.zeros(n, dtype=BF, device=DEV)
    g = _gen(12)
    p[first:] = torch.randn(n - first, generator=g).to(DEV, BF)
    gr[first:] = (0.1 * torch.randn(n - first, generator=g)).to(DEV, BF)
    opt = clp.AdamW([p], lr=LR, weight_decay=0.0, state_bits=8, seed=9)
    before = f64(p[first:])
    opt.step([gr], scale=clp.grpo_grad_norm([gr]).scale)
    (p1, m1, v1), _ = _fp32_step(before, f64(gr[first:]), 0 * before, 0 * before, 1, 0.0)
    um, uv, up = o.random_bits(np.arange(first, n), 9, 1)
    s = opt.states[0]
    _check_8(s.m[first:], s.m_scale[first // 128:], m1, 1, um, 1e-6)
    _check_8(s.v[first:], s.v_scale[first // 128:], np.sqrt(v1), 2, uv, 1e-6)
    step = 2.0 ** (np.floor(np.log2(np.abs(p1))) - 7)
    low = np.floor(np.abs(p1) / step) * step
    part = (np.abs(p1) - low) / step
    want = np.sign(p1) * np.where(part + up / 65536 >= 1, low + step, low)
    clear = (np.abs(part + up / 65536 - 1) > 1e-3) & (part > 1e-3) & (part < 1 - 1e-3)
    assert (f64(p[first:]) == want)[clear].all() and clear.mean() > 0.9
    assert not p[:first].any() and not s.m.view(torch.uint8)[:first:4099].any()
