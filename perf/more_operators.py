"""Cases of the gated feed-forward block and the AdamW operators.

What a training step of a decoder has between the norms and the weights:

- ``glu_fwd``: h = act(x Wg^T) * (x Wu^T), optionally with the two projections kept;
- ``glu_bwd``: the gradients of the projections and of x (from the projections as
  they were kept, or computed again), optionally h again;
- ``glu_wgrad``: the gradients of both weights, optionally added to those so far;
- ``adamw``: one step over many tensors, moments in 32 or in 8 bits, optionally
  clipped by the norm of all gradients.

The moments in 8 bits: 128 consecutive values share an fp32 scale (largest / 448);
values are e4m3 of m / scale, and of sqrt(v) / scale. A value between two neighbours
lo < hi of the format goes to hi where u < (m - lo) / (hi - lo), for the second moment
u < (v - lo^2) / (hi^2 - lo^2); a v above 0 never becomes 0. bf16 weights are rounded
the same way. u comes from 16 bits of a hash of (seed, step, place of the value).
"""

import math
import random

import torch

own = False  # True: the framework's calls; False: the plain form

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 128  # values of a moment that share a scale; tensors begin on a multiple
TOP = 448.0  # the largest e4m3
LR, BETA1, BETA2, EPS, DECAY, MAX_NORM = 2e-5, 0.9, 0.999, 1e-8, 0.01, 0.1
STEPS_DONE = 99  # the runs are of a training under way
# Budget of a drawn case: products of a projection, values of the optimizer.
MOST_PRODUCTS = 16384 * 4096 * 14336
MOST_VALUES = 500_000_000


def listed():
    return [
        # One token of a rollout: the weights are read once, nothing else counts.
        dict(name="glu_fwd_decode", op="glu_fwd", n=1, d=4096, f=14336, dtype="bf16",
             act="silu", mask="none", gates=False),
        # A padded GRPO batch of 8 completions x 1024 slots at hidden size 1536, the
        # projections kept for the backward pass.
        dict(name="glu_fwd_padded", op="glu_fwd", n=8192, d=1536, f=8960, dtype="bf16",
             act="silu", mask="padded", gates=True),
        # The 16384-token batch at hidden size 4096, nothing kept.
        dict(name="glu_fwd_long", op="glu_fwd", n=16384, d=4096, f=14336, dtype="bf16",
             act="silu", mask="none", gates=False),
        # A few rows, widths that fill no tile, the other type and activation.
        dict(name="glu_bwd_odd", op="glu_bwd", n=257, d=520, f=1368, dtype="fp16",
             act="gelu_tanh", mask="none", source="kept", h=False),
        # The padded batch's backward pass from the projections kept.
        dict(name="glu_bwd_kept", op="glu_bwd", n=8192, d=1536, f=8960, dtype="bf16",
             act="silu", mask="padded", source="kept", h=False),
        # The long batch's, the projections and h computed again.
        dict(name="glu_bwd_again", op="glu_bwd", n=16384, d=4096, f=14336, dtype="bf16",
             act="silu", mask="none", source="again", h=True),
        # Weight gradients of the padded batch's valid tokens, added to those before.
        dict(name="glu_wgrad_ragged", op="glu_wgrad", n=5541, d=1536, f=8960, dtype="bf16",
             accumulate=True),
        # And of the long batch.
        dict(name="glu_wgrad_long", op="glu_wgrad", n=16384, d=4096, f=14336, dtype="bf16",
             accumulate=False),
        # Low-rank adapters of 28 layers: 392 small tensors.
        dict(name="adamw_adapters", op="adamw", sizes="adapters", count=28, d=1536, f=8960,
             pdtype="fp32", gdtype="fp32", bits=32, copy="none", clip=True),
        # A head, its norm and the layer below: fp32 weights, the model's bf16 copies
        # written on the way.
        dict(name="adamw_tail", op="adamw", sizes="tail", count=128256, d=4096, f=14336,
             pdtype="fp32", gdtype="fp32", bits=32, copy="bf16", clip=True),
        # Odd sizes, moments in 8 bits.
        dict(name="adamw_odd_8", op="adamw", sizes="random", count=41, d=3_000_000, f=7,
             pdtype="fp32", gdtype="fp16", bits=8, copy="none", clip=False),
        # Two decoder layers in pure bf16, moments in 8 bits.
        dict(name="adamw_layers_8", op="adamw", sizes="layers", count=2, d=4096, f=14336,
             pdtype="bf16", gdtype="bf16", bits=8, copy="none", clip=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["glu_fwd", "glu_fwd", "glu_bwd", "glu_bwd", "glu_wgrad", "adamw", "adamw"])
    if op == "adamw":
        pdtype = rng.choice(["fp32", "fp32", "bf16"])
        return dict(op=op, sizes="random", count=_log_int(rng, 1, 400),
                    d=_log_int(rng, 1000, MOST_VALUES), f=rng.randrange(1 << 20), pdtype=pdtype,
                    gdtype=rng.choice(["fp32", "bf16", "fp16"]), bits=rng.choice([8, 32]),
                    copy=rng.choice(["none", "bf16", "fp16"]) if pdtype == "fp32" else "none",
                    clip=rng.random() < 0.5)
    d = 8 * _log_int(rng, 1, 1024)
    f = 8 * _log_int(rng, 1, 2048)
    n = _log_int(rng, 1, max(1, min(16384, MOST_PRODUCTS // (d * f))))
    case = dict(op=op, n=n, d=d, f=f, dtype=rng.choice(["bf16", "bf16", "fp16"]))
    if op == "glu_wgrad":
        case["accumulate"] = rng.random() < 0.5
        return case
    case.update(act=rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]),
                mask=rng.choice(["none", "none", "padded"]))
    if op == "glu_fwd":
        case["gates"] = rng.random() < 0.5
    else:
        case.update(source=rng.choice(["kept", "again"]), h=rng.random() < 0.5)
    return case


def _lengths(case):
    """Valid slots of the batch's completions (1024 slots each), from the sizes alone."""
    n = case["n"]
    t = min(n, 1024)
    r = random.Random(n)
    return [min(r.randint(t // 4 + 1, t), n - at) for at in range(0, n, t)], t


def _sizes(case):
    """Values of each of the optimizer's tensors."""
    d, f, count = case["d"], case["f"], case["count"]
    if case["sizes"] == "adapters":  # rank 16, A and B of the seven projections of a layer
        pairs = [(d, d), (d, d // 6), (d, d // 6), (d, d), (d, f), (d, f), (f, d)]
        return [16 * side for _ in range(count) for pair in pairs for side in pair]
    if case["sizes"] == "tail":
        return [count * d, d, d * f]
    if case["sizes"] == "layers":
        return [d * d, d * d // 4, d * d // 4, d * d, d * f, d * f, f * d, d, d] * count
    r = random.Random(f)
    parts = [math.exp(r.uniform(0.0, 6.0)) for _ in range(count)]
    return [max(1, int(d * p / sum(parts))) for p in parts]


def _layout(case):
    """(sizes, where each tensor begins, the buffer's length)."""
    sizes = _sizes(case)
    at, begin = 0, []
    for n in sizes:
        begin.append(at)
        at += -(-n // BLOCK) * BLOCK
    return sizes, begin, at


def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        p, g = DTYPES[case["pdtype"]].itemsize, DTYPES[case["gdtype"]].itemsize
        state = 16.0 if case["bits"] == 32 else 2 * 2 * (1 + 4 / BLOCK)
        copy = 0 if case["copy"] == "none" else 2
        return {"bytes": n * (2 * p + g + state + copy), "flops": 16 * n}
    n, d, f = case["n"], case["d"], case["f"]
    if case["op"] == "glu_wgrad":
        return {"bytes": 2 * n * (2 * f + d) + 8 * f * d * (2 if case["accumulate"] else 1),
                "flops": 4 * n * d * f}
    valid = n if case["mask"] == "none" else sum(_lengths(case)[0])
    if case["op"] == "glu_fwd":
        outs = 3 if case["gates"] else 1
        return {"bytes": 2 * (valid * d + 2 * f * d + outs * n * f),
                "flops": 4 * valid * d * f}
    again = case["source"] == "again"
    reads = valid * f + (valid * d if again else 2 * valid * f) + 2 * f * d
    writes = n * f * (3 if case["h"] else 2) + n * d
    return {"bytes": 2 * (reads + writes), "flops": (8 if again else 4) * valid * d * f}


# ------------------------------------------------------------------ inputs ----


def _rows_mask(case, dev):
    """uint8 [n]: completions with trailing padding."""
    if case["mask"] == "none":
        return None
    lens, t = _lengths(case)
    pos = torch.arange(len(lens) * t, device=dev).reshape(len(lens), t)
    keep = (pos % t) < torch.tensor(lens, device=dev)[:, None]
    return keep.reshape(-1)[:case["n"]].to(torch.uint8).contiguous()


def _normed(n, d, g, dev):
    """Rows as a norm leaves them: a few channels far above the rest."""
    x = torch.randn(n, d, generator=g, device=dev)
    big = torch.randint(0, d, (max(1, d // 512),), generator=g, device=dev)
    x[:, big] *= 10.0
    return x


def _moments_8(m, v):
    """Moments (whole blocks) in 8 bits, as an earlier step may have left them."""
    out = []
    for y in (m, v.sqrt()):
        y = y.reshape(-1, BLOCK)
        scale = y.abs().amax(1) / TOP
        q = (y / scale.clamp_min(1e-30)[:, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
        out += [q.reshape(-1), scale]
    return out


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": case, "seed": seed}
    if case["op"] == "adamw":
        sizes, begin, total = _layout(case)
        s["sizes"], s["begin"], s["t"] = sizes, begin, STEPS_DONE
        keep = torch.zeros(total, dtype=torch.bool, device=dev)  # the rest lies between tensors
        for n, at in zip(sizes, begin):
            keep[at:at + n] = True
        s["p"] = (0.02 * torch.randn(total, generator=g, device=dev) * keep).to(
            DTYPES[case["pdtype"]])
        # Gradients of very different size from block to block.
        size = 1e-4 * torch.exp(1.5 * torch.randn(total // BLOCK, 1, generator=g, device=dev))
        noise = torch.randn(total // BLOCK, BLOCK, generator=g, device=dev) * size
        s["g"] = (noise.reshape(-1) * keep).to(DTYPES[case["gdtype"]])
        m = torch.randn(total // BLOCK, BLOCK, generator=g, device=dev) * (0.3 * size)
        v = torch.rand(total // BLOCK, BLOCK, generator=g, device=dev).add_(0.05) * size * size
        m, v = m.reshape(-1) * keep, v.reshape(-1) * keep
        del noise, size
        if case["bits"] == 32:
            s["m"], s["v"] = m, v
        else:
            s["m"], s["m_scale"], s["v"], s["v_scale"] = _moments_8(m, v)
        if case["copy"] != "none":
            s["copy"] = s["p"].to(DTYPES[case["copy"]])
        # Norm weights and other small tensors are not decayed.
        s["decay"] = [DECAY if n > 16384 else 0.0 for n in sizes]
        return s
    n, d, f, t = case["n"], case["d"], case["f"], DTYPES[case["dtype"]]
    x = _normed(n, d, g, dev).to(t)
    s["x"] = x
    if case["op"] == "glu_wgrad":
        for name in ("dgate", "dup"):
            s[name] = (1e-2 * torch.randn(n, f, generator=g, device=dev)).to(t)
        if case["accumulate"]:
            for name in ("add_gate", "add_up"):
                s[name] = 0.1 * torch.randn(f, d, generator=g, device=dev)
        return s
    for name in ("w_gate", "w_up"):
        s[name] = (torch.randn(f, d, generator=g, device=dev) / d ** 0.5).to(t)
    s["mask"] = _rows_mask(case, dev)
    if case["op"] == "glu_bwd":
        s["dh"] = (1e-2 * torch.randn(n, f, generator=g, device=dev)).to(t)
        if case["source"] == "kept":  # the projections that the forward pass kept
            s["gate"], s["up"] = x @ s["w_gate"].t(), x @ s["w_up"].t()
    return s


def _views(flat, s):
    return [flat[at:at + n] for n, at in zip(s["sizes"], s["begin"])]


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "adamw":
        s["params"], s["grads"] = _views(s["p"], s), _views(s["g"], s)
    if own:
        import chunked_log_prob_gb300 as clp

        s["clp"] = clp
        if case["op"] == "adamw":  # the optimizer that the program keeps
            states = list(zip(_views(s["m"], s), _views(s["v"], s)))
            if case["bits"] == 8:
                blocks = [(at // BLOCK, -(-n // BLOCK)) for n, at in zip(s["sizes"], s["begin"])]
                states = [(m, v, s["m_scale"][b:b + k], s["v_scale"][b:b + k])
                          for (m, v), (b, k) in zip(states, blocks)]
            s["opt"] = clp.AdamW(
                s["params"], lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=s["decay"],
                states=[clp.AdamState(*z) for z in states], steps_done=STEPS_DONE, seed=seed,
                copies=None if case["copy"] == "none" else _views(s["copy"], s))
    return s


# -------------------------------------------------------------- plain form ----


def _act(name, g):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    if name == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * 0.5 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * g * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (g + 0.044715 * g ** 3)))
    return torch.clamp(g, min=0.0)


def _act_slope(name, g):
    if name == "silu":
        e = 1.0 / (1.0 + torch.exp(-g))
        return e * (1.0 + g * (1.0 - e))
    if name == "gelu":
        return (0.5 * (1.0 + torch.erf(g * 0.5 ** 0.5))
                + g * torch.exp(-0.5 * g * g) / (2.0 * math.pi) ** 0.5)
    if name == "gelu_tanh":
        c = (2.0 / math.pi) ** 0.5
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)
    return (g > 0).to(g.dtype)


def _rows(y, mask):
    return y if mask is None else torch.where(mask[:, None] != 0, y, torch.zeros_like(y))


def _plain_glu_fwd(s):
    c, t, m = s["case"], DTYPES[s["case"]["dtype"]], s["mask"]
    x = _rows(s["x"].float(), m)
    g, u = x @ s["w_gate"].float().t(), x @ s["w_up"].float().t()
    out = {"h": _rows(_act(c["act"], g) * u, m).to(t)}
    if c["gates"]:
        out["gate"], out["up"] = g.to(t), u.to(t)
    return out


def _plain_glu_bwd(s):
    c, t, m = s["case"], DTYPES[s["case"]["dtype"]], s["mask"]
    wg, wu = s["w_gate"].float(), s["w_up"].float()
    if c["source"] == "kept":
        g, u = _rows(s["gate"].float(), m), _rows(s["up"].float(), m)
    else:
        x = _rows(s["x"].float(), m)
        g, u = x @ wg.t(), x @ wu.t()
    dh = _rows(s["dh"].float(), m)
    a = _act(c["act"], g)
    out = {"dgate": (dh * u * _act_slope(c["act"], g)).to(t), "dup": (dh * a).to(t)}
    if c["h"]:
        out["h"] = (a * u).to(t)
    # dx is that of the gradients as they are handed on.
    out["dx"] = (out["dgate"].float() @ wg + out["dup"].float() @ wu).to(t)
    return out


def _plain_glu_wgrad(s):
    x = s["x"].float()
    dg, du = s["dgate"].float().t() @ x, s["dup"].float().t() @ x
    if s["case"]["accumulate"]:
        dg, du = dg + s["add_gate"], du + s["add_up"]
    return {"dw_gate": dg, "dw_up": du}


LOW32 = 0xFFFFFFFF


def _mix(x):
    """A 32-bit number to another, all bits mixed (multiply and fold)."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & LOW32
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & LOW32
    return x ^ (x >> 16)


def _keys(seed, step):
    """The two keys of a step's hash."""
    a = _mix((seed & LOW32) ^ _mix(((seed >> 32) & LOW32) + 0x3C6EF372))
    b = _mix((step & LOW32) ^ _mix((((step >> 32) & LOW32) + a) & LOW32))
    return b, _mix((b + 0x510E527F) & LOW32)


def _random_bits(total, seed, step, dev):
    """Two hashes for each place 0 <= i < total."""
    k0, k1 = _keys(seed, step)
    i = torch.arange(total, device=dev)
    x = (i & LOW32) ^ k0
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & LOW32
    x = x ^ (x >> 15)
    x = (x + k1 + (i >> 32) * 0x1F83D9AB) & LOW32
    x = (x * 0xBB67AE85) & LOW32
    x = x ^ (x >> 16)
    y = ((x ^ k1) * 0x5BE0CD19) & LOW32
    return x, y ^ (y >> 16)


def _plain_to_e4m3(a, square, u):
    """Codes of a (0 <= a <= 448), rounded up where u (0 to 65535) says so; `square`:
    by the distances of the squares."""
    bits = a.view(torch.int32)
    small = a < 2.0 ** -6
    count = torch.floor(a * 512.0)
    lo = torch.where(small, count / 512.0, (bits & -0x100000).view(torch.float32))
    exponent = (bits & 0x7F800000) - (3 << 23)
    step = torch.where(small, torch.full_like(exponent, (127 - 9) << 23), exponent).view(
        torch.float32)
    code = torch.where(small, count.to(torch.int32), (bits >> 20) - (120 << 3))
    u = u.float()
    if square:
        up = u * ((2.0 * lo + step) * step) < 65536.0 * ((a - lo) * (a + lo))
    else:
        up = u * step < 65536.0 * (a - lo)
    return code + up.to(torch.int32)


def _plain_moment_8(y, square, u):
    """(e4m3, scales) of a moment; for the second one y is its square root."""
    y = y.reshape(-1, BLOCK)
    top = y.abs().amax(1)
    live = top >= 2.0 ** -118
    scale = torch.where(live, top / TOP, torch.zeros_like(top))
    a = y.abs() * torch.where(live, TOP / top, torch.zeros_like(top))[:, None]
    code = _plain_to_e4m3(a.clamp_max(TOP).reshape(-1), square, u)
    y = y.reshape(-1)
    if square:
        some = (y > 0) & live.repeat_interleave(BLOCK)
        code = torch.where(some, code.clamp_min(1), code)
    else:
        code = code | torch.where(y < 0, 0x80, 0)
    return code.to(torch.uint8).view(torch.float8_e4m3fn), scale


def _plain_adamw(s):
    c = s["case"]
    s["t"] += 1
    dev, total = s["p"].device, s["p"].numel()
    g, out = s["g"].float(), {}
    if c["clip"]:
        norm = (g.double() * g.double()).sum().sqrt()
        scale = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0).float()
        out["norm"], out["scale"] = norm.float(), scale
        g = g * scale
    if c["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m = (s["m"].float().reshape(-1, BLOCK) * s["m_scale"][:, None]).reshape(-1)
        r = (s["v"].float().reshape(-1, BLOCK) * s["v_scale"][:, None]).reshape(-1)
        v = r * r
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * (g * g)
    blocks = torch.tensor([-(-n // BLOCK) * BLOCK for n in s["sizes"]], device=dev)
    shrink = torch.tensor([1.0 - LR * w for w in s["decay"]], device=dev)
    shrink = torch.repeat_interleave(shrink, blocks, output_size=total)
    root = v.sqrt()
    step = (LR / (1.0 - BETA1 ** s["t"])) * m
    p = s["p"].float() * shrink - step / (root / (1.0 - BETA2 ** s["t"]) ** 0.5 + EPS)
    if c["bits"] == 8 or c["pdtype"] == "bf16":
        x, y = _random_bits(total, s["seed"], s["t"], dev)
    if c["pdtype"] == "bf16":
        bits = (p.view(torch.int32) + (y & 0xFFFF).to(torch.int32)) & -0x10000
        s["p"].copy_(bits.view(torch.float32))
    else:
        s["p"].copy_(p)
    if c["copy"] != "none":
        s["copy"].copy_(p)
        out["copy"] = s["copy"]
    if c["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        q, scale = _plain_moment_8(m, False, x & 0xFFFF)
        s["m"].copy_(q)
        s["m_scale"].copy_(scale)
        q, scale = _plain_moment_8(root, True, x >> 16)
        s["v"].copy_(q)
        s["v_scale"].copy_(scale)
    return _adamw_outputs(s, out)


def _adamw_outputs(s, out):
    names = ["p", "m", "v"] + (["m_scale", "v_scale"] if s["case"]["bits"] == 8 else [])
    return {**out, **{k: s[k] for k in names}}


# --------------------------------------------------------------------- run ----


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"glu_fwd": _plain_glu_fwd, "glu_bwd": _plain_glu_bwd,
                "glu_wgrad": _plain_glu_wgrad, "adamw": _plain_adamw}[op](s)
    clp = s["clp"]
    if op == "glu_fwd":
        r = clp.grpo_glu_fwd(s["x"], s["w_gate"], s["w_up"], act=c["act"], mask=s["mask"],
                             want_gates=c["gates"])
        return {"h": r.h, "gate": r.gate, "up": r.up} if c["gates"] else {"h": r.h}
    if op == "glu_bwd":
        r = clp.grpo_glu_bwd(s["dh"], s["x"], s["w_gate"], s["w_up"], gate=s.get("gate"),
                             up=s.get("up"), act=c["act"], mask=s["mask"], want_h=c["h"])
        out = {"dgate": r.dgate, "dup": r.dup, "dx": r.dx}
        return {**out, "h": r.h} if c["h"] else out
    if op == "glu_wgrad":
        dg, du = clp.grpo_glu_wgrad(s["dgate"], s["dup"], s["x"], add_gate=s.get("add_gate"),
                                    add_up=s.get("add_up"))
        return {"dw_gate": dg, "dw_up": du}
    out, scale = {}, None
    if c["clip"]:
        norm = clp.grpo_grad_norm(s["grads"], max_norm=MAX_NORM)
        out["norm"], out["scale"], scale = norm.norm, norm.scale, norm.scale
    s["opt"].step(s["grads"], scale=scale)
    if c["copy"] != "none":
        out["copy"] = s["copy"]
    return _adamw_outputs(s, out)


# ------------------------------------------------------------------- exact ----


def _exact_act(name, g):
    """act(g) and its derivative."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    if name == "gelu":
        phi = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        # 0.5 (1 + tanh z) is the logistic function of 2 z
        z = 2 * k * (g + 0.044715 * g * g * g)
        s = torch.sigmoid(z)
        return g * s, s + g * s * (1 - s) * 2 * k * (1 + 0.134145 * g * g)
    on = (g > 0).double()
    return g * on, on


def _exact_bits(total, seed, step, dev):
    """The two 32-bit hashes of each place, in wrapping 64-bit arithmetic."""
    m32 = (1 << 32) - 1

    def fold(z, k):
        return z ^ (z >> k)

    def scramble(z):
        z = fold(z, 16) * 0x6A09E667 & m32
        return fold(fold(z, 15) * 0xBB67AE85 & m32, 16)

    a = scramble((seed & m32) ^ scramble((seed >> 32 & m32) + 0x3C6EF372))
    b = scramble((step & m32) ^ scramble((step >> 32 & m32) + a & m32))
    k1 = scramble(b + 0x510E527F & m32)
    i = torch.arange(total, device=dev, dtype=torch.int64)
    z = fold((i & m32) ^ b, 16) * 0x6A09E667 & m32
    z = (fold(z, 15) + k1 + (i >> 32) * 0x1F83D9AB) & m32
    z = fold(z * 0xBB67AE85 & m32, 16)
    return z, fold((z ^ k1) * 0x5BE0CD19 & m32, 16)


def _exact_8(y, power, u):
    """The e4m3 values and the scales that a moment goes to: y is kept by its power."""
    dev = y.device
    grid = torch.arange(127, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn).double()
    y = y.reshape(-1, BLOCK)
    top = y.abs().amax(1, keepdim=True)
    a = torch.where(top > 0, y.abs() * TOP / top, torch.zeros_like(y)).clamp(max=TOP)
    at = (torch.searchsorted(grid, a, right=True) - 1).clamp(0, 125)
    lo, hi = grid[at], grid[at + 1]
    chance = (a ** power - lo ** power) / (hi ** power - lo ** power)
    del lo, hi
    at = at + (u.reshape(-1, BLOCK).double() / 65536 < chance)
    if power == 2:
        at = torch.where(y > 0, at.clamp(min=1), at)
    return (torch.sign(y) * grid[at]).reshape(-1), (top / TOP)[:, 0]


def _exact_adamw(s):
    c, t = s["case"], STEPS_DONE + 1
    dev, total = s["p"].device, s["p"].numel()
    g, out = s["g"].double(), {}
    if c["clip"]:
        out["norm"] = torch.linalg.vector_norm(g)
        out["scale"] = torch.clamp(MAX_NORM / (out["norm"] + 1e-6), max=1.0)
        g = g * out["scale"]
    m, v = s["m"].double(), s["v"].double()
    if c["bits"] == 8:
        m = (m.reshape(-1, BLOCK) * s["m_scale"].double()[:, None]).reshape(-1)
        v = (v.reshape(-1, BLOCK) * s["v_scale"].double()[:, None]).reshape(-1) ** 2
    m = m + (1 - BETA1) * (g - m)
    v = v + (1 - BETA2) * (g * g - v)
    del g
    p = s["p"].double()
    for n, at, decay in zip(s["sizes"], s["begin"], s["decay"]):
        p[at:at + n] *= 1 - LR * decay
    p -= LR * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    out["p"], out["m"], out["v"] = p, m, v
    if c["bits"] == 8 or c["pdtype"] == "bf16":
        x, y = _exact_bits(total, s["seed"], t, dev)
    if c["pdtype"] == "bf16":
        step = torch.exp2((torch.frexp(p).exponent - 8).double())
        out["p"] = torch.floor(p.abs() / step + (y & 0xFFFF).double() / 65536) * step * p.sign()
        del step
    if c["copy"] != "none":
        out["copy"] = p
    if c["bits"] == 8:
        out["m"], out["m_scale"] = _exact_8(m, 1, x & 0xFFFF)
        out["v"], out["v_scale"] = _exact_8(torch.sqrt(v), 2, x >> 16)
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    t = DTYPES[case["dtype"]]
    x = s["x"].double()
    if case["op"] == "glu_wgrad":
        out = {"dw_gate": torch.mm(s["dgate"].double().t(), x),
               "dw_up": torch.mm(s["dup"].double().t(), x)}
        if case["accumulate"]:
            out["dw_gate"] += s["add_gate"].double()
            out["dw_up"] += s["add_up"].double()
        return out
    alive = 1.0 if s["mask"] is None else (s["mask"] != 0).double()[:, None]
    wg, wu = s["w_gate"].double(), s["w_up"].double()
    if case.get("source") == "kept":
        g, u = s["gate"].double() * alive, s["up"].double() * alive
    else:
        g, u = torch.mm(x * alive, wg.t()), torch.mm(x * alive, wu.t())
    a, slope = _exact_act(case["act"], g)
    if case["op"] == "glu_fwd":
        out = {"h": a * u}
        return {**out, "gate": g, "up": u} if case["gates"] else out
    dh = s["dh"].double() * alive
    out = {"dgate": dh * u * slope, "dup": dh * a}
    if case["h"]:
        out["h"] = a * u
    out["dx"] = torch.mm(out["dgate"].to(t).double(), wg) + torch.mm(out["dup"].to(t).double(), wu)
    return out
