"""One training step of a decoder's last feed-forward block, its tail and its weights.

    residual stream x
    y = RMSnorm(x) w1                     grpo_norm_fwd
    a = silu(y Wg^T) * (y Wu^T)           grpo_glu_fwd (keeps a's 8-bit checkpoint)
    z = x + a Wd^T                        the block's last linear layer, residual add
    h = RMSnorm(z) w2                     grpo_norm_fwd (keeps z's 8-bit checkpoint)
    loss(h Wlm^T)                         grpo_loss_fwd_bwd: dH and dWlm
    dz, dw2                               grpo_norm_bwd, from the checkpoint of z
    dWd = dz^T a, da = dz Wd              grpo_ckpt_wgrad, from the checkpoint of a
    dgate, dup, dy                        grpo_glu_bwd, the projections computed again
    dWg, dWu                              grpo_glu_wgrad
    dx, dw1                               grpo_norm_bwd
    clip by the norm of all gradients     grpo_grad_norm
    new weights                           AdamW.step: fp32 weights, bf16 copies for the
                                          products, moments in 8 bits

Of the block's [N, F] tensors only a's checkpoint is kept from the forward pass: 1.03
bytes a value, against 6 for a and both projections in bf16.

Run: python examples/block_step.py (one GB300).
"""

from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import chunked_log_prob_gb300 as clp  # noqa: E402

NAMES = ("norm1", "gate", "up", "down", "norm2", "head")


@dataclass
class Grads:
    loss: torch.Tensor
    dx: torch.Tensor               # gradient of the residual stream
    weights: dict[str, torch.Tensor]  # fp32, by NAMES


class Block:
    """The weights: fp32, and the bf16 copies that the products read."""

    def __init__(self, weights: dict[str, torch.Tensor], *, lr=1e-5, state_bits=8, eps=1e-6,
                 max_norm=1.0):
        self.master = {k: weights[k].float().contiguous() for k in NAMES}
        self.w = {k: self.master[k].to(torch.bfloat16) for k in NAMES}
        self.eps, self.max_norm = eps, max_norm
        decay = [0.0 if k.startswith("norm") else 0.01 for k in NAMES]
        self.opt = clp.AdamW([self.master[k] for k in NAMES], lr=lr, weight_decay=decay,
                             state_bits=state_bits, copies=[self.w[k] for k in NAMES])

    def grads(self, x, ids, mask, old_logp, ref_logp, adv, seq_len, *, params=None) -> Grads:
        w, rms = self.w, dict(kind="rms", eps=self.eps, mask=mask)
        first = clp.grpo_norm_fwd(x, w["norm1"], **rms)
        fwd = clp.grpo_glu_fwd(first.y, w["gate"], w["up"], mask=mask, want_ckpt=True)
        second = clp.grpo_norm_fwd(x, w["norm2"], residual=fwd.h @ w["down"].t(), want_ckpt=True,
                                   **rms)
        keep_a = fwd.ckpt
        del fwd
        loss, _, dh, dhead = clp.grpo_loss_fwd_bwd(second.y, w["head"], ids, mask, old_logp,
                                                   ref_logp, adv, seq_len, params=params,
                                                   want_logp=False, want_dW=True)
        back = clp.grpo_norm_bwd(dh, second.ckpt, w["norm2"], None, second.rstd, mask=mask)
        ddown = clp.grpo_ckpt_wgrad(back.dx, keep_a)
        glu = clp.grpo_glu_bwd(back.dx @ w["down"], first.y, w["gate"], w["up"], mask=mask)
        dgate, dup = clp.grpo_glu_wgrad(glu.dgate, glu.dup, first.y)
        last = clp.grpo_norm_bwd(glu.dx, x, w["norm1"], None, first.rstd, dres=back.dx, mask=mask)
        return Grads(loss, last.dx, dict(zip(NAMES, (last.dweight, dgate, dup, ddown, back.dweight,
                                                     dhead))))

    def update(self, g: Grads) -> torch.Tensor:
        """Clips and steps; the norm of the gradients."""
        grads = [g.weights[k] for k in NAMES]
        norm = clp.grpo_grad_norm(grads, max_norm=self.max_norm)
        self.opt.step(grads, scale=norm.scale)
        return norm.norm


def random_weights(d, f, head, generator):
    def t(*shape):
        return torch.randn(*shape, generator=generator) / shape[-1] ** 0.5

    ones = torch.ones(d)
    return {"norm1": ones, "gate": t(f, d), "up": t(f, d), "down": t(d, f), "norm2": ones.clone(),
            "head": head.float()}


def main():
    import synth

    dev = torch.device("cuda:0")
    p = synth.make_problem("tiny", seed=0)
    n, d, f = p.n_tokens, p.hidden_size, 4 * p.hidden_size
    g = torch.Generator().manual_seed(1)
    block = Block({k: v.to(dev) for k, v in random_weights(d, f, p.weight, g).items()}, lr=1e-3)
    x = torch.randn(n, d, generator=g).to(dev, torch.bfloat16)
    ids, mask, adv = p.ids.to(dev), p.mask.to(dev), p.adv.to(dev)
    old = torch.full((n,), -8.0, device=dev)
    for step in range(3):
        r = block.grads(x, ids, mask, old, old, adv, p.seq_len)
        norm = block.update(r)
        print(f"step {step}: loss {r.loss.item():.6f}  |gradients| {norm.item():.4e}")


if __name__ == "__main__":
    main()
