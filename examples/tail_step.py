"""One training step of a decoder's tail, its activations kept in 8 bits.

    residual stream x, last block's activation a
    z = x + a Wp^T          the block's last linear layer and the residual add
    h = RMSnorm(z) w        grpo_norm_fwd (keeps z's 8-bit checkpoint)
    loss(h Wlm^T)           grpo_loss_fwd_bwd: dH, without the logits
    dz, dw                  grpo_norm_bwd, from the checkpoint of z
    dWp = dz^T a            grpo_ckpt_wgrad, from the checkpoint of a
    da = dz Wp              into the block

What the backward passes of the norm and of the linear layer read, z and a, is kept
as 1.03 bytes a value instead of 2. h stays in bf16 until the loss has read it (that
call is the head's forward and backward pass in one).

Run: python examples/tail_step.py (one GB300).
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


@dataclass
class Tail:
    """Weights of the tail: projection [D, F], norm [D], lm_head [V, D]."""

    proj: torch.Tensor
    norm: torch.Tensor
    head: torch.Tensor
    eps: float = 1e-6


@dataclass
class StepResult:
    loss: torch.Tensor
    dx: torch.Tensor      # gradient of the residual stream
    da: torch.Tensor      # gradient of the last block's activation
    dproj: torch.Tensor   # fp32 [D, F]
    dnorm: torch.Tensor   # fp32 [D]
    kept_bytes: int       # checkpoints of z and a, and rstd; h is held besides, up to the loss


def tail_step(tail: Tail, x, a, ids, mask, old_logp, ref_logp, adv, seq_len, *, params=None,
              dproj=None, dnorm=None) -> StepResult:
    """Loss and gradients of one batch; dproj and dnorm, where given, are added to
    (in place)."""
    # Forward: what is kept is a's and z's checkpoints and one rstd a row; and h,
    # for the loss.
    keep_a = clp.grpo_ckpt_pack(a, mask=mask)
    fwd = clp.grpo_norm_fwd(x, tail.norm, residual=a @ tail.proj.t(), eps=tail.eps, mask=mask,
                            want_ckpt=True)
    h, rstd, keep_z = fwd.y, fwd.rstd, fwd.ckpt
    del fwd, a
    kept = keep_a.data.numel() + keep_z.data.numel() + 4 * rstd.numel()

    loss, _, dh = clp.grpo_loss_fwd_bwd(h, tail.head, ids, mask, old_logp, ref_logp, adv, seq_len,
                                        params=params, want_logp=False)
    del h
    # Backward, from the checkpoints.
    back = clp.grpo_norm_bwd(dh, keep_z, tail.norm, None, rstd, mask=mask, add_dweight=dnorm,
                             dweight=dnorm)
    dproj = clp.grpo_ckpt_wgrad(back.dx, keep_a, add=dproj, dW=dproj)
    return StepResult(loss, back.dx, back.dx @ tail.proj, dproj, back.dweight, kept)


def main():
    import synth

    dev = torch.device("cuda:0")
    p = synth.make_problem("tiny", seed=0)
    n, d, f = p.n_tokens, p.hidden_size, 2 * p.hidden_size
    g = torch.Generator().manual_seed(1)
    bf = torch.bfloat16
    tail = Tail((torch.randn(d, f, generator=g) / f ** 0.5).to(dev, bf),
                torch.ones(d, dtype=bf, device=dev), p.weight.to(dev))
    x = torch.randn(n, d, generator=g).to(dev, bf)
    a = torch.randn(n, f, generator=g).to(dev, bf)
    ids, mask = p.ids.to(dev), p.mask.to(dev)
    h = clp.grpo_norm_fwd(x, tail.norm, residual=a @ tail.proj.t()).y
    old, _ = clp.grpo_logp_fwd(h, tail.head, ids)
    r = tail_step(tail, x, a, ids, mask, old, old - 0.05, p.adv.to(dev), p.seq_len)
    print(f"loss {r.loss.item():.6f}  |dproj| {r.dproj.norm().item():.4e}  "
          f"|dnorm| {r.dnorm.norm().item():.4e}  z and a kept in {r.kept_bytes / 2**20:.2f} MiB "
          f"(in bf16 {2 * n * (d + f) / 2**20:.2f})")


if __name__ == "__main__":
    main()
