"""The score call as a differentiable torch function.

``scored_logprobs(head, h, targets)`` returns what ``Head.score`` computes of
each hidden row -- the log-probability of its target and the entropy of its
distribution -- as tensors whose gradients reach ``h`` and ``head.W`` through
``Head.score_backward``: logits are recomputed there, never stored
("batch-logprob-gap": the trainer's log-probabilities and the policy loss on
them).
"""
from __future__ import annotations

import torch


class _Score(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, W, targets, head, temperature):
        s = head.score(h, targets, temperature=temperature)
        ctx.save_for_backward(h, targets, s.lse, s.entropy)
        ctx.head, ctx.temperature = head, temperature
        return s.logp, s.entropy

    @staticmethod
    def backward(ctx, dlogp, dentropy):
        h, targets, lse, entropy = ctx.saved_tensors
        need_dh, need_dW = ctx.needs_input_grad[:2]
        if not (need_dh or need_dW):
            return None, None, None, None, None
        if dlogp is None:
            dlogp = torch.zeros_like(lse)
        if dentropy is not None:
            dentropy = dentropy.float().contiguous()
        dh, dW = ctx.head.score_backward(h, targets, lse, entropy, dlogp.float().contiguous(),
                                         dentropy, temperature=ctx.temperature, need_dh=need_dh,
                                         need_dW=need_dW)
        return dh, dW, None, None, None


def scored_logprobs(head, h, targets, temperature: float = 1.0):
    """(logp [B], entropy [B]) of hidden rows h [B, d] and targets int32 [B]
    (DETLM_NO_TARGET: 0 and no gradient of logp), float32, differentiable with
    respect to h and head.W where they require gradients. After an optimizer
    has changed head.W, call head.weights_changed()."""
    return _Score.apply(h, head.W, targets, head, float(temperature))
