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
        # W (a reference) so that autograd notices a change in place before
        # the backward call, whose logits would not fit the saved statistics
        ctx.save_for_backward(h, W, targets, s.lse, s.entropy)
        ctx.head, ctx.temperature = head, temperature
        ctx.set_materialize_grads(False)      # an output the loss does not use: None
        return s.logp, s.entropy

    @staticmethod
    def backward(ctx, dlogp, dentropy):
        h, W, targets, lse, entropy = ctx.saved_tensors
        need_dh, need_dW = ctx.needs_input_grad[:2]
        if not (need_dh or need_dW):
            return None, None, None, None, None
        dlogp = torch.zeros_like(lse) if dlogp is None else dlogp.float().contiguous()
        if dentropy is not None:
            dentropy = dentropy.float().contiguous()
        dh, dW = _ScoreGradient.apply(h, W, targets, lse, entropy, dlogp, dentropy, ctx.head,
                                      ctx.temperature, need_dh, need_dW)
        return dh, dW, None, None, None


class _ScoreGradient(torch.autograd.Function):
    """The gradient call, as a node of its own: with create_graph its results
    depend on h, W and the incoming gradients, and differentiating them has to
    fail instead of finding constants."""

    @staticmethod
    def forward(ctx, h, W, targets, lse, entropy, dlogp, dentropy, head, temperature, need_dh,
                need_dW):
        return head.score_backward(h, targets, lse, entropy, dlogp, dentropy,
                                   temperature=temperature, need_dh=need_dh, need_dW=need_dW)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("scored_logprobs cannot be differentiated twice")


def scored_logprobs(head, h, targets, temperature: float = 1.0):
    """(logp [B], entropy [B]) of hidden rows h [B, d] and targets int32 [B]
    (DETLM_NO_TARGET: 0 and no gradient of logp), float32, differentiable with
    respect to h and head.W where they require gradients, once (a second
    derivative is refused, as is a backward pass after h or head.W was changed
    in place). After an optimizer has changed head.W, call
    head.weights_changed()."""
    return _Score.apply(h, head.W, targets, head, float(temperature))
