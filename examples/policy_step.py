"""One policy-gradient step around the output head, on synthetic hidden rows.

The rollout side serves an int8 head (one scale a channel, each token quantized
from its own values): its scaled logits give the sampled tokens and their
log-probabilities under the served model. The trainer's 16-bit head scores the
same tokens, with entropy and the most likely alternatives; the clipped
importance-ratio objective with an entropy bonus is differentiated through the
score call, and the weight takes a step. The share of tokens whose ratio leaves
[0.9, 1.1] before the step is the mismatch between the two heads ("batch-
logprob-gap").

    python examples/policy_step.py [--rows 512] [--vocab 32000] [--dim 2048]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from invariant_output_head_gb300 import Head, quantize_rows          # noqa: E402
from invariant_output_head_gb300.training import scored_logprobs     # noqa: E402


def serve(W, h, temperature):
    """Tokens drawn from the int8 head, and their log-probabilities there."""
    w_scale = W.float().abs().amax(dim=1).clamp_min(1e-12) / 127.0
    Wq = (W.float() / w_scale[:, None]).round().clamp(-127, 127).to(torch.int8)
    head = Head(Wq, "int8")
    q, mult, shift = quantize_rows(h)
    x_scale = torch.ldexp(torch.ones_like(w_scale[:1]).expand(len(h)), shift) / mult.clamp_min(1)
    z = head.scaled_logits(q, x_scale.contiguous(), w_scale) / temperature
    logp = torch.log_softmax(z, dim=1)
    noise = -torch.log(-torch.log(torch.rand_like(z).clamp(1e-20, 1 - 1e-7)))
    tokens = (z + noise).argmax(dim=1)
    assert head.check() == 0
    head.close()
    return tokens.int(), logp.gather(1, tokens[:, None])[:, 0]


def objective(logp, entropy, logp_served, advantage, clip=0.2, bonus=0.01):
    ratio = torch.exp(logp - logp_served)
    clipped = ratio.clamp(1 - clip, 1 + clip)
    return torch.minimum(ratio * advantage, clipped * advantage).mean() + bonus * entropy.mean()


def main(rows=512, vocab=32000, dim=2048, temperature=1.0, lr=0.05, seed=0, say=print):
    torch.manual_seed(seed)
    W = (torch.randn(vocab, dim, device="cuda") * 0.02).bfloat16().requires_grad_()
    h = torch.randn(rows, dim, device="cuda").bfloat16()
    tokens, logp_served = serve(W.detach(), h, temperature)
    advantage = torch.randn(rows, device="cuda")

    head = Head(W, "bf16")
    head.reserve_score(rows, 4)
    head.reserve_backward(rows)
    top = head.score(h, tokens, top_k=4, temperature=temperature)
    out_of_band = ((top.logp - logp_served).exp().sub(1).abs() > 0.1).float().mean().item()
    values = []
    for _ in range(2):                       # before and after one ascent step
        logp, entropy = scored_logprobs(head, h, tokens, temperature)
        value = objective(logp, entropy, logp_served, advantage)
        values.append(value.item())
        if len(values) == 1:
            value.backward()
            with torch.no_grad():
                W += (lr * W.grad.float()).to(W.dtype)
            head.weights_changed()
    assert head.check() == 0
    head.close()
    say(f"tokens out of the ratio band: {out_of_band:.4f}")
    say(f"first row's alternatives: {top.top_token[0].tolist()} "
        f"log p {[round(x, 3) for x in top.top_logp[0].tolist()]}")
    say(f"objective before {values[0]:.6f}, after one step {values[1]:.6f}")
    return out_of_band, values


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--rows", type=int, default=512)
    a.add_argument("--vocab", type=int, default=32000)
    a.add_argument("--dim", type=int, default=2048)
    a = a.parse_args()
    main(a.rows, a.vocab, a.dim)
