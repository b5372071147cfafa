"""Plain 64-bit forms of the score call, its gradient and the scaled logits,
and the bounds their GPU results are held to.

Inputs are small integers times powers of two, so every logit is exact in fp32
in any order of addition: ids can be compared for equality, ties included.
"""
from __future__ import annotations

import numpy as np

NO_TARGET = -1


def grid_inputs(seed, V, d, B, n_ties=2, masked=0.0):
    """(W [V, d], h [B, d] float64 on a grid that bf16 and fp16 hold exactly,
    targets int32 [B]); some rows of W are copies of others (exact ties)."""
    rng = np.random.Generator(np.random.PCG64(seed))
    step = 2.0 ** -round(np.log2(np.sqrt(d) * 16 / 2.5))
    W = np.clip(np.rint(rng.standard_normal((V, d)) * 16), -63, 63) * step
    for _ in range(n_ties if V > 1 else 0):
        a, b = rng.integers(0, V, 2)
        W[b] = W[a]
    targets = rng.integers(0, V, B).astype(np.int32)
    lean = rng.random((B, 1)) * (np.log(V) + 1.0) / (0.125 * step * d * 256.0)
    h = np.rint(rng.standard_normal((B, d)) * 8 + lean * W[targets] / step)
    h = np.clip(h, -31, 31) * 0.125
    if masked:
        targets[rng.random(B) < masked] = NO_TARGET
    return W, h, targets


def to_dev(x, dtype):
    import torch
    t = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    return torch.from_numpy(np.ascontiguousarray(x)).to(t).cuda()


def logsoftmax(z):
    m = z.max(axis=1, keepdims=True)
    lse = m + np.log(np.exp(z - m).sum(axis=1, keepdims=True))
    return z - lse, lse[:, 0]


def score(W, h, targets, K, T):
    z = h @ W.T
    logp, lse = logsoftmax(z / T)
    p = np.exp(logp)
    H = -(p * logp).sum(axis=1)
    n = np.arange(len(h))
    lp = np.where(targets >= 0, logp[n, np.maximum(targets, 0)], 0.0)
    top = np.argsort(-z, axis=1, kind="stable")[:, :K]     # equal logits: lowest index first
    return {"logp": lp, "entropy": H, "lse": lse, "top_token": top,
            "top_logp": np.take_along_axis(logp, top, axis=1)}


# The fp32 evaluation on exact logits (see score_stats.cuh). One term e^(t/T),
# t = z - m exact: 2^-23 |t / T| from the product with log2(e) / T and that
# constant's own rounding, 2^-22 from ex2.approx; weighted by p the first part
# is at most 2^-23 (H + 1) <= 2e-6 for H < 14. Sums: 16 additions, then at most
# 7 merges within a tile's row range and 7 + (tiles per leaf) in the tree, each
# two roundings and one scaled side (2^-22): below 32 * 3e-7 = 1e-5 for the
# sizes here. S and U therefore carry at most 2e-5 of themselves. log S then
# has that absolute error; the entropy log S - U / (S T), whose two terms are
# non-negative, 2e-5 (1 + 2 H); a log-probability adds the roundings of
# (z - m) / T and of the difference.
REL = 2e-5


def logp_tol(logp, lse):
    return REL + 2.0 ** -22 * (np.abs(logp) + 1.0)


def lse_tol(lse):
    return REL + 2.0 ** -22 * (np.abs(lse) + 1.0)


def entropy_tol(H):
    return REL * (1.0 + 2.0 * H)


def gradient(W, h, targets, dlogp, dentropy, T):
    logp, lse = logsoftmax((h @ W.T) / T)
    p = np.exp(logp)
    H = -(p * logp).sum(axis=1)
    has = (targets >= 0) & (targets < len(W))
    g = np.where(has, dlogp, 0.0)
    dz = -p * g[:, None]
    dz[np.arange(len(h)), np.where(has, targets, 0)] += g
    if dentropy is not None:
        dz -= dentropy[:, None] * p * (logp + H[:, None])
    dz /= T
    return {"dz": dz, "dh": dz @ W, "dW": dz.T @ h, "lse": lse, "entropy": H}


def loss(W, h, targets, dlogp, dentropy, T):
    """The scalar whose gradient the backward call takes."""
    logp, _ = logsoftmax((h @ W.T) / T)
    has = (targets >= 0) & (targets < len(W))
    lp = logp[np.arange(len(h)), np.where(has, targets, 0)]
    out = (np.where(has, dlogp, 0.0) * lp).sum()
    if dentropy is not None:
        out += (dentropy * -(np.exp(logp) * logp).sum(axis=1)).sum()
    return out


def gradient_tol(ref, W, h, p_terms, dtype):
    """Elementwise bounds of (dh, dW): each dz within half a unit of the 16-bit
    type plus 1e-5 of its parts (p_terms: the sum of their magnitudes, which
    for terms that cancel exceeds |dz|), summed without cancellation; sums in
    fp32 (2e-5 of the magnitudes); the output's own rounding."""
    u = 2.0 ** -9 if dtype == "bf16" else 2.0 ** -12
    tiny = 0.0 if dtype == "bf16" else 2.0 ** -25     # fp16 outputs: half a subnormal step
    each = u * np.abs(ref["dz"]) + (u + 3e-5) * p_terms
    dh = each @ np.abs(W) + 2e-5 * (p_terms @ np.abs(W)) + 2 * u * np.abs(ref["dh"]) + tiny
    dW = each.T @ np.abs(h) + 2e-5 * (p_terms.T @ np.abs(h)) + 2 * u * np.abs(ref["dW"]) + tiny
    return dh, dW
