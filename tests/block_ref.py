"""Plain 64-bit forms of the e4m3 head's operators and of a beam-search step
(torch on the CPU or the GPU; no code of the package)."""
import math

import torch

BLOCK = 128


def quantize(x, rows):
    """(q, scale) in float64: x [B, d] in blocks of rows x 128."""
    B, d = x.shape
    x = x.double()
    q = torch.empty_like(x)
    scale = torch.empty((-(-B // rows), -(-d // BLOCK)), dtype=torch.float64, device=x.device)
    for i in range(scale.shape[0]):
        for j in range(scale.shape[1]):
            at = (slice(i * rows, (i + 1) * rows), slice(j * BLOCK, (j + 1) * BLOCK))
            part = x[at]
            most = float(part.abs().max())
            if not bool(torch.isfinite(part).all()):
                scale[i, j], q[at] = math.nan, math.nan
                continue
            e = -126
            if most > 0:
                m, p = math.frexp(most / 448)      # most / 448 = m 2^p, m < 1
                e = max(p - 1 if m == 0.5 else p, -126)
            s = 2.0 ** e if most > 0 else 1.0
            y = part / s
            step = 2.0 ** (torch.frexp(y.abs().clamp_min(2.0 ** -6)).exponent - 1 - 3).double()
            scale[i, j], q[at] = s, torch.round(y / step) * step
    return q, scale


def logits(q, xs, W, ws):
    """(z, A): the scaled products' sum and the sum of their magnitudes."""
    V, d = W.shape
    x = q.double() * xs.double().repeat_interleave(BLOCK, dim=1)[:, :d]
    w = W.double() * ws.double().repeat_interleave(BLOCK, dim=1)[:, :d].repeat_interleave(
        BLOCK, dim=0)[:V]
    return x @ w.t(), x.abs() @ w.abs().t()


def logits_tol(A, z, blocks, dtype):
    """Bound on a logit of `blocks` chunks. A chunk is four steps of the tensor
    core's accumulation, each off by at most two half-steps of fp32 of what it
    has added up (its products are exact); each of the fused multiply-adds, and
    the product of the scales, rounds once. All are relative to magnitudes that
    A bounds. Then the output's own half step (and its smallest number's)."""
    u = 2.0 ** -24
    tol = (8 + blocks + 1) * u * A
    half = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dtype]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -140
    return tol + (z.abs() + tol) * half + tiny


def select(logits, scores, n_out, T=1.0, finished=None, end_token=0):
    """(parent, token, score) with score in float64, by sorting every candidate:
    score falling, then beam, then logit falling, then token."""
    n_seq, beams = scores.shape
    V = logits.shape[1]
    z = logits.double().cpu()
    own = scores.double().cpu()
    parents, tokens, values = [], [], []
    for s in range(n_seq):
        total = torch.full((beams, V), -math.inf, dtype=torch.float64)
        raw = torch.full((beams, V), -math.inf, dtype=torch.float64)
        for b in range(beams):
            if not math.isfinite(own[s, b]):
                continue
            if finished is not None and bool(finished[s, b]):
                total[b, end_token] = own[s, b]
                continue
            row = z[s * beams + b]
            if bool(torch.isnan(row).any()) or float(row.max()) in (math.inf, -math.inf):
                continue
            total[b] = torch.log_softmax(row / T, dim=0) + own[s, b]
            raw[b] = row
        # stable sorts, the least important first (tokens are in order)
        order = torch.sort(raw.view(-1), descending=True, stable=True).indices
        order = order[torch.sort(order // V, stable=True).indices]
        order = order[torch.sort(total.view(-1)[order], descending=True, stable=True).indices]
        order = order[:n_out]
        value = total.view(-1)[order]
        pad = n_out - len(order)
        value = torch.cat([value, torch.full((pad,), -math.inf, dtype=torch.float64)])
        order = torch.cat([order, torch.zeros(pad, dtype=order.dtype)])
        none = value == -math.inf
        parents.append(torch.where(none, -1, order // V))
        tokens.append(torch.where(none, -1, order % V))
        values.append(value)
    return torch.stack(parents).int(), torch.stack(tokens).int(), torch.stack(values)


def score_tol(score, own, z_range, V, T):
    """Bound on a candidate's score. The row's sum S: an exponent is off by two
    half-steps of itself (|e| 2^e <= 0.54), ex2.approx by 2^-22, an addition of
    a tile's tree (4 + 5 levels) and of the joins (two roundings each, about 20
    at 152064 entries) by half a step: in all less than 2^-22 + 2^-23 + 50 2^-24
    of S, and log S of it by as much. Then the difference of the logits, its
    product with the rounded 1 / T, log S, the two sums: half a step each of
    what they are."""
    u = 2.0 ** -24
    return 56 * u + u * (4 * z_range / T + 3 * (math.log(V) + 1) + 2 * own + 2 * score)


def reorder(state, out, parent, used=None, dim=None):
    """out's rows after the step, [rows, ...]."""
    n_seq, beams = parent.shape
    beams_in = state.shape[0] // n_seq
    want = out.clone()
    for s in range(n_seq):
        for j in range(beams):
            p = int(parent[s, j])
            if not 0 <= p < beams_in:
                continue
            src, dst = state[s * beams_in + p], want[s * beams + j]
            if used is not None and dim is not None:
                src, dst = src.narrow(dim - 1, 0, used), dst.narrow(dim - 1, 0, used)
            dst.copy_(src)
    return want
