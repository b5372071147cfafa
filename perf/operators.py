"""Cases of the operators around the output head's probabilities: scoring of
tokens (log-probability, entropy, most likely alternatives), the gradient of
that score, and the scaled logits of an int8 head.

Each case is one call of one operator. `run` computes it in plain torch
operations, or, where `own` is true, through the package's public calls.

Inputs of the float heads are drawn on a grid (h in steps of 2^-3, W in steps
of a power of two, a few bits each, normally distributed), so every logit is a
sum of integers below 2^24 in units of the grid: its fp32 value is the same in
any order of addition, ties between alternatives are real ties, and the ids
returned are well defined (the lowest index first).
"""
import math

import torch

own = False

NO_TARGET = -1        # a position without a token to score (prompt or padding)
H_STEP = 2.0 ** -3
TORCH_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
LARGEST = 8192 * 151936 * 1536


def listed():
    return [
        # one decode step of one request on the 32000-entry head: latency
        {"name": "score one token", "op": "score", "B": 1, "V": 32000, "d": 2048, "K": 8,
         "dtype": "bf16", "T": 1.0, "masked": 0.0},
        # a serving batch that returns 20 alternatives a token
        {"name": "score serving batch", "op": "score", "B": 32, "V": 152064, "d": 3584, "K": 20,
         "dtype": "bf16", "T": 0.7, "masked": 0.0},
        # a prompt scored on a head whose sizes are multiples of no tile
        {"name": "score ragged prompt", "op": "score", "B": 301, "V": 50001, "d": 1000, "K": 5,
         "dtype": "fp16", "T": 1.0, "masked": 0.1},
        # a trainer's batch of rollout tokens
        {"name": "score trainer batch", "op": "score", "B": 8192, "V": 151936, "d": 1536, "K": 8,
         "dtype": "bf16", "T": 1.0, "masked": 0.1},
        # the gradient of a few tokens: both weight-sized passes dominate
        {"name": "gradient few tokens", "op": "gradient", "B": 48, "V": 32000, "d": 2048,
         "dtype": "bf16", "T": 1.0, "masked": 0.0, "entropy": False},
        # a ragged micro-batch in fp16 with a loss scale
        {"name": "gradient ragged batch", "op": "gradient", "B": 777, "V": 50001, "d": 1000,
         "dtype": "fp16", "T": 0.9, "masked": 0.2, "entropy": True},
        # the trainer's batch: log-probability and entropy bonus
        {"name": "gradient trainer batch", "op": "gradient", "B": 8192, "V": 151936, "d": 1536,
         "dtype": "bf16", "T": 1.0, "masked": 0.1, "entropy": True},
        # one decode step of the int8 head, logits for a sampler
        {"name": "int8 one token", "op": "int8", "B": 1, "V": 128256, "d": 4096, "out": "f32"},
        # a decode batch
        {"name": "int8 decode batch", "op": "int8", "B": 32, "V": 128256, "d": 4096, "out": "bf16"},
        # ragged sizes, fp16 logits
        {"name": "int8 ragged batch", "op": "int8", "B": 205, "V": 50001, "d": 1040, "out": "fp16"},
        # a prompt's logits at every position
        {"name": "int8 prompt", "op": "int8", "B": 2048, "V": 128256, "d": 4096, "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("score", "gradient", "int8"))
    step = 16 if op == "int8" else 8
    while True:
        B, V = _log_int(rng, 1, 8192), _log_int(rng, 500, 152064)
        d = step * _log_int(rng, 64 // step, 4096 // step)
        if B * V * d <= LARGEST // (4 if op == "int8" else 1):
            break
    if op == "int8":
        return {"op": op, "B": B, "V": V, "d": d, "out": rng.choice(("f32", "bf16", "fp16"))}
    case = {"op": op, "B": B, "V": V, "d": d, "dtype": rng.choice(("bf16", "bf16", "fp16")),
            "T": rng.choice((1.0, 1.0, 0.6, 1.3)), "masked": rng.choice((0.0, 0.1, 0.5))}
    if op == "score":
        case["K"] = rng.choice((0, 1, 2, 5, 8, 13, 20, 32))
    else:
        case["entropy"] = rng.choice((True, False))
    return case


# ------------------------------------------------------------------- inputs
def _grid(gen, shape, sigma, most):
    x = torch.randn(shape, generator=gen, device="cuda")
    return x.mul_(sigma).round_().clamp_(-most, most)


def _float_inputs(case, seed):
    """W and h on the grid; each hidden row leans, by a random amount, to the
    token it is scored with, as a trained head's rows do (its probability
    ranges from that of any other token to about a third)."""
    B, V, d = case["B"], case["V"], case["d"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = TORCH_DTYPES[case["dtype"]]
    w_step = 2.0 ** -round(math.log2(math.sqrt(d) * 16 / 2.5))   # logits of deviation about 2.5
    W = _grid(gen, (V, d), 16.0, 63.0)
    targets = torch.randint(V, (B,), generator=gen, device="cuda", dtype=torch.int32)
    most = (math.log(V) + 1.0) * case["T"] / (H_STEP * w_step * d * 16.0 ** 2)
    lean = torch.rand((B, 1), generator=gen, device="cuda") * most
    h = torch.randn((B, d), generator=gen, device="cuda") * 8.0 + lean * W[targets.long()]
    h = h.round_().clamp_(-31.0, 31.0)
    gone = torch.rand((B,), generator=gen, device="cuda") < case["masked"]
    targets = torch.where(gone, torch.full_like(targets, NO_TARGET), targets)
    return (W * w_step).to(dt), (h * H_STEP).to(dt), targets, gen


def _loss_gradients(case, gen):
    """Gradients of a policy objective averaged over the batch: an advantage a
    token, an entropy bonus; fp16 training multiplies the loss by a scale."""
    B = case["B"]
    scale = (16384.0 if case["dtype"] == "fp16" else 1.0) / B
    dlogp = torch.randn((B,), generator=gen, device="cuda") * scale
    dentropy = None
    if case["entropy"]:
        dentropy = (0.5 + torch.rand((B,), generator=gen, device="cuda")) * (-0.05 * scale)
    return dlogp, dentropy


def _int8_inputs(case, seed):
    B, V, d = case["B"], case["V"], case["d"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def rows(n, sigma):
        x = torch.randn((n, d), generator=gen, device="cuda") * sigma
        scale = x.abs().amax(dim=1) / 127.0
        return (x / scale[:, None]).round_().clamp_(-127, 127).to(torch.int8), scale

    q, x_scale = rows(B, 1.0)
    Wq, w_scale = rows(V, 0.02)
    return q, x_scale, Wq, w_scale


def prepare(case, seed):
    state = {"case": case}
    if case["op"] == "int8":
        q, x_scale, Wq, w_scale = _int8_inputs(case, seed)
        state.update(q=q, x_scale=x_scale, W=Wq, w_scale=w_scale)
    else:
        W, h, targets, gen = _float_inputs(case, seed)
        state.update(W=W, h=h, targets=targets)
        if case["op"] == "gradient":
            # what the scoring call of the same step left behind
            dlogp, dentropy = _loss_gradients(case, gen)
            stats = _plain_stats(_plain_logits(h, W) / case["T"])[0]
            state.update(dlogp=dlogp, dentropy=dentropy, lse=stats["lse"],
                         entropy=stats["entropy"])
    if own:
        from invariant_output_head_gb300 import Head
        head = Head(state["W"])
        state["head"] = head
        if case["op"] == "score":
            head.reserve_score(case["B"], case["K"])
            state["out"] = head.score_buffers(case["B"], case["K"])
        elif case["op"] == "gradient":
            head.reserve_backward(case["B"])
            state["out"] = (torch.empty_like(state["h"]), torch.empty_like(state["W"]))
        else:
            head.reserve(case["B"])
            state["out"] = torch.empty((case["B"], case["V"]), device="cuda",
                                       dtype=TORCH_DTYPES[case["out"]])
    return state


# --------------------------------------------------------------- plain forms
def _plain_logits(h, W):
    return h.float() @ W.float().t()


def _plain_stats(z):
    m = z.amax(dim=1, keepdim=True)
    t = z - m
    e = torch.exp(t)
    s = e.sum(dim=1)
    u = (e * t).sum(dim=1)
    log_s = torch.log(s)
    return {"lse": m[:, 0] + log_s, "entropy": log_s - u / s}, m, log_s[:, None]


def _plain_top(z, K):
    """The K largest of each row, the lowest index first among equal ones: the
    order of the value's bits (as a signed number) over the reversed index."""
    bits = (z + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    last = torch.arange(z.shape[1], device=z.device).neg_().add_(0x7FFFFFFF)
    key = (order << 32) + last
    return 0x7FFFFFFF - (key.topk(K, dim=1).values & 0x7FFFFFFF)


def _plain_score(s):
    case = s["case"]
    raw = _plain_logits(s["h"], s["W"])
    z = raw / case["T"]
    out, m, log_s = _plain_stats(z)
    t = s["targets"].long()
    logp = (z.gather(1, t.clamp_min(0)[:, None]) - m - log_s)[:, 0]
    out["logp"] = torch.where(t >= 0, logp, torch.zeros_like(logp))
    if case["K"]:
        top = _plain_top(raw, case["K"])
        out["top_token"] = top.int()
        out["top_logp"] = z.gather(1, top) - m - log_s
    return out


def _plain_gradient(s):
    case = s["case"]
    h, W, t = s["h"].float(), s["W"].float(), s["targets"].long()
    logp = (h @ W.t()) / case["T"] - s["lse"][:, None]
    gl = torch.where(t >= 0, s["dlogp"], torch.zeros_like(s["dlogp"]))
    p = torch.exp(logp)
    if s["dentropy"] is None:
        dz = p * -gl[:, None]
    else:
        dz = -p * (gl[:, None] + s["dentropy"][:, None] * (logp + s["entropy"][:, None]))
    dz.scatter_add_(1, t.clamp_min(0)[:, None], gl[:, None])
    dz = dz / case["T"]
    return {"dh": (dz @ W).to(s["h"].dtype), "dW": (dz.t() @ h).to(s["W"].dtype)}


def _plain_int8(s):
    acc = s["q"].float() @ s["W"].float().t()
    y = acc * (s["x_scale"][:, None] * s["w_scale"][None, :])
    return y.to(TORCH_DTYPES[s["case"]["out"]])


def run(state):
    case = state["case"]
    if own:
        head = state["head"]
        if case["op"] == "score":
            r = head.score(state["h"], state["targets"], top_k=case["K"], temperature=case["T"],
                           out=state["out"])
            out = {"lse": r.lse, "entropy": r.entropy, "logp": r.logp}
            if case["K"]:
                out["top_token"], out["top_logp"] = r.top_token, r.top_logp
            return out
        if case["op"] == "gradient":
            dh, dW = head.score_backward(state["h"], state["targets"], state["lse"],
                                         state["entropy"], state["dlogp"], state["dentropy"],
                                         temperature=case["T"], out=state["out"])
            return {"dh": dh, "dW": dW}
        return head.scaled_logits(state["q"], state["x_scale"], state["w_scale"],
                                  out=state["out"])
    if case["op"] == "score":
        return _plain_score(state)
    return _plain_gradient(state) if case["op"] == "gradient" else _plain_int8(state)


def work(case):
    B, V, d = case["B"], case["V"], case["d"]
    product = 2.0 * B * V * d
    if case["op"] == "int8":
        size = 4 if case["out"] == "f32" else 2
        return {"bytes": V * d + B * d + 4 * (V + B) + size * B * V, "flops": product}
    operands = 2 * (V + B) * d
    if case["op"] == "score":
        return {"bytes": operands + 4 * B * (1 + 3 + 2 * case["K"]), "flops": product}
    # the logits again, then one product for each gradient
    return {"bytes": 2 * operands + 4 * B * (5 if case["entropy"] else 3), "flops": 3 * product}


# ------------------------------------------------------------------ 64 bits
def _blocks(case):
    rows = max(1, min(case["B"], (1 << 27) // case["V"]))
    return [slice(i, min(i + rows, case["B"])) for i in range(0, case["B"], rows)]


def _exact_score(case, seed):
    W, h, targets, _ = _float_inputs(case, seed)
    W64 = W.double().t().contiguous()
    parts = []
    for rows in _blocks(case):
        z = torch.matmul(h[rows].double(), W64).div_(case["T"])
        lse = torch.logsumexp(z, dim=1)
        logp = z - lse[:, None]
        t = targets[rows].long()
        at = torch.arange(len(t), device="cuda")
        got = {"lse": lse, "entropy": -(logp.exp() * logp).sum(dim=1),
               "logp": torch.where(t < 0, 0.0, logp[at, t.clamp(min=0)])}
        if case["K"]:
            ids, values = [], []
            for _ in range(case["K"]):
                best = logp.argmax(dim=1)
                ids.append(best)
                values.append(logp[at, best])
                logp[at, best] = -math.inf
            got["top_token"] = torch.stack(ids, dim=1).int()
            got["top_logp"] = torch.stack(values, dim=1)
        parts.append(got)
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_gradient(case, seed):
    W, h, targets, gen = _float_inputs(case, seed)
    dlogp, dentropy = _loss_gradients(case, gen)
    W64 = W.double()
    dW = torch.zeros_like(W64)
    dh = torch.empty(h.shape, dtype=torch.float64, device="cuda")
    for rows in _blocks(case):
        h64 = h[rows].double()
        logp = torch.log_softmax((h64 @ W64.t()) / case["T"], dim=1)
        p = logp.exp()
        t = targets[rows].long()
        has = (t >= 0).double()
        g = dlogp[rows].double() * has
        onehot = torch.zeros_like(p)
        onehot[torch.arange(len(t), device="cuda"), t.clamp(min=0)] = has
        dz = g[:, None] * (onehot - p)
        if dentropy is not None:
            H = -(p * logp).sum(dim=1, keepdim=True)
            dz -= dentropy[rows].double()[:, None] * p * (logp + H)
        dz /= case["T"]
        dh[rows] = dz @ W64
        dW += dz.t() @ h64
    return {"dh": dh, "dW": dW}


def _exact_int8(case, seed):
    q, x_scale, Wq, w_scale = _int8_inputs(case, seed)
    W64 = Wq.double().t().contiguous()
    out = torch.empty((case["B"], case["V"]), dtype=torch.float64, device="cuda")
    for rows in _blocks(case):
        out[rows] = (q[rows].double() @ W64) * x_scale[rows].double()[:, None]
    return out * w_scale.double()[None, :]


def exact(case, seed):
    if case["op"] == "int8":
        return _exact_int8(case, seed)
    return _exact_score(case, seed) if case["op"] == "score" else _exact_gradient(case, seed)
