"""Cases of the operators of a beam-search step on an 8-bit floating-point
head: rows and weights quantised to e4m3 with a scale for each block of 128,
the logits of such a head, the selection over beams and vocabulary, and the
reordering of the beams' states.

Each case is one call of one operator. `run` computes it in plain torch
operations, or, where `own` is true, through the package's public calls.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TORCH_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
# the costliest listed case of each operator, in the unit of its own size
LARGEST = {"quantize": 128256 * 4096, "logits": 2048 * 128256 * 4096, "select": 512 * 128256,
           "reorder": 8 * 256 * 8 * 511 * 128}
CLOSE = 1e-4          # scores of different beams are at least this far apart


def listed():
    return [
        # the hidden rows of one decode batch: latency
        {"name": "quantise decode rows", "op": "quantize", "B": 32, "d": 4096, "dtype": "bf16",
         "rows": 1, "gone": 0.0},
        # a prompt's rows in fp32, d a multiple of no block, some blocks empty
        {"name": "quantise ragged prompt", "op": "quantize", "B": 5001, "d": 1040, "dtype": "f32",
         "rows": 1, "gone": 0.02},
        # a head's weight, once when it is loaded
        {"name": "quantise weight", "op": "quantize", "B": 128256, "d": 4096, "dtype": "bf16",
         "rows": 128, "gone": 0.0},
        # one decode step of one request on the 32000-entry head: latency
        {"name": "logits one token", "op": "logits", "B": 1, "V": 32000, "d": 2048, "out": "f32"},
        # four requests of eight beams
        {"name": "logits decode batch", "op": "logits", "B": 32, "V": 128256, "d": 4096,
         "out": "bf16"},
        # sizes that are multiples of no tile, fp16 logits
        {"name": "logits ragged batch", "op": "logits", "B": 205, "V": 50001, "d": 1040,
         "out": "fp16"},
        # a prompt's logits at every position
        {"name": "logits prompt", "op": "logits", "B": 2048, "V": 128256, "d": 4096, "out": "bf16"},
        # one request of four beams: latency
        {"name": "select one request", "op": "select", "N": 1, "beams": 4, "V": 32000, "n_out": 8,
         "dtype": "f32", "T": 1.0, "masked": 0.0, "finished": False},
        # a few requests with constrained vocabularies and finished beams
        {"name": "select ragged batch", "op": "select", "N": 7, "beams": 5, "V": 50001, "n_out": 10,
         "dtype": "fp16", "T": 0.8, "masked": 0.3, "finished": True},
        # a serving batch
        {"name": "select serving batch", "op": "select", "N": 64, "beams": 8, "V": 128256,
         "n_out": 16, "dtype": "bf16", "T": 1.0, "masked": 0.0, "finished": False},
        # one request's caches after a step
        {"name": "reorder one request", "op": "reorder", "N": 1, "beams": 4, "L": 8, "H": 4,
         "length": 77, "room": 128, "D": 64, "dtype": "bf16"},
        # a serving batch's caches, the used part of rows with room for more
        {"name": "reorder serving batch", "op": "reorder", "N": 32, "beams": 8, "L": 8, "H": 8,
         "length": 511, "room": 600, "D": 128, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantize", "logits", "logits", "select", "select", "reorder"))
    if op == "quantize":
        while True:
            B, d = _log_int(rng, 1, 128256), 16 * _log_int(rng, 4, 512)
            if B * d <= LARGEST[op]:
                break
        return {"op": op, "B": B, "d": d, "dtype": rng.choice(("bf16", "fp16", "f32")),
                "rows": rng.choice((1, 1, 128)), "gone": rng.choice((0.0, 0.02, 0.3))}
    if op == "logits":
        while True:
            B, V = _log_int(rng, 1, 4096), _log_int(rng, 500, 152064)
            d = 16 * _log_int(rng, 4, 512)
            if B * V * d <= LARGEST[op]:
                break
        return {"op": op, "B": B, "V": V, "d": d, "out": rng.choice(("f32", "bf16", "fp16"))}
    beams = rng.choice((1, 2, 3, 4, 5, 8, 12, 16, 32))
    if op == "select":
        while True:
            N, V = _log_int(rng, 1, 256), _log_int(rng, 1000, 152064)
            if N * beams * V <= LARGEST[op]:
                break
        return {"op": op, "N": N, "beams": beams, "V": V,
                "n_out": rng.choice((beams, min(64, 2 * beams), rng.randint(1, 64))),
                "dtype": rng.choice(("f32", "bf16", "fp16")), "T": rng.choice((1.0, 1.0, 0.7, 1.3)),
                "masked": rng.choice((0.0, 0.3, 0.9)), "finished": rng.choice((True, False))}
    while True:
        N, L, H = _log_int(rng, 1, 64), rng.randint(1, 16), rng.choice((1, 2, 4, 8))
        length, D = _log_int(rng, 1, 2000), rng.choice((32, 64, 80, 128))
        if N * beams * L * H * length * D <= LARGEST[op]:
            break
    return {"op": op, "N": N, "beams": beams, "L": L, "H": H, "length": length,
            "room": length + rng.randint(0, 100), "D": D, "dtype": rng.choice(("bf16", "fp16", "f32"))}


# ------------------------------------------------------------------- inputs
def _generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def _quantize_inputs(case, seed):
    """Rows of their own size, a few channels far larger than the others (as
    hidden rows have them), and blocks with nothing in them."""
    B, d, gen = case["B"], case["d"], _generator(seed)
    x = torch.randn((B, d), generator=gen, device="cuda")
    x *= torch.exp2(torch.rand((B, 1), generator=gen, device="cuda") * 8.0 - 4.0)
    x *= torch.where(torch.rand((d,), generator=gen, device="cuda") < 0.01, 30.0, 1.0)
    if case["gone"]:
        full = torch.rand((B, -(-d // BLOCK)), generator=gen, device="cuda") >= case["gone"]
        x *= full.repeat_interleave(BLOCK, dim=1)[:, :d]
    return x.to(TORCH_DTYPES[case["dtype"]])


def _to_blocks(x, rows):
    """x in e4m3 with the scale amax / 448 for each block of rows x 128, as
    checkpoints hold them."""
    n, d = x.shape
    nb, db = -(-n // rows), -(-d // BLOCK)
    x = torch.nn.functional.pad(x, (0, db * BLOCK - d, 0, nb * rows - n))
    blocks = x.view(nb, rows, db, BLOCK)
    scale = blocks.abs().amax(dim=(1, 3)).clamp_min(1e-30) / E4M3_MAX
    q = (blocks / scale[:, None, :, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(nb * rows, db * BLOCK)[:n, :d].contiguous(), scale


def _logits_inputs(case, seed):
    B, V, d, gen = case["B"], case["V"], case["d"], _generator(seed)
    x = torch.randn((B, d), generator=gen, device="cuda")
    x *= torch.where(torch.rand((d,), generator=gen, device="cuda") < 0.01, 10.0, 1.0)
    W = torch.randn((V, d), generator=gen, device="cuda")
    W *= torch.exp2(torch.rand((V, 1), generator=gen, device="cuda") - 0.5) * (2.0 / math.sqrt(d))
    q, x_scale = _to_blocks(x, 1)
    W, w_scale = _to_blocks(W, BLOCK)
    return q, x_scale, W, w_scale


def _near(case, logits, scores, finished):
    """The sequences in which two candidates of different beams come within
    CLOSE of each other among the n_out + 1 best (64 bits)."""
    N, beams, n = case["N"], case["beams"], case["n_out"] + 1
    z = logits.double() / case["T"]
    best = z.topk(min(n, case["V"]), dim=1).values - z.logsumexp(dim=1, keepdim=True)
    best = best.view(N, beams, -1)
    if finished is not None:
        best = torch.where(finished[:, :, None], -math.inf, best)
        best[:, :, 0] = torch.where(finished, 0.0, best[:, :, 0])
    best = best + scores.double()[:, :, None]
    beam = torch.arange(beams, device="cuda")[None, :, None].expand_as(best).reshape(N, -1)
    best, order = best.reshape(N, -1).sort(dim=1, descending=True)
    beam = beam.gather(1, order)[:, :n]
    gap = best[:, :n - 1] - best[:, 1:n]
    # (no other candidate is as near as these to the ones chosen, but for ties
    # of one beam, whose order the logits give)
    return ((gap < CLOSE) & (beam[:, :-1] != beam[:, 1:])).any(dim=1)


def _select_inputs(case, seed):
    """Logits of a trained model's spread, some tokens ruled out (with -inf, or
    with the type's lowest value), beams in falling order of their scores, one
    of them dead now and then. Logits lie on a grid, so ties within a beam are
    real ones; scores of a sequence whose beams would tie within what 32 bits
    resolve are drawn again."""
    N, beams, V, gen = case["N"], case["beams"], case["V"], _generator(seed)
    dt = TORCH_DTYPES[case["dtype"]]
    logits = torch.randn((N * beams, V), generator=gen, device="cuda").mul_(2.5 * 1024).round_()
    logits = logits.div_(1024).to(dt)
    if case["masked"]:
        gone = torch.rand((N * beams, V), generator=gen, device="cuda") < case["masked"]
        worst = torch.full((N * beams, 1), torch.finfo(dt).min, dtype=dt, device="cuda")
        worst[::2] = -math.inf
        logits = torch.where(gone, worst, logits)
    finished = None
    if case["finished"]:
        finished = torch.rand((N, beams), generator=gen, device="cuda") < 0.25

    def fresh():
        s = -3.0 * torch.rand((N, beams), generator=gen, device="cuda") - 5.0
        dead = torch.rand((N, beams), generator=gen, device="cuda") < 0.05
        dead[:, 0] = False
        return torch.where(dead, -math.inf, s.sort(dim=1, descending=True).values)

    scores = fresh()
    for _ in range(64):
        near = _near(case, logits, scores, finished)
        if not bool(near.any()):
            break
        scores = torch.where(near[:, None], fresh(), scores)
    return logits, scores, finished


def _reorder_inputs(case, seed):
    N, beams, gen = case["N"], case["beams"], _generator(seed)
    rows, shape = N * beams, (N * beams, case["H"], case["room"], case["D"])
    dt = TORCH_DTYPES[case["dtype"]]
    caches = [torch.randn(shape, generator=gen, device="cuda", dtype=dt) for _ in range(case["L"])]
    tokens = torch.randint(32000, (rows, case["room"]), generator=gen, device="cuda",
                           dtype=torch.int32)
    parent = torch.randint(beams, (N, beams), generator=gen, device="cuda", dtype=torch.int32)
    return caches, tokens, parent


def prepare(case, seed):
    state = {"case": case}
    if case["op"] == "quantize":
        state["x"] = _quantize_inputs(case, seed)
    elif case["op"] == "logits":
        q, x_scale, W, w_scale = _logits_inputs(case, seed)
        state.update(q=q, x_scale=x_scale, W=W, w_scale=w_scale)
    elif case["op"] == "select":
        logits, scores, finished = _select_inputs(case, seed)
        state.update(logits=logits, scores=scores, finished=finished)
    else:
        caches, tokens, parent = _reorder_inputs(case, seed)
        # the other half of a double buffer, rows that have not been written yet
        state.update(src=caches + [tokens], parent=parent,
                     dst=[torch.zeros_like(c) for c in caches + [tokens]])
    if own:
        _own_prepare(state)
    return state


def _own_prepare(state):
    """The heads, reserved workspaces and output buffers that a serving loop
    keeps."""
    from invariant_output_head_gb300 import BeamStates, Head, beam_buffers, block_buffers
    case = state["case"]
    if case["op"] == "quantize":
        state["out"] = block_buffers(case["B"], case["d"], case["rows"], device="cuda")
    elif case["op"] == "logits":
        state["head"] = Head(state["W"])
        state["out"] = torch.empty((case["B"], case["V"]), device="cuda",
                                   dtype=TORCH_DTYPES[case["out"]])
    elif case["op"] == "select":
        # the head whose logits these are: its weight is not read by this call
        state["head"] = Head(torch.zeros((case["V"], 16), dtype=torch.bfloat16, device="cuda"))
        state["head"].reserve_beams(case["N"] * case["beams"], case["n_out"])
        state["out"] = beam_buffers(case["N"], case["n_out"], device="cuda")
    else:
        state["states"] = BeamStates(state["src"], out=state["dst"],
                                     token_dim=[2] * case["L"] + [1])


# --------------------------------------------------------------- plain forms
def _plain_quantize(s):
    rows, x = s["case"]["rows"], s["x"].float()
    n, d = x.shape
    nb, db = -(-n // rows), -(-d // BLOCK)
    x = torch.nn.functional.pad(x, (0, db * BLOCK - d, 0, nb * rows - n)).view(nb, rows, db, BLOCK)
    amax = x.abs().amax(dim=(1, 3))
    m, e = torch.frexp(amax)             # amax = m 2^e, 1/2 <= m < 1; 448 = 0.875 2^9
    e = (e - 9 + (m > 0.875).int()).clamp_min(-126)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))
    q = (x / scale[:, None, :, None]).to(torch.float8_e4m3fn)
    return {"q": q.view(nb * rows, db * BLOCK)[:n, :d].contiguous(), "scale": scale}


def _plain_logits(s):
    case = s["case"]
    B, V, d = case["B"], case["V"], case["d"]
    x = s["q"].float() * s["x_scale"].repeat_interleave(BLOCK, dim=1)[:, :d]
    W = s["W"].float() * s["w_scale"].repeat_interleave(BLOCK, dim=1)[:, :d].repeat_interleave(
        BLOCK, dim=0)[:V]
    return (x @ W.t()).to(TORCH_DTYPES[case["out"]])


def _plain_select(s):
    case = s["case"]
    N, beams, V, n = case["N"], case["beams"], case["V"], case["n_out"]
    raw = s["logits"].float()
    z = raw / case["T"]
    m = z.amax(dim=1, keepdim=True)
    log_s = torch.log(torch.exp(z - m).sum(dim=1, keepdim=True))
    # each beam's best: the order of the logit's bits over the reversed index
    bits = (raw + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    key = (order << 32) + torch.arange(V, device="cuda").neg_().add_(0x7FFFFFFF)
    k = min(n, V)
    token = 0x7FFFFFFF - (key.topk(k, dim=1).values & 0x7FFFFFFF)
    score = (z.gather(1, token) - m - log_s).view(N, beams, k) + s["scores"][:, :, None]
    token = token.view(N, beams, k)
    if s["finished"] is not None:
        first = torch.arange(k, device="cuda") == 0
        done = torch.where(first, s["scores"][:, :, None], -math.inf)
        score = torch.where(s["finished"][:, :, None], done, score)
        token = torch.where(s["finished"][:, :, None], END, token)
    # every place has a candidate or -inf, which stands for none
    pad = max(0, n - beams * k)
    score = torch.nn.functional.pad(score.reshape(N, -1), (0, pad), value=-math.inf)
    token = torch.nn.functional.pad(token.reshape(N, -1), (0, pad))
    score, at = score.sort(dim=1, descending=True, stable=True)
    score, at = score[:, :n].contiguous(), at[:, :n]
    none = score == -math.inf
    parent = torch.where(none, -1, at // k)
    token = torch.where(none, -1, token.gather(1, at))
    return {"parent": parent.int(), "token": token.int(), "score": score}


END = 2               # the end token that finished beams propose


def _plain_reorder(s):
    case = s["case"]
    N, beams, length = case["N"], case["beams"], case["length"]
    first = torch.arange(0, N * beams, beams, device="cuda")[:, None]
    row = (s["parent"] + first).view(-1)
    for c, d in zip(s["src"][:-1], s["dst"][:-1]):
        d[..., :length, :] = c[..., :length, :].index_select(0, row)
    s["dst"][-1][:, :length] = s["src"][-1][:, :length].index_select(0, row)
    return s["dst"]


PLAIN = {"quantize": _plain_quantize, "logits": _plain_logits, "select": _plain_select,
         "reorder": _plain_reorder}


def run(state):
    case = state["case"]
    if not own:
        return PLAIN[case["op"]](state)
    if case["op"] == "quantize":
        from invariant_output_head_gb300 import quantize_blocks
        q, scale = quantize_blocks(state["x"], case["rows"], out=state["out"])
        return {"q": q, "scale": scale}
    if case["op"] == "logits":
        return state["head"].block_scaled_logits(state["q"], state["x_scale"], state["w_scale"],
                                                 out=state["out"])
    if case["op"] == "select":
        r = state["head"].beam_select(state["logits"], state["scores"], case["n_out"],
                                      temperature=case["T"], finished=state["finished"],
                                      end_token=END, out=state["out"])
        return {"parent": r.parent, "token": r.token, "score": r.score}
    state["states"].reorder(state["parent"], used=case["length"])
    return state["dst"]


def work(case):
    size = {"bf16": 2, "fp16": 2, "f32": 4}
    if case["op"] == "quantize":
        n = case["B"] * case["d"]
        scales = -(-case["B"] // case["rows"]) * -(-case["d"] // BLOCK)
        return {"bytes": n * (size[case["dtype"]] + 1) + 4 * scales, "flops": 2.0 * n}
    if case["op"] == "logits":
        B, V, d = case["B"], case["V"], case["d"]
        scales = -(-d // BLOCK) * (B + -(-V // BLOCK))
        return {"bytes": (V + B) * d + 4 * scales + size[case["out"]] * B * V,
                "flops": 2.0 * B * V * d}
    if case["op"] == "select":
        rows = case["N"] * case["beams"]
        return {"bytes": size[case["dtype"]] * rows * case["V"] + 4 * rows
                + 12 * case["N"] * case["n_out"], "flops": 3.0 * rows * case["V"]}
    row = case["L"] * case["H"] * case["length"] * case["D"] * size[case["dtype"]] + 4 * case["length"]
    return {"bytes": case["N"] * case["beams"] * (2 * row + 4), "flops": 0}


# ------------------------------------------------------------------ 64 bits
def _exact_quantize(case, seed):
    """Blocks by index, the exponent by comparing with powers of two, and the
    rounding to a 3-bit fraction as a multiple of the step at that exponent."""
    x, rows = _quantize_inputs(case, seed), case["rows"]
    B, d = x.shape
    nb, db = -(-B // rows), -(-d // BLOCK)
    scale = torch.empty((nb, db), dtype=torch.float64, device="cuda")
    q = torch.empty((B, d), dtype=torch.float64, device="cuda")
    for j in range(db):
        part = x[:, j * BLOCK:(j + 1) * BLOCK].double()
        most = part.abs().amax(dim=1)
        top = torch.zeros(nb, dtype=torch.float64, device="cuda")
        top.scatter_reduce_(0, torch.arange(B, device="cuda") // rows, most, "amax")
        e = torch.ceil(torch.log2(torch.where(top > 0, top, E4M3_MAX) / E4M3_MAX))
        e = torch.where(top <= E4M3_MAX * torch.exp2(e - 1), e - 1, e)
        e = torch.where(top > E4M3_MAX * torch.exp2(e), e + 1, e).clamp_min(-126)
        s = torch.where(top > 0, torch.exp2(e), 1.0)
        scale[:, j] = s
        y = part / s.repeat_interleave(rows)[:B, None]
        a = y.abs()
        step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
        q[:, j * BLOCK:(j + 1) * BLOCK] = torch.round(y / step) * step
    return {"q": q, "scale": scale}


def _exact_logits(case, seed):
    q, x_scale, W, w_scale = _logits_inputs(case, seed)
    B, V, d = case["B"], case["V"], case["d"]
    out = torch.zeros((B, V), dtype=torch.float64, device="cuda")
    for c in range(-(-d // BLOCK)):
        k = slice(c * BLOCK, (c + 1) * BLOCK)
        left = q[:, k].double() * x_scale[:, c].double()[:, None]
        right = W[:, k].double() * w_scale[:, c].double().repeat_interleave(BLOCK)[:V, None]
        out += left @ right.t()
    return out


def _exact_select(case, seed):
    logits, scores, finished = _select_inputs(case, seed)
    N, beams, V, n = case["N"], case["beams"], case["V"], case["n_out"]
    parts = {"parent": [], "token": [], "score": []}
    for i in range(N):
        z = logits[i * beams:(i + 1) * beams].double() / case["T"]
        total = torch.log_softmax(z, dim=1) + scores[i].double()[:, None]
        if finished is not None:
            total[finished[i]] = -math.inf
            total[finished[i], END] = scores[i].double()[finished[i]]
        total = total.view(-1)
        # more than are wanted, then the lowest index first among equal ones
        value, index = total.topk(min(n, total.numel()))
        index = torch.nonzero(total >= value[-1])[:, 0]
        value = total[index]
        if value.numel() < n:
            value = torch.cat([value, value.new_full((n - value.numel(),), -math.inf)])
            index = torch.cat([index, index.new_zeros(n - index.numel())])
        value, order = value.sort(descending=True, stable=True)
        value, index = value[:n], index[order][:n]
        none = value == -math.inf
        parts["parent"].append(torch.where(none, -1, index // V))
        parts["token"].append(torch.where(none, -1, index % V))
        parts["score"].append(value)
    got = {k: torch.stack(v) for k, v in parts.items()}
    return {"parent": got["parent"].int(), "token": got["token"].int(), "score": got["score"]}


def exact(case, seed):
    if case["op"] == "quantize":
        return _exact_quantize(case, seed)
    if case["op"] == "logits":
        return _exact_logits(case, seed)
    return _exact_select(case, seed) if case["op"] == "select" else None
