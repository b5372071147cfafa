"""Beam selection and the reordering of states against plain forms."""
import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def t():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def head_of(t, V):
    from invariant_output_head_gb300 import Head
    return Head(t.zeros(V, 16, dtype=t.bfloat16, device="cuda"))


def dtype_of(t, name):
    return {"f32": t.float32, "bf16": t.bfloat16, "fp16": t.float16}[name]


def step_inputs(t, n_seq, beams, V, name, seed):
    """Logits on a grid of 2^-8 (ties of a beam are real ones) and scores whose
    beams' candidates lie apart: multiples of an irrational step."""
    g = t.Generator().manual_seed(seed)
    z = (t.randn(n_seq * beams, V, generator=g) * 2.5 * 256).round() / 256
    s = -t.rand(n_seq, beams, generator=g) * 4 - 3
    return z.to(dtype_of(t, name)), s


def check(t, head, z, s, n_out, T=1.0, finished=None, end=0):
    """The call against the sorted candidates. Two candidates of different beams
    whose scores are nearer than their bounds may come in either order."""
    from tests import block_ref
    got = head.beam_select(z.cuda(), s.cuda(), n_out, temperature=T, end_token=end,
                           finished=None if finished is None else finished.cuda())
    assert head.check() == 0
    parent, token, score = (x.cpu() for x in got)
    want_p, want_t, want_s = block_ref.select(z, s, n_out, T, finished, end)
    zf = z.float()
    live = zf[zf.isfinite()]
    spread = float(live.max() - live.min()) if len(live) else 0.0
    near = block_ref.score_tol(want_s.abs().nan_to_num(posinf=0.0), float(s[s.isfinite()].abs().max())
                               if bool(s.isfinite().any()) else 0.0, spread, z.shape[1], T)
    assert t.equal(score == -math.inf, want_s == -math.inf)
    real = want_s > -math.inf
    assert bool(((score.double() - want_s).abs() <= near)[real].all())
    same = (parent == want_p) & (token == want_t)
    if not bool(same.all()):
        # where they differ, a candidate of another beam within both bounds
        for q, j in (~same).nonzero().tolist():
            p, v = int(parent[q, j]), int(token[q, j])
            own = block_ref.select(z[q * s.shape[1] + p][None], s[q, p].view(1, 1), z.shape[1], T)
            at = (own[1][0] == v).nonzero()[0, 0]
            assert abs(float(own[2][0, at] - want_s[q, j])) <= 2 * float(near[q, j])
            assert p != int(want_p[q, j])
    return got


@pytest.mark.parametrize("name", ["f32", "bf16", "fp16"])
@pytest.mark.parametrize("n_seq, beams, V, n_out", [
    (1, 1, 1, 1), (1, 1, 1, 5), (2, 3, 7, 64), (1, 4, 511, 8), (3, 2, 512, 4), (2, 5, 513, 10),
    (1, 4, 4096, 8), (2, 4, 4097, 64), (1, 32, 2000, 64), (5, 8, 9999, 16), (1, 1, 50001, 64),
    (1, 4, 32000, 8), (150, 5, 3001, 7), (700, 1, 1025, 3)])
def test_selection_against_64_bits(t, n_seq, beams, V, n_out, name):
    z, s = step_inputs(t, n_seq, beams, V, name, V + n_out)
    check(t, head_of(t, V), z, s, n_out)


@pytest.mark.parametrize("T", [0.3, 0.8, 1.7, 30.0])
def test_selection_at_a_temperature(t, T):
    z, s = step_inputs(t, 3, 4, 5000, "f32", 9)
    check(t, head_of(t, 5000), z, s, 12, T=T)


@pytest.mark.parametrize("name", ["f32", "bf16", "fp16"])
def test_masks_dead_beams_and_finished_ones(t, name):
    V = 9000
    z, s = step_inputs(t, 6, 4, V, name, 21)
    low = t.finfo(z.dtype).min
    z[0] = -math.inf                       # a row with nothing
    z[1, 1:] = -math.inf                   # one token
    z[2, :8000] = -math.inf                # whole tiles masked
    z[3, 100:] = low                       # the type's lowest value is a number
    z[4, 17], z[5, 8999] = math.nan, math.inf
    z[6, :] = low
    z[8:12] = -math.inf                    # a sequence with nothing at all
    s[1, 2], s[1, 3] = -math.inf, math.nan
    s[3, 0] = math.inf
    finished = t.zeros(6, 4, dtype=t.bool)
    finished[4, 1] = finished[5, 0] = finished[5, 1] = finished[5, 2] = finished[5, 3] = True
    s[5, 3] = -math.inf                    # finished and dead: nothing
    z[4 * 4 + 1, 5] = math.nan             # a finished beam's logits are not read
    head = head_of(t, V)
    got = check(t, head, z, s, 16, finished=finished, end=V - 1)
    assert got.parent[2].tolist() == [-1] * 16
    assert sorted(got.parent[5].tolist())[-3:] == [0, 1, 2] and got.token[5, 0] == V - 1
    check(t, head, z, s, 64)
    check(t, head, z, s, 9, finished=finished.to(t.uint8) * 200, end=3)
    assert head.check() == 0


@pytest.mark.parametrize("V", [600, 5000, 40000])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "two values", "zeros of both signs"])
def test_runs_of_equal_and_sorted_logits(t, V, kind):
    """More entries above any first threshold than the list holds."""
    z = {"equal": t.zeros(V) + 1.25, "rising": t.arange(V) / 64.0, "falling": -t.arange(V) / 64.0,
         "two values": (t.arange(V) % 2) * 2.0 - 1,
         "zeros of both signs": t.where(t.arange(V) % 3 == 0, -0.0, 0.0)}[kind]
    z = z[None].repeat(4, 1).float()
    z[2:] -= 0.5
    s = t.tensor([[-1.0, -1.3], [-2.0, -2.0]])
    for n_out in (1, 7, 64):
        got = check(t, head_of(t, V), z, s, n_out)
    if kind == "equal":
        assert got.token[0].tolist() == list(range(64)) and got.parent[1].tolist() == [0] * 64


def test_equal_beams_rank_by_beam(t):
    """The first step of a search: every beam the same, all but one unused."""
    z, _ = step_inputs(t, 1, 1, 3000, "f32", 4)
    z = z.repeat(4, 1)
    got = check(t, head_of(t, 3000), z, t.zeros(1, 4), 6)
    assert int((z[0] == z[0].max()).sum()) == 1 and got.parent[0, :4].tolist() == [0, 1, 2, 3]
    check(t, head_of(t, 3000), z, t.tensor([[0.0, -1e9, -1e9, -1e9]]), 6)


def test_a_sequences_bits_do_not_depend_on_its_batch(t):
    V = 20000
    z, s = step_inputs(t, 300, 3, V, "bf16", 5)
    z, s = z.cuda(), s.cuda()
    head = head_of(t, V)
    whole = head.beam_select(z, s, 9)
    for n in (1, 2, 40, 299):
        part = head.beam_select(z[:3 * n].contiguous(), s[:n].contiguous(), 9)
        for a, b in zip(part, whole):
            assert t.equal(a, b[:n]), n
    last = head.beam_select(z[-3:].contiguous(), s[-1:].contiguous(), 9)
    assert all(t.equal(a[0], b[-1]) for a, b in zip(last, whole))


@pytest.mark.parametrize("name", ["bf16", "fp16", "f32"])
def test_logits_at_any_address(t, name):
    V = 5001
    z, s = step_inputs(t, 2, 3, V, name, 6)
    head = head_of(t, V)
    want = head.beam_select(z.cuda(), s.cuda(), 11)
    for shift in (1, 2, 3):
        room = t.full((6 * V + 8,), 99.0, dtype=z.dtype, device="cuda")
        room[shift:shift + 6 * V] = z.cuda().view(-1)
        got = head.beam_select(room[shift:shift + 6 * V].view(6, V), s.cuda(), 11)
        assert all(t.equal(a, b) for a, b in zip(got, want)), shift


def test_scores_in_place_and_reserved_calls(t):
    V = 3000
    z, s = step_inputs(t, 5, 4, V, "f32", 8)
    head = head_of(t, V)
    head.reserve_beams(20, 8)
    want = head.beam_select(z.cuda(), s.cuda(), 4)
    scores = s.cuda()
    from invariant_output_head_gb300 import beam_buffers
    out = beam_buffers(5, 4, "cuda")._replace(score=scores)
    got = head.beam_select(z.cuda(), scores, 4, out=out)
    assert all(t.equal(a, b) for a, b in zip(got, want)) and got.score is scores


def test_selection_refusals(t):
    from invariant_output_head_gb300 import DetlmError
    V = 100
    z, s = step_inputs(t, 2, 3, V, "f32", 1)
    z, s = z.cuda(), s.cuda()
    head = head_of(t, V)
    done = t.zeros(2, 3, dtype=t.bool, device="cuda")
    for bad in (dict(n_out=0), dict(n_out=65), dict(temperature=0.0), dict(temperature=math.nan),
                dict(temperature=1e-39), dict(finished=done, end_token=100),
                dict(finished=done, end_token=-1)):
        with pytest.raises(DetlmError):
            head.beam_select(z, s, **(dict(n_out=4) | bad))
    with pytest.raises(DetlmError):
        head.beam_select(t.zeros(33, V, device="cuda"), t.zeros(1, 33, device="cuda"), 4)
    for args in ((-1, 4), (4, 0), (4, 65)):
        with pytest.raises(DetlmError):
            head.reserve_beams(*args)
    none = head.beam_select(z[:0], s[:0], 4)
    assert none.parent.shape == (0, 4)
    # a shard has part of the logits
    from invariant_output_head_gb300 import ShardHead
    shard = ShardHead(t.zeros(512, 16, dtype=t.bfloat16, device="cuda"), 1024, 2, 0)
    with pytest.raises(DetlmError):
        shard.beam_select(t.zeros(6, 512, device="cuda"), s, 4)
    with pytest.raises(DetlmError):
        shard.reserve_beams(6, 4)


# -------------------------------------------------------------------- reorder
def filled(t, shape, dtype, seed):
    g = t.Generator().manual_seed(seed)
    size = t.empty(0, dtype=dtype).element_size()
    raw = t.randint(0, 256, (*shape[:-1], shape[-1] * size), generator=g, dtype=t.uint8)
    return raw.view(dtype)


def same(t, a, b):
    return t.equal(a.contiguous().view(-1).view(t.uint8), b.contiguous().view(-1).view(t.uint8))


CASES = [   # rows' shape, token axis, type
    ((3, 20, 16), 2, "bfloat16"), ((20, 3, 16), 1, "float16"), ((37,), 1, "int32"), ((5, 7), 1, "uint8"),
    ((2, 9, 3), 2, "bfloat16"), ((4, 31, 80), 2, "float32"), ((1,), None, "float32"),
    ((6, 33), None, "int64"), ((2, 5, 11), 3, "int16"), ((3, 500, 64), 2, "float8_e4m3fn")]


@pytest.mark.parametrize("n_seq, beams", [(1, 1), (3, 4), (2, 7), (5, 8), (1, 13), (2, 32)])
@pytest.mark.parametrize("shape, dim, name", CASES)
def test_states_move_to_their_parents(t, shape, dim, name, n_seq, beams):
    from invariant_output_head_gb300 import BeamStates
    from tests import block_ref
    dtype = getattr(t, name)
    x = filled(t, (n_seq * beams, *shape), dtype, beams)
    raw = filled(t, (n_seq * beams, *shape), dtype, beams + 1)
    g = t.Generator().manual_seed(n_seq)
    parent = t.randint(-1, beams + 1, (n_seq, beams), generator=g, dtype=t.int32)
    positions = None if dim is None else shape[dim - 1]
    bits = {1: t.uint8, 2: t.int16, 4: t.int32, 8: t.int64}[x.element_size()]
    for used in (None, *({0, 1, positions // 2, positions} if positions else ())):
        want = block_ref.reorder(x.view(bits), raw.view(bits), parent, used, dim).view(dtype)
        dst = raw.cuda()
        BeamStates([x.cuda()], out=[dst], token_dim=dim).reorder(parent.cuda(), used=used)
        assert same(t, dst.cpu(), want), used
        want = block_ref.reorder(x.view(bits), x.view(bits), parent, used, dim).view(dtype)
        here = x.cuda()
        BeamStates([here], token_dim=dim).reorder(parent.cuda(), used=used)
        assert same(t, here.cpu(), want), used


def test_many_states_strided_ones_and_other_numbers_of_beams(t):
    from invariant_output_head_gb300 import BeamStates
    from tests import block_ref
    g = t.Generator().manual_seed(3)
    # keys and values in one tensor, moved in place beside each other
    both = t.randn(6, 2, 3, 10, 16, generator=g)
    parent = t.tensor([[2, 2, 0], [1, 0, 1]], dtype=t.int32)
    kv = both.cuda()
    BeamStates([kv[:, 0], kv[:, 1]], token_dim=2).reorder(parent.cuda(), used=4)
    want = both.clone()
    for i in range(2):
        want[:, i] = block_ref.reorder(both[:, i], both[:, i], parent, 4, 2)
    assert t.equal(kv.cpu(), want)
    # a prompt's state to the beams of the first step, and fewer beams after it
    one = t.randn(2, 5, 7, generator=g)
    many = t.zeros(8, 5, 7).cuda()
    BeamStates([one.cuda()], out=[many]).reorder(t.zeros(2, 4, dtype=t.int32).cuda())
    assert t.equal(many.cpu(), one.repeat_interleave(4, dim=0))
    few = t.zeros(4, 5, 7).cuda()
    src = t.randn(8, 5, 7, generator=g)
    pick = t.tensor([[3, 1], [0, 0]], dtype=t.int32)
    BeamStates([src.cuda()], out=[few]).reorder(pick.cuda())
    assert t.equal(few.cpu(), src[[3, 1, 4, 4]])
    # more states than a launch holds, of several grains
    xs = [filled(t, (12, 3 + i), t.uint8, i) for i in range(120)]
    parent = t.randint(0, 4, (3, 4), generator=g, dtype=t.int32)
    ys = [x.cuda() for x in xs]
    BeamStates(ys).reorder(parent.cuda())
    assert all(t.equal(y.cpu(), block_ref.reorder(x, x, parent)) for x, y in zip(xs, ys))
    # a row longer than 2^31 bytes of positions apart
    big = t.zeros(4, 2, 1 << 29, dtype=t.uint8, device="cuda")
    big[1, 1, -5:] = 9
    BeamStates([big[:, :, -16:]]).reorder(t.tensor([[0, 1, 1, 0]], dtype=t.int32).cuda())
    assert big[2, 1, -5:].tolist() == [9] * 5 and int(big[3].max()) == 0


def test_more_sequences_than_a_grid_has_rows(t):
    from invariant_output_head_gb300 import BeamStates
    n = 70001
    x = t.arange(n * 2 * 3, dtype=t.int32, device="cuda").view(n * 2, 3)
    parent = t.zeros(n, 2, dtype=t.int32, device="cuda")
    parent[::2, 0] = 1
    got = x.clone()
    BeamStates([got]).reorder(parent)
    row = (parent + 2 * t.arange(n, dtype=t.int32, device="cuda")[:, None]).view(-1).long()
    assert t.equal(got, x[row])


def test_selection_of_many_sequences_of_few_tokens(t):
    V = 40
    z, s = step_inputs(t, 3000, 2, V, "bf16", 2)
    check(t, head_of(t, V), z, s, 5)


@pytest.mark.parametrize("n_out", [1, 25, 33, 64])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_parts_of_every_size(t, rows, n_out):
    """Rows of few tiles over many blocks: parts of one tile to a row's all."""
    for V in (1023, 1024, 3100, 9000, 33000):
        z, s = step_inputs(t, rows, 1, V, "fp16", V + rows)
        check(t, head_of(t, V), z, s, n_out)


# ------------------------------------------------------------------- together
@pytest.mark.parametrize("beams", [4, 5])
def test_a_search_on_an_e4m3_head(t, beams):
    """Steps of a search as a decode loop runs them: rows quantised, logits,
    selection, states moved; each against its plain form."""
    from invariant_output_head_gb300 import BeamStates, Head, quantize_blocks
    from tests import block_ref
    n_seq, V, d, steps = 3, 2000, 272, 4
    g = t.Generator(device="cuda").manual_seed(11)
    W, ws = quantize_blocks(t.randn(V, d, generator=g, device="cuda") * 0.2, 128)
    head = Head(W)
    embed = t.randn(V, d, generator=g, device="cuda", dtype=t.bfloat16)
    hidden = t.randn(n_seq * beams, d, generator=g, device="cuda", dtype=t.bfloat16)
    history = t.zeros(n_seq * beams, steps, dtype=t.int32, device="cuda")
    states = BeamStates([hidden, history])
    scores = t.zeros(n_seq, beams, device="cuda")
    scores[:, 1:] = -math.inf
    plain = [[] for _ in range(n_seq * beams)]
    for step in range(steps):
        q, xs = quantize_blocks(hidden)
        z = head.block_scaled_logits(q, xs, ws)
        want, A = block_ref.logits(q.float(), xs, W.float(), ws)
        assert bool(((z - want).abs() <= block_ref.logits_tol(A, want, xs.shape[1], z.dtype)).all())
        r = check(t, head, z.cpu(), scores.cpu(), beams)
        states.reorder(r.parent)
        history[:, step] = r.token.view(-1)
        hidden += 0.5 * embed[r.token.view(-1).long()]
        scores = r.score
        plain = [plain[s * beams + int(p)] + [int(v)] for s in range(n_seq)
                 for p, v in zip(r.parent[s], r.token[s])]
    assert history.tolist() == plain
    assert bool(scores.isfinite().all()) and head.check() == 0


def test_a_step_captured_into_a_graph(t):
    from invariant_output_head_gb300 import BeamStates, Head, beam_buffers, block_buffers, quantize_blocks
    n_seq, beams, V, d = 4, 4, 6000, 256
    g = t.Generator(device="cuda").manual_seed(12)
    W, ws = quantize_blocks(t.randn(V, d, generator=g, device="cuda") * 0.2, 128)
    head = Head(W)
    head.reserve_beams(16, beams)
    x = t.randn(16, d, generator=g, device="cuda")
    cache = t.randn(16, 2, 8, 16, generator=g, device="cuda")
    scores = -t.rand(n_seq, beams, generator=g, device="cuda")
    rows, out = block_buffers(16, d, device="cuda"), beam_buffers(n_seq, beams, "cuda")
    z = t.empty(16, V, device="cuda")
    states = BeamStates([cache], token_dim=2)

    def step():
        quantize_blocks(x, out=rows)
        head.block_scaled_logits(*rows, ws, out=z)
        head.beam_select(z, scores, beams, out=out)
        states.reorder(out.parent, used=5)
    first = cache.clone()
    step()
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(t.randn(16, d, generator=g, device="cuda"))
        cache.copy_(first)
        step()
        t.cuda.synchronize()
        want = [v.clone() for v in (z, *out, cache)]
        for v in (z, *out):
            v.zero_()
        cache.copy_(first)
        graph.replay()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip((z, *out, cache), want)), seed
    assert head.check() == 0


def test_a_step_on_another_stream(t):
    from invariant_output_head_gb300 import BeamStates, Head, quantize_blocks
    g = t.Generator(device="cuda").manual_seed(13)
    W, ws = quantize_blocks(t.randn(9000, 256, generator=g, device="cuda") * 0.2, 128)
    head = Head(W)
    x = t.randn(300, 256, generator=g, device="cuda")
    scores = -t.rand(75, 4, generator=g, device="cuda")
    cache = t.randn(300, 40, generator=g, device="cuda")

    def step(stream, state):
        rows = quantize_blocks(x, stream=stream)
        z = head.block_scaled_logits(*rows, ws, stream=stream)
        r = head.beam_select(z, scores, 4, stream=stream)
        BeamStates([state]).reorder(r.parent, stream=stream)
        return [z, *r, state]
    want = step(None, cache.clone())
    t.cuda.synchronize()
    side = t.cuda.Stream()
    mine = cache.clone()
    t.cuda.synchronize()
    got = step(side, mine)
    side.synchronize()
    assert all(t.equal(a, b) for a, b in zip(got, want))
