"""Beam selection's sums and scores at logits of every magnitude: whole tiles
masked with large negative numbers, temperatures from tiny to huge."""
import math

import pytest

pytestmark = pytest.mark.gpu

TILE = 1024                                   # logits that the call sums at a time


@pytest.fixture(scope="module")
def t():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def head_of(t, V):
    from invariant_output_head_gb300 import Head
    return Head(t.zeros(V, 16, dtype=t.bfloat16, device="cuda"))


def sum_bound(V, E, f):
    """Bound on the relative error of a row's sum S of 2^x, x = (z - m) log2(e) /
    T, in half-steps u = 2^-24. Every x is made of parts of one sign (to a tile's
    maximum, then from join to join to the row's), each a difference (1), times
    a rounded log2(e) / T (1 / T is off by f, log2(e) by 1, their product by f
    again), rounded (1): (3 + 2 f) u of |x| ln 2, which over the sum is (3 + 2 f) E
    with E the mean of |z - m| / T under the softmax. In the fused form a tile's exponents are off by up to 1/2 from that,
    u / 2 more, and a factor puts it back: one 2^x (4: it is good to 2^-22) and a
    product (1). 2^x of an element: 4. Additions in a tile: 3 + 3 + 5. A join: 2^x
    (4), product, addition; as many as a lane has tiles, and 5."""
    joins = -(-(-(-V // TILE)) // 32) + 5
    return 0.5 + 5 + 4 + 11 + 6 * joins + (3 + 2 * f) * E


def check_each(t, head, z, s, n_out, T=1.0, finished=None, end=0):
    """The call against 64 bits, every candidate within its own bound: its score
    from its own distance to its row's maximum; each beam's candidates the first
    of its own by (logit falling, token); all of them in order, and none that
    is better left out."""
    n_seq, beams = s.shape
    V = z.shape[1]
    got = head.beam_select(z.cuda(), s.cuda(), n_out, temperature=T, end_token=end,
                           finished=None if finished is None else finished.cuda())
    assert head.check() == 0
    parent, token, score = (x.cpu() for x in got)
    u, T = 2.0 ** -24, float(t.tensor(T, dtype=t.float32))
    f = max(1.0, T * 2.0 ** -126)             # 1 / T in 32 bits: half-steps of it (more below 2^-126)
    for q in range(n_seq):
        total, bound, order = [], [], []
        for b in range(beams):
            row, own = z[q * beams + b].double(), float(s[q, b])
            m = float(row.max())
            if finished is not None and bool(finished[q, b]) and math.isfinite(own):
                # its own score, as it is, for the end token alone
                total.append(t.full((V,), -math.inf, dtype=t.float64))
                total[-1][end] = own
                bound.append(t.zeros(V, dtype=t.float64))
                order.append(t.tensor([end]))
                continue
            if not math.isfinite(own) or math.isnan(m) or math.isinf(m):
                total.append(t.full((V,), -math.inf, dtype=t.float64))
                bound.append(t.zeros(V, dtype=t.float64))
            else:
                far = (row - m) / T
                p = t.softmax(far, dim=0)
                L = float(t.logsumexp(far, dim=0))
                E = float((p * -far.clamp_min(-1e300)).sum())
                x = far - L + own
                D = -far
                total.append(x)
                # difference, 1 / T and product; logf (an ulp) of S; the two sums;
                # products of u left out: 1 %
                bound.append(1.01 * u * ((2 + f) * D + sum_bound(V, E, f) + 2 * L + (D + L) + x.abs()) + 2.0 ** -148)
            order.append(t.sort(row, descending=True, stable=True).indices)
        total, bound = t.stack(total), t.stack(bound)
        total[total.float() == -math.inf] = -math.inf        # no number in 32 bits
        want = total.view(-1).sort(descending=True).values[:n_out]
        real = int((want > -math.inf).sum())
        assert parent[q, real:].tolist() == [-1] * (n_out - real), q
        assert token[q, real:].tolist() == [-1] * (n_out - real), q
        assert score[q, real:].tolist() == [-math.inf] * (n_out - real), q
        assert bool((parent[q, :real] >= 0).all()) and bool((score[q, :real] > -math.inf).all()), q
        p, v, x = parent[q, :real].long(), token[q, :real].long(), score[q, :real]
        tol = bound[p, v]
        assert bool(((x.double() - total[p, v]).abs() <= tol).all()), \
            (q, float(((x.double() - total[p, v]).abs() / tol).max()))
        assert bool((x[:-1] >= x[1:]).all())
        assert bool(((total[p, v] - want[:real]).abs() <= 2 * tol.maximum(bound.view(-1)[
            total.view(-1).sort(descending=True).indices[:real]])).all()), q
        for b in range(beams):
            mine = v[p == b]
            assert t.equal(mine, order[b][:len(mine)]), (q, b)
    return got


def rows(t, n, V, dtype, seed):
    g = t.Generator().manual_seed(seed)
    return (t.randn(n, V, generator=g) * 2.5).to(dtype)


FILLS = ["low", -1e9, -1e10, -1e12, -1e30, -math.inf]


@pytest.mark.parametrize("T", [0.1, 0.3, 1.0, 1.5, 2.0, 30.0])
@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("name", ["float32", "bfloat16", "float16"])
def test_whole_tiles_masked(t, name, fill, T):
    """The first tile, some in the middle, the last (of one logit and of
    many), all but one, in the rows of one sequence; more rows so that tiles
    fall to parts of every length."""
    dtype = getattr(t, name)
    fill = max(t.finfo(dtype).min if fill == "low" else fill,
               -math.inf if fill == -math.inf else t.finfo(dtype).min)
    for V in (8 * TILE + 1, 5 * TILE + 700, TILE + 1):
        z = rows(t, 6, V, dtype, V)
        z[0, :TILE] = fill
        z[1, 2 * TILE:4 * TILE] = fill
        z[2, V // TILE * TILE:] = fill
        z[3, TILE:] = fill
        z[4, :V // TILE * TILE] = fill
        s = -t.rand(1, 6, generator=t.Generator().manual_seed(V)) * 4
        head = head_of(t, V)
        # a sequence of its own for each (a beam that is lost shows), and together
        check_each(t, head, z, s.view(6, 1), 12, T)
        check_each(t, head, z, s, 40, T)


@pytest.mark.parametrize("T", [5e-39, 1e-20, 1e-8, 1e-5, 1e-3, 1e8])
@pytest.mark.parametrize("name", ["float32", "bfloat16", "float16"])
def test_extreme_temperatures(t, name, T):
    """Logits of ordinary size, whose distances to the maximum do not stay so."""
    for V in (3000, 9000):
        z = rows(t, 4, V, getattr(t, name), 3) + 20
        check_each(t, head_of(t, V), z, t.tensor([[-0.5], [-1.0], [-2.0], [0.0]]), 16, T)


@pytest.mark.parametrize("T", [1.0, 0.7, 3.0])
@pytest.mark.parametrize("name", ["float32", "bfloat16"])
@pytest.mark.parametrize("at", [1e4, 1e7, 3e8, -3e8, 1e10, -1e10, 1e20, -1e30])
def test_logits_far_from_zero(t, name, at, T):
    """Whole rows about one large number, on its steps: exponents on both sides
    of where the form of a tile's sum changes."""
    dtype = getattr(t, name)
    V = 4 * TILE + 3
    base = t.tensor(at, dtype=dtype)
    step = abs(float(base.double())) * 2.0 ** (-23 if dtype == t.float32 else -7)
    k = t.randint(-3, 4, (3, V), generator=t.Generator().manual_seed(7))
    z = (base.double() + k * step).to(dtype)
    check_each(t, head_of(t, V), z, t.tensor([[-0.5], [-1.0], [-2.0]]), 10, T)


def test_one_masked_tile_leaves_other_rows_bits(t):
    """A row's bits are its own: masked tiles beside it change nothing."""
    V = 6 * TILE
    z = rows(t, 8, V, t.bfloat16, 1)
    s = t.zeros(8, 1)
    head = head_of(t, V)
    before = head.beam_select(z.cuda(), s.cuda(), 8)
    z[3, TILE:3 * TILE] = -1e30
    after = head.beam_select(z.cuda(), s.cuda(), 8)
    keep = [0, 1, 2, 4, 5, 6, 7]
    assert all(t.equal(a[keep], b[keep]) for a, b in zip(before, after))
    assert (after.parent[3] == 0).all()


@pytest.mark.parametrize("T", [1.0, 2.0, 8.0, 1e30, 1e37, 1e38, 3e38])
@pytest.mark.parametrize("name", ["float32", "bfloat16"])
def test_logits_farther_apart_than_32_bits_hold(t, name, T):
    """Logits of both ends of the type's range: their difference overflows, the
    scores and the weights in the sum need not."""
    V = 5 * TILE + 9
    z = t.rand(4, V, generator=t.Generator().manual_seed(2)) * 6e38 - 3e38
    z[1, :3 * TILE] = -3.3e38               # tiles at the two ends
    z[1, 3 * TILE:] = 3.3e38
    z[2, :-1], z[2, -1] = t.finfo(getattr(t, name)).min, 1e38
    z[3, 5:] = -math.inf
    check_each(t, head_of(t, V), z.to(getattr(t, name)), t.tensor([[-0.5], [-1.0], [-2.0], [0.0]]), 16, T)


@pytest.mark.parametrize("T", [0.7, 1.0, 2.5])
@pytest.mark.parametrize("name", ["float32", "bfloat16", "float16"])
def test_masked_finished_and_dead_beams_together(t, name, T):
    dtype = getattr(t, name)
    V = 9 * TILE + 77
    z = rows(t, 24, V, dtype, 5)
    low = t.finfo(dtype).min
    z[0] = -math.inf                        # a row with nothing
    z[1, 1:] = -math.inf                    # one token
    z[2, :8 * TILE] = low
    z[3, 100:] = max(-1e10, low)
    z[4, 17], z[5, V - 1] = math.nan, math.inf
    z[6] = low                              # every token alike
    z[9, TILE:] = max(-1e30, low)
    z[13, 5] = math.nan                     # of a finished beam: not read
    s = -t.rand(6, 4, generator=t.Generator().manual_seed(6)) * 4 - 3
    s[1, 1], s[1, 3], s[2, 0] = -math.inf, math.nan, math.inf
    finished = t.zeros(6, 4, dtype=t.bool)
    finished[2, 1] = finished[3, 1] = finished[5, 0] = finished[5, 1] = finished[5, 2] = True
    finished[1, 1] = True                   # finished and dead: nothing
    head = head_of(t, V)
    for n_out, end in ((4, 0), (16, V - 1), (64, 3)):
        check_each(t, head, z, s, n_out, T, finished, end)
    check_each(t, head, z, s, 16, T, finished.to(t.uint8) * 128, 9)


def test_outputs_in_page_locked_host_memory(t):
    """As of the other calls: a device address of page-locked memory will do."""
    from invariant_output_head_gb300 import binding as b
    from invariant_output_head_gb300 import Head, quantize_blocks
    g = t.Generator(device="cuda").manual_seed(4)
    V, d, n, beams = 1000, 256, 50, 4
    W, ws = quantize_blocks(t.randn(V, d, generator=g, device="cuda"), 128)
    head = Head(W)
    x = t.randn(n * beams, d, generator=g, device="cuda")
    scores = -t.rand(n, beams, generator=g, device="cuda")
    stream = t.cuda.current_stream().cuda_stream
    for B in (3 * beams, n * beams):
        q, xs = quantize_blocks(x[:B].contiguous())
        z = head.block_scaled_logits(q, xs, ws)
        r = head.beam_select(z, scores[:B // beams], beams)
        rows_ = x[:B].clone()
        b.BeamStates([rows_]).reorder(r.parent)
        pin = [t.empty(v.shape, dtype=v.dtype).pin_memory() for v in (q, xs, z, *r, rows_)]
        b.detlm_quantize_blocks(x.data_ptr(), b.DETLM_FP32, B, d, 1, pin[0].data_ptr(),
                                pin[1].data_ptr(), stream)
        b.detlm_head_block_scaled_logits(head.handle, q.data_ptr(), xs.data_ptr(), ws.data_ptr(), B,
                                         b.DETLM_FP32, pin[2].data_ptr(), stream)
        b.detlm_head_beam_select(head.handle, z.data_ptr(), b.DETLM_FP32, scores.data_ptr(), None, 0,
                                 B // beams, beams, beams, 1.0, *(v.data_ptr() for v in pin[3:6]), stream)
        state = (b._State * 1)()
        e = state[0]
        e.src, e.dst, e.src_row, e.dst_row = x.data_ptr(), pin[6].data_ptr(), 4 * d, 4 * d
        e.n_seg, e.seg_bytes = 1, 4 * d
        b.detlm_beam_reorder(b.ctypes.addressof(state), 1, r.parent.data_ptr(), B // beams, beams,
                             beams, -1, stream)
        t.cuda.synchronize()
        assert head.check() == 0
        for got, want in zip(pin, (q, xs, z, *r, rows_)):
            assert t.equal(got.view(-1).view(t.uint8), want.cpu().view(-1).view(t.uint8))
