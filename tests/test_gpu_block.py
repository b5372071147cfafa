"""Block quantisation and block-scaled logits of the e4m3 head against 64-bit
forms, and the bits of a row whatever its batch."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def t():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def dtype_of(t, name):
    return {"f32": t.float32, "bf16": t.bfloat16, "fp16": t.float16}[name]


def rows_of(t, B, d, name, seed):
    """Rows of spread magnitudes, empty blocks, values at the borders."""
    g = t.Generator().manual_seed(seed)
    x = t.randn(B, d, generator=g) * t.exp2(t.rand(B, 1, generator=g) * 12 - 6)
    x[t.rand(B, d, generator=g) < 0.1] = 0.0
    if d > 128:
        x[B // 2, 128:256] = 0.0
    x[0, :8] = t.tensor([448.0, -448.0, 449.0, 464.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 0.0])
    return x.to(dtype_of(t, name))


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("name", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("B, d", [(1, 16), (1, 128), (3, 144), (127, 272), (130, 1040), (257, 64)])
def test_quantisation_is_the_one_right_value(t, B, d, name, rows):
    from invariant_output_head_gb300 import quantize_blocks
    from tests import block_ref
    x = rows_of(t, B, d, name, 7 * B + d)
    q, scale = quantize_blocks(x.cuda(), rows)
    want_q, want_s = block_ref.quantize(x, rows)
    assert q.dtype == t.float8_e4m3fn and q.shape == (B, d)
    assert t.equal(scale.cpu().double(), want_s)
    assert t.equal(q.cpu().float().double(), want_q)


@pytest.mark.parametrize("rows", [1, 128])
def test_quantisation_of_extremes(t, rows):
    from invariant_output_head_gb300 import quantize_blocks
    from tests import block_ref
    x = t.zeros(256, 256)
    x[0, 0], x[0, 130] = 3.4e38, 1e-45
    x[128, 3], x[128, 200] = float("nan"), float("-inf")
    x[130, 4], x[200, 255] = 2.0 ** -126, -2.0 ** -130
    for y in (x, x.bfloat16()):
        q, scale = quantize_blocks(y.cuda(), rows)
        want_q, want_s = block_ref.quantize(y, rows)
        assert t.equal(scale.cpu().double().nan_to_num(nan=-1), want_s.nan_to_num(nan=-1))
        assert t.equal(q.cpu().float().double().nan_to_num(nan=999), want_q.nan_to_num(nan=999))


def test_quantisation_into_given_tensors_leaves_their_neighbours(t):
    from invariant_output_head_gb300 import quantize_blocks
    x = rows_of(t, 5, 144, "bf16", 3).cuda()
    q = t.full((9, 144), 7, dtype=t.uint8, device="cuda")
    s = t.full((9, 2), -3.0, device="cuda")
    quantize_blocks(x, 1, out=(q[2:7].view(t.float8_e4m3fn), s[2:7]))
    want = quantize_blocks(x)
    assert t.equal(q[2:7], want[0].view(t.uint8)) and t.equal(s[2:7], want[1])
    assert bool((q[:2] == 7).all() and (q[7:] == 7).all())
    assert bool((s[:2] == -3).all() and (s[7:] == -3).all())


# --------------------------------------------------------------------- logits
def head_inputs(t, B, V, d, seed, dyadic=False):
    """Quantised rows and weight; scales of a checkpoint (any floats) or dyadic."""
    g = t.Generator(device="cuda").manual_seed(seed)
    q = t.randn(B, d, generator=g, device="cuda") * 60
    W = t.randn(V, d, generator=g, device="cuda") * 100
    q, W = (x.clamp(-448, 448).to(t.float8_e4m3fn) for x in (q, W))
    nb = -(-d // 128)
    xs = t.exp2(t.rand(B, nb, generator=g, device="cuda") * 6 - 9)
    ws = t.exp2(t.rand(-(-V // 128), nb, generator=g, device="cuda") * 4 - 12)
    if dyadic:
        xs, ws = (t.exp2(s.log2().round()) for s in (xs, ws))
    return q, xs, W, ws


SIZES = [(1, 1, 16), (1, 127, 128), (2, 1000, 144), (7, 33, 272), (16, 4097, 64), (17, 500, 1040),
         (31, 129, 512), (33, 32000, 256), (48, 777, 2048), (64, 5000, 400), (65, 300, 1024),
         (80, 999, 272), (97, 2500, 528), (128, 161, 640), (129, 1, 16), (130, 1000, 272),
         (255, 128, 144), (256, 2049, 384), (257, 255, 1040), (513, 3001, 528), (700, 640, 2176)]


@pytest.mark.parametrize("out", ["f32", "bf16", "fp16"])
@pytest.mark.parametrize("B, V, d", SIZES)
def test_logits_against_64_bits(t, B, V, d, out):
    from invariant_output_head_gb300 import Head
    from tests import block_ref
    q, xs, W, ws = head_inputs(t, B, V, d, B + V + d, dyadic=out == "bf16")
    head = Head(W)
    z = head.block_scaled_logits(q, xs, ws, out_dtype=dtype_of(t, out))
    assert head.check() == 0
    want, A = block_ref.logits(q.float(), xs, W.float(), ws)
    tol = block_ref.logits_tol(A, want, xs.shape[1], z.dtype)
    assert z.dtype == dtype_of(t, out) and z.shape == (B, V)
    assert bool(((z.double() - want).abs() <= tol).all())


def test_products_of_one_sign_and_of_the_largest_values(t):
    """All products positive (any one-sided loss adds up), and all at 448^2."""
    from invariant_output_head_gb300 import Head
    from tests import block_ref
    for d, big in ((4096, False), (16384, False), (1040, True)):
        q, xs, W, ws = head_inputs(t, 140, 300, d, d)
        q, W = (x.float().abs() for x in (q, W))
        if big:
            q, W = t.full_like(q, 448.0), t.full_like(W, 448.0)
        q, W = q.to(t.float8_e4m3fn), W.to(t.float8_e4m3fn)
        head = Head(W)
        want, A = block_ref.logits(q.float(), xs, W.float(), ws)
        tol = block_ref.logits_tol(A, want, xs.shape[1], t.float32)
        for rows in (1, 100, 140):
            z = head.block_scaled_logits(q[:rows], xs[:rows], ws)
            assert head.check() == 0
            assert bool(((z.double() - want[:rows]).abs() <= tol[:rows]).all()), (d, big, rows)


@pytest.mark.parametrize("V, d, out", [(5000, 1040, "f32"), (32000, 512, "bf16"), (1001, 2048, "fp16")])
def test_a_rows_bits_do_not_depend_on_its_batch(t, V, d, out):
    from invariant_output_head_gb300 import Head
    q, xs, W, ws = head_inputs(t, 600, V, d, V)
    head = Head(W)
    whole = head.block_scaled_logits(q, xs, ws, out_dtype=dtype_of(t, out))
    for B in (1, 2, 16, 17, 33, 64, 65, 100, 128, 129, 256, 257, 599):
        for first in (0, 600 - B):
            at = slice(first, first + B)
            z = head.block_scaled_logits(q[at].contiguous(), xs[at].contiguous(), ws,
                                         out_dtype=dtype_of(t, out))
            assert t.equal(z, whole[at]), (B, first)
    # and on the other rows' values
    q2 = q.clone()
    q2.view(t.uint8)[1:] = 0x7F                         # NaN
    z = head.block_scaled_logits(q2, xs, ws, out_dtype=dtype_of(t, out))
    assert t.equal(z[0], whole[0]) and bool(z[1:].isnan().all())
    assert head.check() == 0


def test_a_block_that_is_not_finite_reaches_its_row_and_no_other(t):
    from invariant_output_head_gb300 import Head, quantize_blocks
    g = t.Generator(device="cuda").manual_seed(5)
    x = t.randn(40, 400, generator=g, device="cuda")
    q, xs, W, ws = head_inputs(t, 40, 700, 400, 6)
    x[3, 390], x[9, 2] = float("inf"), float("nan")
    head = Head(W)
    z = head.block_scaled_logits(*quantize_blocks(x), ws)
    bad = t.zeros(40, dtype=t.bool, device="cuda")
    bad[[3, 9]] = True
    assert bool(z[bad].isnan().all()) and bool(z[~bad].isfinite().all())


@pytest.mark.parametrize("B", [5, 200])
@pytest.mark.parametrize("V, name, shift", [(999, "bf16", 1), (1000, "bf16", 3), (1000, "f32", 1),
                                            (1001, "f32", 2), (1003, "fp16", 0)])
def test_logits_into_unaligned_tensors(t, B, V, name, shift):
    from invariant_output_head_gb300 import Head
    q, xs, W, ws = head_inputs(t, B, V, 272, V)
    head = Head(W)
    want = head.block_scaled_logits(q, xs, ws, out_dtype=dtype_of(t, name))
    room = t.full((B * V + 16,), 5.0, dtype=dtype_of(t, name), device="cuda")
    out = room[shift:shift + B * V].view(B, V)
    head.block_scaled_logits(q, xs, ws, out=out)
    assert t.equal(out, want)
    assert bool((room[:shift] == 5).all() and (room[shift + B * V:] == 5).all())


def test_no_rows(t):
    from invariant_output_head_gb300 import Head, quantize_blocks
    q, xs, W, ws = head_inputs(t, 1, 300, 64, 1)
    head = Head(W)
    none = quantize_blocks(t.empty(0, 64, device="cuda"))
    assert none[0].shape == (0, 64) and none[1].shape == (0, 1)
    assert head.block_scaled_logits(*none, ws).shape == (0, 300)


def test_other_calls_refuse_an_e4m3_head(t):
    from invariant_output_head_gb300 import DetlmError, Head, DETLM_EUNSUPPORTED
    q, xs, W, ws = head_inputs(t, 4, 300, 64, 1)
    head = Head(W)
    i32 = t.zeros(4, dtype=t.int32, device="cuda")
    i64 = t.zeros(4, dtype=t.int64, device="cuda")
    f32 = t.zeros(4, device="cuda")
    for call in (lambda: head.greedy(q), lambda: head.logprob(q, i32), lambda: head.score(q, i32),
                 lambda: head.greedy_gated(q), lambda: head.sample(q, 1.0, i64, i64),
                 lambda: head.verify(q, i32.view(2, 2)), lambda: head.reserve_score(4),
                 lambda: head.score_backward(q, i32, f32, f32, f32),
                 lambda: head.reserve_backward(4), lambda: head.greedy_from_float(q.float()),
                 lambda: head.scaled_logits(q, f32, t.zeros(300, device="cuda"))):
        with pytest.raises(DetlmError) as e:
            call()
        assert e.value.status == DETLM_EUNSUPPORTED
    head.reserve(300)
    head.weights_changed()
    assert t.isfinite(head.block_scaled_logits(q, xs, ws)).all()
    with pytest.raises(DetlmError):
        Head(t.zeros(30, 64, dtype=t.bfloat16, device="cuda")).block_scaled_logits(q, xs, ws)


@pytest.mark.parametrize("B", [3, 200])
def test_a_stalled_kernel_times_out_and_the_head_recovers(t, B):
    from invariant_output_head_gb300 import Head, binding
    q, xs, W, ws = head_inputs(t, B, 3000, 512, 2)
    head = Head(W)
    want = head.block_scaled_logits(q, xs, ws)
    binding.detlm_head_debug(head.handle, binding.DETLM_DEBUG_STALL, 50_000_000)
    head.block_scaled_logits(q, xs, ws)
    assert head.check() == binding.DETLM_ETIMEOUT
    binding.detlm_head_debug(head.handle, 0, 0)
    assert t.equal(head.block_scaled_logits(q, xs, ws), want)
    assert head.check() == 0


def test_a_weight_quantised_in_place_right_before_the_call(t):
    """Each call uses the weight that the call before it on the stream wrote."""
    from invariant_output_head_gb300 import Head, quantize_blocks
    g = t.Generator(device="cuda").manual_seed(7)
    V, d = 20000, 1024
    Ws = [t.randn(V, d, generator=g, device="cuda", dtype=t.bfloat16) for _ in range(6)]
    q, xs = quantize_blocks(t.randn(3, d, generator=g, device="cuda"))
    want = []
    for W in Ws:
        Wq, ws = quantize_blocks(W, 128)
        t.cuda.synchronize()
        want.append(Head(Wq).block_scaled_logits(q, xs, ws))
    weight = quantize_blocks(Ws[-1], 128)
    head = Head(weight[0])
    got = [t.empty_like(want[0]) for _ in Ws]
    t.cuda.synchronize()
    for W, z in zip(Ws, got):
        quantize_blocks(W, 128, out=weight)
        head.weights_changed()
        head.block_scaled_logits(q, xs, weight[1], out=z)
    assert all(t.equal(a, b) for a, b in zip(got, want))
    assert head.check() == 0


def test_two_heads_on_two_streams(t):
    from invariant_output_head_gb300 import Head
    cases = [head_inputs(t, B, 8000, 512, B) for B in (3, 300)]
    heads = [Head(c[2]) for c in cases]
    want = [h.block_scaled_logits(c[0], c[1], c[3]) for h, c in zip(heads, cases)]
    t.cuda.synchronize()
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    got = [[h.block_scaled_logits(c[0], c[1], c[3], stream=s) for _ in range(8)]
           for h, c, s in zip(heads, cases, streams)]
    t.cuda.synchronize()
    assert all(t.equal(z, w) for zs, w in zip(got, want) for z in zs)
    assert [h.check() for h in heads] == [0, 0]


def test_addresses_that_are_refused(t):
    from invariant_output_head_gb300 import DetlmError, Head, quantize_blocks
    q, xs, W, ws = head_inputs(t, 2, 300, 64, 1)
    room = t.zeros(200, dtype=t.float32, device="cuda")
    with pytest.raises(DetlmError):
        quantize_blocks(room[1:129].view(2, 64))                # rows between 16 bytes
    with pytest.raises(DetlmError):
        quantize_blocks(room[:2 * 40].view(2, 40))              # d no multiple of 16
    bytes_ = t.zeros(300, dtype=t.uint8, device="cuda")
    with pytest.raises(DetlmError):
        Head(W).block_scaled_logits(bytes_[8:136].view(t.float8_e4m3fn).view(2, 64), xs, ws)


@pytest.mark.parametrize("B", [5, 100, 200])
def test_rows_quantised_right_before_the_call(t, B):
    """The quantisation of many rows is still under way when the product of the
    last of them is launched: it reads the rows and scales of this quantisation,
    not of the one before."""
    from invariant_output_head_gb300 import Head, block_buffers, quantize_blocks
    n, d, V = 6000, 8192, 1000
    g = t.Generator(device="cuda").manual_seed(B)
    W = t.randn(V, d, device="cuda", generator=g).mul_(60).clamp_(-448, 448).to(t.float8_e4m3fn)
    head = Head(W)
    ws = t.rand(8, 64, device="cuda", generator=g) + 0.5
    xs = [t.randn(n, d, device="cuda", generator=g) * 10.0 ** (4 * i) for i in range(2)]
    want = []
    for x in xs:
        q, s = quantize_blocks(x)
        t.cuda.synchronize()
        want.append(head.block_scaled_logits(q[-B:], s[-B:], ws))
        t.cuda.synchronize()
    out = block_buffers(n, d, device="cuda")
    for i in range(20):
        quantize_blocks(xs[i % 2], out=out)
        got = head.block_scaled_logits(out[0][-B:], out[1][-B:], ws)
        assert t.equal(got, want[i % 2])


def test_a_vocabulary_of_the_largest_size(t):
    """V = 2^31 - 1: the last group of rows ends one short of 2^31."""
    from invariant_output_head_gb300 import Head
    if t.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("not enough free memory")
    V, d = 2 ** 31 - 1, 16
    W = t.zeros(V, d, dtype=t.uint8, device="cuda")
    at = [0, 31, 2 ** 30 + 5, V - 40, V - 1]
    for i, v in enumerate(at):
        W[v] = 0x38 + 8 * i                       # 2^i
    ws = t.ones(2 ** 24, 1, device="cuda")
    ws[-1] = 0.5
    q = t.full((1, d), 0x38, dtype=t.uint8, device="cuda").view(t.float8_e4m3fn)
    out = t.full((1, V), 7.0, dtype=t.bfloat16, device="cuda")
    Head(W.view(t.float8_e4m3fn)).block_scaled_logits(q, t.ones(1, 1, device="cuda"), ws, out=out)
    assert [float(out[0, v]) for v in at] == [16.0, 32.0, 64.0, 64.0, 128.0]
    for v in at:
        out[0, v] = 0.0
    assert not bool(out.view(t.int16).any())
