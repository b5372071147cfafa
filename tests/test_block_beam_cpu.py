"""Refusals of the e4m3 head's and the beam calls, on the host (no GPU), and
the layout of states."""
import ctypes
import math
import random

import pytest

torch = pytest.importorskip("torch")

from invariant_output_head_gb300 import binding as b          # noqa: E402
from tests import block_ref                                    # noqa: E402


@pytest.fixture(scope="module")
def lib():
    from invariant_output_head_gb300 import build
    build.build()
    return b.load_library()


class _OnDevice(torch.Tensor):
    """A host tensor that says it is a CUDA tensor (on `where`)."""
    is_cuda = True
    where = torch.device("cuda:0")

    @property
    def device(self):
        return self.where


class _OnOther(_OnDevice):
    where = torch.device("cuda:1")


def fake(*shape, dtype=torch.float32, other=False):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_OnOther if other else _OnDevice)


@pytest.fixture
def calls(monkeypatch):
    made = []
    for name in ("detlm_quantize_blocks", "detlm_head_block_scaled_logits",
                 "detlm_head_beam_select", "detlm_beam_reorder"):
        monkeypatch.setattr(b, name, lambda *a, name=name: made.append((name, a)))
    monkeypatch.setattr(b, "_stream_ptr", lambda s: 0)
    monkeypatch.setattr(b, "_on_device", lambda t, call: call())
    return made


def head_of(W, dtype):
    h = b.Head.__new__(b.Head)
    h.W, h.dtype, h.handle = W, dtype, None
    h.V, h.d = W.shape
    return h


# ------------------------------------------------------------------- C entries
P = 0x7F0000000000          # never read: the checks come first


@pytest.mark.parametrize("args", [
    (P, 2, 4, 64, 1, P, P),            # int8 rows
    (P, 4, 4, 64, 1, P, P),            # e4m3 rows
    (P, 0, -1, 64, 1, P, P),
    (P, 0, 2**31, 64, 1, P, P),
    (P, 0, 4, 0, 1, P, P),
    (P, 0, 4, 24, 1, P, P),            # not whole 16-byte rows
    (P, 0, 4, 64, 0, P, P),
    (P, 0, 4, 64, 64, P, P),           # blocks of another shape
    (None, 0, 4, 64, 1, P, P),
    (P + 8, 0, 4, 64, 1, P, P),
    (P, 0, 4, 64, 1, P + 8, P),
    (P, 0, 4, 64, 1, None, P),
    (P, 0, 4, 64, 1, P, P + 2),
    (P, 0, 4, 64, 1, P, None),
    (P, 0, 2**31 - 1, 2**20, 1, P, P),     # more blocks than a launch has
])
def test_quantize_blocks_refuses(lib, args):
    assert lib.detlm_quantize_blocks(*args, None) == b.DETLM_EINVAL


def test_no_rows_are_no_work(lib):
    assert lib.detlm_quantize_blocks(None, 0, 0, 64, 1, None, None, None) == b.DETLM_OK
    assert lib.detlm_beam_reorder(None, 0, None, 0, 4, 4, -1, None) == b.DETLM_OK
    assert lib.detlm_beam_reorder(None, 0, None, 3, 4, 4, -1, None) == b.DETLM_OK


def test_calls_on_null_handles(lib):
    assert lib.detlm_head_block_scaled_logits(None, P, P, P, 1, 3, P, None) == b.DETLM_EINVAL
    assert lib.detlm_head_reserve_beams(None, 4, 4) == b.DETLM_EINVAL
    assert lib.detlm_head_beam_select(None, P, 3, P, None, 0, 1, 4, 4, 1.0, P, P, P, None) == \
        b.DETLM_EINVAL


def test_create_refuses_e4m3_heads_of_other_sizes(lib):
    for d in (8, 24, 16400):
        out = ctypes.c_void_p(0)
        assert lib.detlm_head_create(ctypes.byref(out), P, 100, d, b.DETLM_E4M3) == b.DETLM_EINVAL
    out = ctypes.c_void_p(0)
    assert lib.detlm_head_create_shard(ctypes.byref(out), P, 1000, 64, b.DETLM_E4M3, 2, 0) == \
        b.DETLM_EUNSUPPORTED
    assert lib.detlm_greedy_noalloc(P, 100, 64, b.DETLM_E4M3, P, 1, P, P, None, None, None) == \
        b.DETLM_EUNSUPPORTED


def state(src=P, dst=P + 4096, row=1024, dst_row=None, seg=64, dst_seg=None, n_seg=2, size=32, position=0):
    s = (b._State * 1)()
    s[0].src, s[0].dst = src, dst
    s[0].src_row, s[0].dst_row = row, row if dst_row is None else dst_row
    s[0].src_seg, s[0].dst_seg = seg, seg if dst_seg is None else dst_seg
    s[0].n_seg, s[0].seg_bytes, s[0].position_bytes = n_seg, size, position
    return s


@pytest.mark.parametrize("s, parent, n_seq, beams_in, beams_out", [
    (state(), None, 1, 4, 4),
    (state(), P + 2, 1, 4, 4),
    (state(), P, -1, 4, 4),
    (state(), P, 1, 0, 4),
    (state(), P, 1, 4, 33),
    (state(), P, 1, 33, 4),
    (state(), P, 2**29, 4, 4),
    (state(src=None), P, 1, 4, 4),
    (state(dst=None), P, 1, 4, 4),
    (state(n_seg=-1), P, 1, 4, 4),
    (state(size=-1), P, 1, 4, 4),
    (state(position=-4), P, 1, 4, 4),
    (state(dst=P), P, 1, 4, 5),                  # in place to more rows
    (state(dst=P, dst_row=512), P, 1, 4, 4),     # in place with another stride
    (state(dst=P, dst_seg=32), P, 1, 4, 4),
    (state(size=2**36, n_seg=1), P, 1, 4, 4),    # columns past 31 bits
    (state(size=2**30 + 1, n_seg=2), P, 1, 4, 4),
])
def test_reorder_refuses(lib, s, parent, n_seq, beams_in, beams_out):
    assert lib.detlm_beam_reorder(ctypes.addressof(s), 1, parent, n_seq, beams_in, beams_out,
                                  -1, None) == b.DETLM_EINVAL


def test_reorder_refuses_a_table_that_is_missing(lib):
    assert lib.detlm_beam_reorder(None, 1, P, 1, 4, 4, -1, None) == b.DETLM_EINVAL
    assert lib.detlm_beam_reorder(None, -1, P, 1, 4, 4, -1, None) == b.DETLM_EINVAL


# --------------------------------------------------------------------- binding
def test_quantize_blocks_arguments(calls):
    b.quantize_blocks(fake(5, 64), out=(fake(5, 64, dtype=torch.float8_e4m3fn), fake(5, 1)))
    assert [c[0] for c in calls] == ["detlm_quantize_blocks"]
    q, s = fake(5, 160, dtype=torch.float8_e4m3fn), fake(5, 2)
    x = fake(5, 160)
    bad = [(torch.zeros(5, 160), 1, (q, s)), (x, 2, (q, s)), (fake(5, 320)[:, ::2], 1, (q, s)),
           (fake(5, 160, dtype=torch.int8), 1, (q, s)), (x, 1, (fake(5, 160), s)),
           (x, 1, (q[:4], s)), (x, 1, (q, fake(5, 1))), (x, 128, (q, s)),
           (x, 1, (q, fake(5, 2, dtype=torch.float64))), (x, 1, (q, fake(5, 2, other=True))),
           (x, 1, (fake(5, 160, dtype=torch.float8_e4m3fn, other=True), s))]
    for x, rows, out in bad:
        with pytest.raises(ValueError):
            b.quantize_blocks(x, rows, out=out)
    assert len(calls) == 1


def test_block_scaled_logits_arguments(calls):
    e4m3 = torch.float8_e4m3fn
    head = head_of(fake(300, 272, dtype=e4m3), "e4m3")
    q, xs, ws, out = fake(5, 272, dtype=e4m3), fake(5, 3), fake(3, 3), fake(5, 300)
    head.block_scaled_logits(q, xs, ws, out=out)
    assert len(calls) == 1
    bad = [(q.view(torch.int8), xs, ws, out), (q, fake(5, 2), ws, out), (q, xs, fake(2, 3), out),
           (q, xs.double(), ws, out), (q, xs, ws, fake(5, 299)), (q, xs, ws, fake(4, 300)),
           (q, xs, ws, fake(5, 300, dtype=torch.int32)), (q, xs, ws, fake(5, 300, other=True)),
           (fake(5, 256, dtype=e4m3), xs, ws, out), (q, xs, fake(3, 6)[:, ::2], out),
           (fake(5, 272, dtype=e4m3, other=True), xs, ws, out)]
    for args in bad:
        with pytest.raises(ValueError):
            head.block_scaled_logits(*args[:3], out=args[3])
    with pytest.raises(ValueError):
        head.block_scaled_logits(q, xs, ws, out_dtype=torch.float16, out=out)
    with pytest.raises(b.DetlmError):
        head_of(fake(300, 272, dtype=torch.int8), "int8").block_scaled_logits(q, xs, ws, out=out)
    assert len(calls) == 1


def test_beam_select_arguments(calls):
    head = head_of(fake(50, 16, dtype=torch.bfloat16), "bf16")
    z, s = fake(12, 50), fake(3, 4)
    out = b.Beams(fake(3, 8, dtype=torch.int32), fake(3, 8, dtype=torch.int32), fake(3, 8))
    done = fake(3, 4, dtype=torch.bool)
    head.beam_select(z, s, 8, finished=done, out=out)
    assert len(calls) == 1
    bad = [dict(logits=fake(11, 50)), dict(logits=fake(12, 49)), dict(logits=z.double()),
           dict(logits=fake(12, 50, dtype=torch.int32)), dict(scores=fake(12)),
           dict(scores=s.double()), dict(logits=fake(12, 100)[:, ::2]),
           dict(finished=fake(3, 4)), dict(finished=fake(4, 3, dtype=torch.bool)),
           dict(n_out=7), dict(scores=fake(3, 4, other=True)), dict(logits=fake(12, 50, other=True)),
           dict(out=b.Beams(out.token, out.token.long(), out.score)),
           dict(out=b.Beams(out.token, out.token, out.score.double()))]
    for change in bad:
        args = dict(logits=z, scores=s, n_out=8, finished=done, out=out) | change
        with pytest.raises(ValueError):
            head.beam_select(**args)
    assert len(calls) == 1


def test_states_layouts_and_refusals(calls):
    cache = fake(8, 3, 20, 16, dtype=torch.bfloat16)
    tokens = fake(8, 20, dtype=torch.int32)
    parent = fake(2, 4, dtype=torch.int32)
    st = b.BeamStates([cache, tokens], token_dim=[2, 1])
    st.reorder(parent, used=7)
    (_, args), = calls
    assert args[1:7] == (2, parent.data_ptr(), 2, 4, 4, 7)
    e = st._table[0]
    assert (e.src, e.dst, e.src_row, e.src_seg, e.n_seg, e.seg_bytes, e.position_bytes) == \
        (cache.data_ptr(), cache.data_ptr(), 3 * 20 * 32, 20 * 32, 3, 20 * 32, 32)
    e = st._table[1]
    assert (e.n_seg, e.seg_bytes, e.position_bytes) == (1, 80, 4)
    st.reorder(parent)                                   # all of it
    assert calls.pop()[1][6] == -1
    # positions first, no positions, slices of one tensor
    assert [getattr(b.BeamStates([cache.view(8, 20, 3, 16)], token_dim=1)._table[0], k)
            for k in ("n_seg", "seg_bytes")] == [1, 20 * 96]
    assert b.BeamStates([cache])._table[0].seg_bytes == 3 * 20 * 32
    both = fake(8, 2, 3, 20, 16)
    b.BeamStates([both[:, 0], both[:, 1]], token_dim=2)
    with pytest.raises(ValueError):
        st.reorder(parent, used=21)
    with pytest.raises(ValueError):
        st.reorder(parent, used=-1)
    with pytest.raises(ValueError):
        st.reorder(fake(2, 3, dtype=torch.int32))
    with pytest.raises(ValueError):
        st.reorder(fake(2, 4, dtype=torch.int64))
    with pytest.raises(ValueError):
        st.reorder(fake(2, 4, dtype=torch.int32, other=True))
    with pytest.raises(ValueError):
        b.BeamStates([cache]).reorder(parent, used=3)    # no axis of positions
    with pytest.raises(ValueError):
        b.BeamStates([cache, cache])
    with pytest.raises(ValueError):
        b.BeamStates([])
    with pytest.raises(ValueError):
        b.BeamStates([cache, tokens], token_dim=[2])
    with pytest.raises(ValueError):
        b.BeamStates([torch.zeros(8, 4)])
    with pytest.raises(ValueError):
        b.BeamStates([cache], token_dim=0)
    with pytest.raises(ValueError):
        b.BeamStates([cache, fake(9, 4)])
    with pytest.raises(ValueError):
        b.BeamStates([cache], out=[cache])               # in place is without out
    with pytest.raises(ValueError):
        b.BeamStates([cache[:6]], out=[cache[2:]])
    with pytest.raises(ValueError):
        b.BeamStates([cache], out=[fake(8, 3, 20, 16)])  # another type
    with pytest.raises(ValueError):
        b.BeamStates([cache], out=[fake(8, 3, 20, 8, dtype=torch.bfloat16)])
    with pytest.raises(ValueError):
        b.BeamStates([cache[:, :, :5, ::2]])             # pieces at two strides
    with pytest.raises(ValueError):
        b.BeamStates([cache], out=[fake(1, 3, 20, 16, dtype=torch.bfloat16).expand(8, 3, 20, 16)])


def test_selection_over_part_of_its_scores_is_refused(calls):
    head = head_of(fake(50, 16, dtype=torch.bfloat16), "bf16")
    z, pool = fake(12, 50), fake(40)
    i32 = [fake(3, n, dtype=torch.int32) for n in (4, 4, 8, 8)]
    s = pool[8:20].view(3, 4)
    head.beam_select(z, s, 4, out=b.Beams(*i32[:2], s))
    head.beam_select(z, s, 4, out=b.Beams(*i32[:2], pool[20:32].view(3, 4)))
    assert len(calls) == 2
    for n, score in ((4, pool[9:21]), (4, pool[:12]), (8, pool[8:32]), (8, pool[:24])):
        with pytest.raises(ValueError):
            head.beam_select(z, s, n, out=b.Beams(*i32[n // 2 - 2:][:2], score.view(3, n)))
    assert len(calls) == 2


def test_states_that_share_memory_are_refused(calls):
    both = fake(8, 2, 3, 20, 16)
    flat = both.view(-1)
    kv = fake(8, 3, 32)
    turned = fake(3, 8, 40).transpose(0, 1)              # pieces of all rows between a row's
    b.BeamStates([turned, kv[..., :16], kv[..., 16:]])
    b.BeamStates([both[:, 0]], out=[both[:, 1]])
    b.BeamStates([flat[:640].view(8, 80), flat[640:1280].view(8, 80)])
    for states in ([both[:, 0], both], [both[:, 0], both[:, 0, 1:]], [both[:, 0], both[:, :, 2]],
                   [flat[:640].view(8, 80), flat[639:1279].view(8, 80)], [flat.unfold(0, 80, 40)],
                   [kv[..., :17], kv[..., 16:]], [turned, turned[:, 1:]],
                   [turned[:, :, :20], turned[:, :, 19:]]):
        with pytest.raises(ValueError):
            b.BeamStates(states)
    with pytest.raises(ValueError):
        b.BeamStates([both[:4, 0]], out=[both[3:7, 0]])
    # every layout of a few bytes against the bytes themselves
    def places(p, step, rows, seg, n, size):
        return [p + r * step + k * seg + i for r in range(rows) for k in range(n) for i in range(size)]
    rng = random.Random(5)
    found = [0, 0]
    for _ in range(4000):
        n = rng.randint(1, 3)
        layout = (rng.choice([1, 2, 4, 6, 8, 12]), rng.randint(1, 4),
                  rng.choice([2, 3, 6, 12]) if n > 1 else 0, n, rng.randint(1, 3))
        one = (100, *layout)
        two = (100 + rng.randint(-30, 30), layout[0], rng.randint(1, 4), *layout[2:])
        mine = places(*one)
        assert b._shared(one) == (len(set(mine)) < len(mine))
        if b._shared(one) or b._shared(two):
            continue
        shared = b._shared(one, two)
        assert shared == bool(set(mine) & set(places(*two)))
        found[shared] += 1
    assert min(found) > 200


# ------------------------------------------------------------------- reference
def test_reference_quantisation_is_torchs_rounding():
    """The reference's rounding to e4m3 against torch's conversion, and its
    scales at the borders of 448 2^e."""
    y = torch.cat([torch.linspace(-448, 448, 100001, dtype=torch.float64),
                   torch.linspace(-0.05, 0.05, 5001, dtype=torch.float64)])
    y = torch.cat([y, torch.full((128 - len(y) % 128,), 448.0, dtype=torch.float64)]).view(-1, 128)
    y = y.float().double()
    y[:, 0] = 448.0
    q, s = block_ref.quantize(y, 1)
    assert torch.equal(s, torch.ones_like(s))
    assert torch.equal(q, y.float().to(torch.float8_e4m3fn).double())
    x = torch.zeros(6, 128, dtype=torch.float64)
    x[0, 5], x[1, 5], x[2, 5] = 448.0, 448.0 + 2.0 ** -15, 449.0
    x[3, 5], x[4, 5], x[5, 5] = 2.0 ** -149, math.nan, 0.0
    q, s = block_ref.quantize(x, 1)
    assert s[:4, 0].tolist() == [1.0, 2.0, 2.0, 2.0 ** -126] and bool(s[4].isnan()) and s[5, 0] == 1


def test_reference_selection_on_a_small_case():
    z = torch.tensor([[0.0, 1.0, 1.0], [3.0, -math.inf, 0.0]])
    p, t, v = block_ref.select(z, torch.tensor([[-1.0, -1.5]]), 5)
    a = torch.log_softmax(z[0].double(), 0) - 1.0
    c = torch.log_softmax(z[1].double(), 0) - 1.5
    assert p.tolist() == [[1, 0, 0, 0, 1]] and t.tolist() == [[0, 1, 2, 0, 2]]
    assert torch.allclose(v[0], torch.stack([c[0], a[1], a[2], a[0], c[2]]))
