"""Numbers past the C integers of the beam calls are refused, not wrapped (no
GPU)."""
import pytest

torch = pytest.importorskip("torch")

from invariant_output_head_gb300 import binding as b                        # noqa: E402
from tests.test_block_beam_cpu import calls, fake, head_of                  # noqa: E402, F401


def refused(call):
    with pytest.raises(b.DetlmError) as e:
        call()
    assert e.value.status == b.DETLM_EINVAL


def test_end_tokens_outside_the_vocabulary(calls):                          # noqa: F811
    head = head_of(fake(50, 16, dtype=torch.bfloat16), "bf16")
    z, s, done = fake(12, 50), fake(3, 4), fake(3, 4, dtype=torch.bool)
    out = b.Beams(fake(3, 8, dtype=torch.int32), fake(3, 8, dtype=torch.int32), fake(3, 8))
    for end in (50, -1, 2**31, 2**32 + 5, -2**32 + 5, 2**64 + 5):
        refused(lambda: head.beam_select(z, s, 8, finished=done, end_token=end, out=out))
    assert not calls
    for end in (0, 5, 49):
        head.beam_select(z, s, 8, finished=done, end_token=end, out=out)
        assert calls.pop()[1][5] == end
    # without finished beams no end token is proposed, whatever it is
    head.beam_select(z, s, 8, end_token=-1, out=out)
    assert len(calls) == 1


def test_numbers_of_continuations_past_32_bits(calls, monkeypatch):         # noqa: F811
    head = head_of(fake(50, 16, dtype=torch.bfloat16), "bf16")
    made = []
    monkeypatch.setattr(b, "detlm_head_reserve_beams", lambda *a: made.append(a))
    monkeypatch.setattr(b, "beam_buffers", lambda *a: pytest.fail("buffers of a refused call"))
    for n in (0, 65, 2**32 + 5, -2**32 + 5):
        refused(lambda: head.beam_select(fake(12, 50), fake(3, 4), n))
        refused(lambda: head.reserve_beams(12, n))
    for rows in (-1, 2**31, 2**64 + 12):
        refused(lambda: head.reserve_beams(rows, 8))
    assert not calls and not made
    head.reserve_beams(12, 8)
    assert made == [(None, 12, 8)]
