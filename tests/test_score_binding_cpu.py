"""Argument checks of the score call's binding that need no GPU: tensors that
only claim to be on one, and the library call replaced by a list."""
import pytest

torch = pytest.importorskip("torch")

from invariant_output_head_gb300 import binding          # noqa: E402


class _OnDevice(torch.Tensor):
    """A host tensor that says it is a CUDA tensor (on `where`)."""
    is_cuda = True
    where = torch.device("cuda:0")

    @property
    def device(self):
        return self.where


class _OnOther(_OnDevice):
    where = torch.device("cuda:1")


@pytest.fixture
def head(monkeypatch):
    h = binding.Head.__new__(binding.Head)
    h.W = torch.zeros(40, 16, dtype=torch.bfloat16).as_subclass(_OnDevice)
    h.dtype, h.V, h.d, h.handle = "bf16", 40, 16, None
    h.calls = []
    monkeypatch.setattr(binding, "detlm_head_score", lambda *a: h.calls.append(a))
    monkeypatch.setattr(binding, "_stream_ptr", lambda s: 0)
    monkeypatch.setattr(h, "score_buffers", lambda *a: binding.Score(None, None, None, None, None),
                        raising=False)
    return h


def test_rows_of_the_heads_type_are_scored(head):
    head.score(torch.zeros(3, 16, dtype=torch.bfloat16).as_subclass(_OnDevice))
    assert len(head.calls) == 1


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32, torch.int8, torch.float64])
def test_rows_of_another_type_are_refused(head, dtype):
    with pytest.raises(ValueError):
        head.score(torch.zeros(3, 16, dtype=dtype).as_subclass(_OnDevice))
    assert head.calls == []


def test_rows_on_another_device_are_refused(head):
    with pytest.raises(ValueError):
        head.score(torch.zeros(3, 16, dtype=torch.bfloat16).as_subclass(_OnOther))
    assert head.calls == []
