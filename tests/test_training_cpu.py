"""The differentiable score's dealings with autograd, on a stand-in head that
computes the two calls in plain torch operations."""
import pytest

torch = pytest.importorskip("torch")

from invariant_output_head_gb300.binding import Score                   # noqa: E402
from invariant_output_head_gb300.training import scored_logprobs        # noqa: E402


class _Head:
    def __init__(self, W):
        self.W = W
        self.given = []          # (dlogp, dentropy) of each gradient call

    def score(self, h, targets, temperature=1.0):
        with torch.no_grad():
            logp = torch.log_softmax(h @ self.W.t() / temperature, dim=1)
            lse = torch.logsumexp(h @ self.W.t() / temperature, dim=1)
            return Score(logp.gather(1, targets.long()[:, None])[:, 0],
                         -(logp.exp() * logp).sum(dim=1), lse, None, None)

    def score_backward(self, h, targets, lse, entropy, dlogp, dentropy, temperature=1.0,
                       need_dh=True, need_dW=True):
        self.given.append((dlogp, dentropy))
        logp = h @ self.W.t() / temperature - lse[:, None]
        dz = -logp.exp() * dlogp[:, None]
        if dentropy is not None:
            dz = dz - dentropy[:, None] * logp.exp() * (logp + entropy[:, None])
        dz[torch.arange(len(h)), targets.long()] += dlogp
        dz = dz / temperature
        return (dz @ self.W if need_dh else None), (dz.t() @ h if need_dW else None)


@pytest.fixture
def case():
    g = torch.Generator().manual_seed(3)
    W = torch.randn(30, 8, generator=g).requires_grad_()
    h = torch.randn(5, 8, generator=g).requires_grad_()
    t = torch.randint(0, 30, (5,), generator=g, dtype=torch.int32)
    return _Head(W), h, t


def _reference(head, h, t, T=1.0):
    logp = torch.log_softmax(h @ head.W.t() / T, dim=1)
    return logp.gather(1, t.long()[:, None])[:, 0], -(logp.exp() * logp).sum(dim=1)


def test_gradients_of_either_output(case):
    """An output that the loss does not use costs no term of the gradient."""
    head, h, t = case
    for pick in ((1, 0), (0, 1), (1, 1)):
        logp, entropy = scored_logprobs(head, h, t, 0.8)
        rlogp, rentropy = _reference(head, h, t, 0.8)
        loss, rloss = 0, 0
        if pick[0]:
            loss, rloss = loss + logp.sin().sum(), rloss + rlogp.sin().sum()
        if pick[1]:
            loss, rloss = loss + entropy.cos().sum(), rloss + rentropy.cos().sum()
        got = torch.autograd.grad(loss, (h, head.W))
        want = torch.autograd.grad(rloss, (h, head.W))
        for a, b in zip(got, want):
            assert torch.allclose(a, b, rtol=1e-4, atol=1e-5)
        dlogp, dentropy = head.given[-1]
        assert (dentropy is not None) == bool(pick[1])
        assert dlogp is not None and bool((dlogp != 0).any()) == bool(pick[0])


def test_a_second_derivative_is_refused(case):
    """The gradient call is not differentiable: a gradient penalty has to say
    so instead of ending without that term."""
    head, h, t = case
    logp, _ = scored_logprobs(head, h, t)
    (plain,) = torch.autograd.grad(logp.sum(), h, retain_graph=True)
    assert not plain.requires_grad
    (dh,) = torch.autograd.grad(logp.sum(), h, create_graph=True)
    with pytest.raises(RuntimeError, match="twice"):
        (logp.sum() + dh.square().sum()).backward()


def test_weights_changed_between_forward_and_backward_are_refused(case):
    """The log-sum-exp of the old weights does not fit logits of the new."""
    head, h, t = case
    logp, _ = scored_logprobs(head, h, t)
    with torch.no_grad():
        head.W += 0.1
    with pytest.raises(RuntimeError, match="inplace"):
        logp.sum().backward()


def test_rows_changed_between_forward_and_backward_are_refused(case):
    head, h, t = case
    logp, _ = scored_logprobs(head, h, t)
    with torch.no_grad():
        h += 0.1
    with pytest.raises(RuntimeError, match="inplace"):
        logp.sum().backward()
