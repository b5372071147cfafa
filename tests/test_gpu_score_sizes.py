"""The score call and its gradient at hidden sizes of several accumulation
chunks (512 elements of d in the score, 2048 in the gradient's first product),
on logits that round, and beside the log-prob and greedy calls."""
import numpy as np
import pytest

from tests import score_ref as ref
from tests.test_gpu_score import _check_score, _gradient_case, _head, _host, _p_terms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V,d,B,K,T,dtype", [
    (1000, 4096, 3, 5, 1.0, "bf16"), (700, 4104, 130, 8, 0.8, "fp16"),
    (2001, 2056, 40, 20, 1.0, "bf16"), (600, 8192, 300, 4, 1.0, "bf16"),
    (1352, 5120, 5200, 2, 1.0, "bf16"), (513, 1032, 257, 0, 1.3, "fp16"),
])
def test_score_of_several_chunks(V, d, B, K, T, dtype):
    import torch
    W, h, t = ref.grid_inputs(51 + V + B, V, d, B, masked=0.1)
    head = _head(W, dtype)
    got = head.score(ref.to_dev(h, dtype), torch.from_numpy(t).cuda(), top_k=K, temperature=T)
    assert head.check() == 0
    _check_score(got, ref.score(W, h, t, K, T), K, T)


@pytest.mark.parametrize("V,d,B,dtype,T,with_entropy", [
    (500, 4096, 5, "bf16", 1.0, True), (700, 4104, 130, "fp16", 0.9, True),
    (300, 2056, 40, "bf16", 1.0, False), (600, 8192, 300, "bf16", 1.0, True),
    (33000, 2112, 129, "bf16", 1.0, True), (400, 5120, 2200, "fp16", 1.2, True),
])
def test_gradient_of_several_chunks(V, d, B, dtype, T, with_entropy):
    import torch
    W, h, t, dlogp, dent = _gradient_case(V, d, B, dtype, T, with_entropy)
    head = _head(W, dtype)
    hd, td = ref.to_dev(h, dtype), torch.from_numpy(t).cuda()
    s = head.score(hd, td, temperature=T)
    de = None if dent is None else torch.from_numpy(dent).cuda()
    dh, dW = head.score_backward(hd, td, s.lse, s.entropy, torch.from_numpy(dlogp).cuda(), de,
                                 temperature=T)
    assert head.check() == 0
    want = ref.gradient(W, h, t, dlogp, dent, T)
    tol_h, tol_W = ref.gradient_tol(want, W, h, _p_terms(W, h, t, dlogp, dent, T), dtype)
    assert (np.abs(_host(dh) - want["dh"]) <= tol_h).all()
    assert (np.abs(_host(dW) - want["dW"]) <= tol_W).all()


def _normal(V, d, B, dtype, seed=1):
    """W, h of normal values (no grid: logits round), as 64-bit arrays of the
    16-bit values, targets, and the magnitudes sum_k |h_k W_k| of each logit."""
    import torch
    g = torch.Generator().manual_seed(seed + V + d + B)
    to = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    W = (torch.randn(V, d, generator=g) * 3.0 / np.sqrt(d)).to(to)
    h = torch.randn(B, d, generator=g).to(to)
    t = torch.randint(0, V, (B,), generator=g, dtype=torch.int32)
    W64, h64 = W.double().numpy(), h.double().numpy()
    return W.cuda(), h.cuda(), t.cuda(), W64, h64, t.numpy(), np.abs(h64) @ np.abs(W64).T


def _logit_tol(d, chunk, A):
    """A chunk's sum in the tensor core: an MMA step adds 16 products to the
    running sum; taking each step's alignment and addition to lose at most a
    unit of fp32's last place (2^-23) of the magnitudes so far, chunk / 16 of
    them; then one rounding (2^-24) for each chunk added to the others."""
    return (chunk / 16 * 2.0 ** -23 + (d / chunk + 1) * 2.0 ** -24) * A


_ROUNDING = [(1000, 520, 7, "bf16"), (1000, 4096, 5, "bf16"), (900, 4104, 200, "fp16"),
             (800, 8192, 300, "bf16"), (3000, 1536, 1100, "fp16"), (1352, 1024, 4400, "bf16")]


@pytest.mark.parametrize("V,d,B,dtype", _ROUNDING)
def test_score_of_logits_that_round(V, d, B, dtype):
    """A logit's error e moves log-sum-exp by at most its largest over the row,
    log p by twice that, the entropy by |dH/dz| = p |log p + H| summed, at most
    2 H + 1 times it."""
    from invariant_output_head_gb300 import Head
    W, h, t, W64, h64, t64, A = _normal(V, d, B, dtype)
    head = Head(W)
    s = head.score(h, t, top_k=4)
    want = ref.score(W64, h64, t64, 4, 1.0)
    e = _logit_tol(d, 512, A).max(axis=1)
    assert (np.abs(_host(s.lse) - want["lse"]) <= e + ref.lse_tol(want["lse"])).all()
    assert (np.abs(_host(s.logp) - want["logp"]) <= 2 * e + ref.logp_tol(want["logp"], 0)).all()
    assert (np.abs(_host(s.entropy) - want["entropy"])
            <= (2 * want["entropy"] + 1) * e + ref.entropy_tol(want["entropy"])).all()
    # alternatives: in order, each as probable as the place it takes
    top = s.top_token.cpu().numpy()
    logp, _ = ref.logsoftmax(h64 @ W64.T)
    mine = np.take_along_axis(logp, top, axis=1)
    tol = 2 * e[:, None] + ref.logp_tol(want["top_logp"], 0)
    assert (np.abs(mine - want["top_logp"]) <= tol).all()
    assert (np.abs(_host(s.top_logp) - mine) <= tol).all()
    assert all(len(set(r)) == 4 for r in top.tolist())
    assert head.check() == 0


@pytest.mark.parametrize("V,d,B,dtype", _ROUNDING)
def test_score_beside_the_logprob_and_greedy_calls(V, d, B, dtype):
    """Their logits are sums of 128-element chunks: the log-probabilities agree
    to both calls' errors, and the first alternative is the greedy token unless
    the two logits are that close."""
    from invariant_output_head_gb300 import Head
    W, h, t, W64, h64, t64, A = _normal(V, d, B, dtype)
    head = Head(W)
    s = head.score(h, t, top_k=2)
    lp = _host(head.logprob(h, t))
    e = (_logit_tol(d, 512, A) + _logit_tol(d, 128, A)).max(axis=1)
    assert (np.abs(_host(s.logp) - lp) <= 2 * e + 2 * ref.logp_tol(lp, 0)).all()
    token = head.greedy(h)[0].cpu().numpy()
    first = s.top_token[:, 0].cpu().numpy()
    z = h64 @ W64.T
    n = np.arange(B)
    assert (np.abs(z[n, token] - z[n, first]) <= 2 * e)[token != first].all()
    assert head.check() == 0


@pytest.mark.parametrize("V,d,B,dtype", [(1000, 520, 7, "bf16"), (500, 4096, 140, "bf16"),
                                         (700, 4104, 130, "fp16"), (3000, 1536, 400, "bf16")])
def test_gradient_of_logits_that_round(V, d, B, dtype):
    """gradient_tol's parts, and the logits' errors e: p is off by 2 e of
    itself (log-sum-exp takes part), p (log p + H) by that and the factor's own
    error, 2 e + (2 H + 1) e: (2 H + 5) e of the parts' magnitudes covers both."""
    import torch
    from invariant_output_head_gb300 import Head
    W, h, t, W64, h64, t64, A = _normal(V, d, B, dtype)
    rng = np.random.Generator(np.random.PCG64(3))
    dl = (rng.standard_normal(B) * 8).astype(np.float32)
    de = (rng.standard_normal(B) * 0.5).astype(np.float32)
    head = Head(W)
    s = head.score(h, t)
    dh, dW = head.score_backward(h, t, s.lse, s.entropy, torch.from_numpy(dl).cuda(),
                                 torch.from_numpy(de).cuda())
    want = ref.gradient(W64, h64, t64, dl, de, 1.0)
    terms = _p_terms(W64, h64, t64, dl, de, 1.0)
    tol_h, tol_W = ref.gradient_tol(want, W64, h64, terms, dtype)
    p = np.exp(ref.logsoftmax(h64 @ W64.T)[0])
    e = (_logit_tol(d, 2048, A) + _logit_tol(d, 512, A)).max(axis=1)[:, None]
    more = (2 * want["entropy"][:, None] + 5) * e * (terms + p * np.abs(de)[:, None])
    assert (np.abs(_host(dh) - want["dh"]) <= tol_h + more @ np.abs(W64)).all()
    assert (np.abs(_host(dW) - want["dW"]) <= tol_W + more.T @ np.abs(h64)).all()
    assert head.check() == 0
