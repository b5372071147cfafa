"""The score call, its gradient and the scaled logits at the ends of their
ranges: workspaces of many rows, logits far apart or infinite."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_B,B", [
    (30000, 29127),     # the last row count of nine segments a pass; 30000 has eight
    (26300, 26214),     # the last of all ten
])
def test_reserved_gradients_of_many_rows_allocate_nothing(max_B, B):
    """dz of the whole vocabulary does not fit one pass: fewer rows can need
    more memory than more rows."""
    import torch
    from invariant_output_head_gb300 import Head
    V, d = 151936, 8
    g = torch.Generator(device="cuda").manual_seed(B)
    W = torch.randn(V, d, generator=g, device="cuda").bfloat16()
    h = torch.randn(B, d, generator=g, device="cuda").bfloat16()
    t = torch.randint(0, V, (B,), generator=g, device="cuda", dtype=torch.int32)
    dl = torch.randn(B, generator=g, device="cuda") / B
    grads = (torch.empty_like(h), torch.empty_like(W))
    first = Head(W)                        # (kernels are loaded by their first launch)
    s = first.score(h, t)
    first.score_backward(h, t, s.lse, s.entropy, dl, out=grads)
    first.close()
    head = Head(W)
    head.reserve_score(B)
    head.reserve_backward(max_B)
    out = head.score_buffers(B)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    s = head.score(h, t, out=out)
    head.score_backward(h, t, s.lse, s.entropy, dl, out=grads)
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free
    assert head.check() == 0
    head.close()


def _far_apart(B, top, rest, x):
    """A head of 300 entries whose logits are top * x for the last and rest * x
    for the others, on B equal rows."""
    import torch
    from invariant_output_head_gb300 import Head
    W = torch.zeros(300, 16, dtype=torch.bfloat16, device="cuda")
    W[:, 0] = rest
    W[299, 0] = top
    h = torch.zeros(B, 16, dtype=torch.bfloat16, device="cuda")
    h[:, 0] = x
    return Head(W), h


@pytest.mark.parametrize("B", [4, 300])
@pytest.mark.parametrize("top,rest,x", [
    (2.0 ** 20, -(2.0 ** 20), 2.0 ** 100),       # far apart, and far from zero
    (0.0, -(2.0 ** 100), 2.0 ** 100),            # the others' logits are -inf
    (2.0 ** 27, -(2.0 ** 27), 2.0 ** 100),       # their distance is not finite
])
def test_score_of_a_distribution_on_one_token(top, rest, x, B):
    import torch
    head, h = _far_apart(B, top, rest, x)
    t = torch.full((B,), 299, dtype=torch.int32, device="cuda")
    t[0] = 7
    for K in (2, 0):
        s = head.score(h, t, top_k=K)
        assert (s.lse == top * x).all() and (s.entropy == 0).all()
        assert (s.logp[1:] == 0).all()
        assert s.logp[0].item() == torch.tensor((rest - top) * x).item()     # -inf past fp32
    s = head.score(h, t, top_k=2)
    assert s.top_token.tolist() == [[299, 0]] * B and (s.top_logp[:, 0] == 0).all()
    assert head.check() == 0


@pytest.mark.parametrize("B", [4, 300])
def test_infinite_logits_at_a_huge_temperature(B):
    """A logit of -inf has no probability at any temperature."""
    import torch
    head, h = _far_apart(B, 0.0, -(2.0 ** 100), 2.0 ** 100)
    head.W[298] = 0.0
    t = torch.full((B,), 298, dtype=torch.int32, device="cuda")
    for T in (1.0, 1e36, 1e38, 3e38):
        s = head.score(h, t, temperature=T)
        log2 = 0.6931471805599453
        # one rounding each of log S and of the differences, 2^-23 of them
        for got, want in ((s.lse, log2), (s.entropy, log2), (s.logp, -log2)):
            assert ((got.double() - want).abs() <= 2e-7).all()
    assert head.check() == 0


def test_temperatures_whose_inverse_overflows_are_refused():
    """1 / T and log2(e) / T, by which logits are scaled, have to be finite."""
    import torch
    from invariant_output_head_gb300 import DETLM_EINVAL, DetlmError
    head, h = _far_apart(3, 1.0, 0.0, 1.0)
    t = torch.zeros(3, dtype=torch.int32, device="cuda")
    ok = head.score(h, t, temperature=5e-39)
    assert (ok.entropy == 0).all() and not torch.isnan(ok.lse).any()
    for T in (1e-39, 2.9e-39, 3e-39, 4e-39):
        for call in (lambda: head.score(h, t, temperature=T),
                     lambda: head.score_backward(h, t, ok.lse, ok.entropy, ok.entropy,
                                                 temperature=T)):
            with pytest.raises(DetlmError) as e:
                call()
            assert e.value.status == DETLM_EINVAL
    assert head.check() == 0


@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("B", [4, 300])
@pytest.mark.parametrize("top,rest,x", [
    (2.0 ** 20, -(2.0 ** 20), 2.0 ** 100),       # far apart, and far from zero
    (0.0, -(2.0 ** 100), 2.0 ** 100),            # the others' logits are -inf
    (2.0 ** 27, -(2.0 ** 27), 2.0 ** 100),       # their distance is not finite
])
def test_gradient_of_a_distribution_on_one_token(top, rest, x, B, entropy):
    """p is 1 on the last entry and 0 elsewhere, so dz is g at the target and
    -g at the last entry; the entropy term is 0 (p (log p + H) -> 0). All of it
    is exact: one row a target, powers of two."""
    import torch
    head, h = _far_apart(B, top, rest, x)
    t = torch.full((B,), 299, dtype=torch.int32, device="cuda")
    t[0] = 7
    s = head.score(h, t)
    assert (s.lse == top * x).all() and (s.entropy == 0).all()
    dl = torch.full((B,), 2.0 ** -90, device="cuda")
    de = torch.full((B,), 0.5, device="cuda") if entropy else None
    dh, dW = head.score_backward(h, t, s.lse, s.entropy, dl, de)
    want_h = torch.zeros_like(h)
    want_h[0, 0] = 2.0 ** -90 * (rest - top)
    want_W = torch.zeros_like(head.W)
    want_W[7, 0] = 2.0 ** -90 * x
    want_W[299, 0] = -(2.0 ** -90) * x
    assert torch.equal(dh, want_h) and torch.equal(dW, want_W)
    assert head.check() == 0


def _fp16_gradient(V, d, B, seed):
    from tests import score_ref as ref
    import numpy as np
    import torch
    from invariant_output_head_gb300 import Head
    W, h, t = ref.grid_inputs(seed, V, d, B)
    rng = np.random.Generator(np.random.PCG64(seed))
    dl, de = rng.standard_normal(B), 0.1 * rng.standard_normal(B)
    head = Head(ref.to_dev(W, "fp16"))
    hd, td = ref.to_dev(h, "fp16"), torch.from_numpy(t).cuda()
    return W, h, t, head, hd, td, head.score(hd, td), dl.astype(np.float32), de.astype(np.float32)


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_fp16_rows_beside_one_whose_gradient_is_not_finite(value):
    """A row whose loss overflowed leaves the other rows' dh as it is without
    that row, bit for bit. (Its own dh, and dW, are not finite.)"""
    import torch
    *_, head, hd, td, s, dl, de = _fp16_gradient(3000, 72, 90, 17)
    dl, de = torch.from_numpy(dl * 1e-3).cuda(), torch.from_numpy(de * 1e-3).cuda()
    keep = torch.arange(90, device="cuda") != 40
    want, _ = head.score_backward(*(x[keep].contiguous() for x in (hd, td, s.lse, s.entropy, dl, de)),
                                  need_dW=False)
    assert (want != 0).float().mean() > 0.9
    dl[40] = value
    got, dW = head.score_backward(hd, td, s.lse, s.entropy, dl, de, temperature=1.0)
    assert torch.equal(got[keep], want)
    assert not torch.isfinite(got[40]).any() and not torch.isfinite(dW).all()
    assert head.check() == 0


@pytest.mark.parametrize("ratio", [2.0 ** -8, 2.0 ** -18])
def test_fp16_rows_beside_rows_of_larger_gradients(ratio):
    """dz is held in fp16 times a power of two S of the whole call. C, the
    largest (|dlogp| + |dentropy| (1 + log V)) / T, times S lies in [2^13, 2^14):
    a stored value is off by at most half a step of the subnormals, 2^-25 / S <=
    2^-38 C, beyond its 11 bits, in the call and in the smaller one alike. dh
    adds 5e-5 of the terms' magnitudes for the exponentials and the sums and,
    rounded twice, 2^-10 of itself and a step of fp16's subnormals."""
    import numpy as np
    import torch
    from tests import score_ref as ref
    V, B, small = 3000, 200, 50
    W, h, t, head, hd, td, s, dl, de = _fp16_gradient(V, 72, B, 23)
    dl[:small] *= ratio
    de[:small] *= ratio
    args = [hd, td, s.lse, s.entropy, torch.from_numpy(dl).cuda(), torch.from_numpy(de).cuda()]
    full = head.score_backward(*args, need_dW=False)[0][:small].double().cpu().numpy()
    part = head.score_backward(*(x[:small].contiguous() for x in args), need_dW=False)[0]
    part = part.double().cpu().numpy()
    C = (np.abs(dl) + np.abs(de) * (1 + np.log(V))).max()
    logp, _ = ref.logsoftmax(h[:small] @ W.T)
    p = np.exp(logp)
    H = -(p * logp).sum(axis=1, keepdims=True)
    terms = p * (np.abs(dl[:small, None]) + np.abs(de[:small, None]) * (np.abs(logp) + H))
    terms[np.arange(small), t[:small]] += np.abs(dl[:small])
    rounded = 2.0 ** -10 * np.abs(part) + 2.0 ** -24 + 5e-5 * (terms @ np.abs(W))
    assert (np.abs(full - part) <= 2.0 ** -37 * C * np.abs(W).sum(axis=0) + rounded).all()
    # and against the formula, with the call's own C
    g = ref.gradient(W, h, t, dl, de, 1.0)["dh"][:small]
    each = 2.0 ** -11 * (terms @ np.abs(W))
    assert (np.abs(full - g) <= 2.0 ** -38 * C * np.abs(W).sum(axis=0) + each + rounded).all()
    assert head.check() == 0
