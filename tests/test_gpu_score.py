"""The score call (log-probability, entropy, most likely tokens), its gradient
and the scaled logits of an int8 head, against plain 64-bit forms."""
import numpy as np
import pytest

from tests import score_ref as ref

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _head(W, dtype):
    from invariant_output_head_gb300 import Head
    return Head(ref.to_dev(W, dtype), dtype)


def _host(x):
    return None if x is None else x.detach().float().cpu().numpy().astype(np.float64)


def _check_score(got, want, K, T):
    assert (np.abs(_host(got.lse) - want["lse"]) <= ref.lse_tol(want["lse"])).all()
    assert (np.abs(_host(got.entropy) - want["entropy"]) <= ref.entropy_tol(want["entropy"])).all()
    if got.logp is not None:
        assert (np.abs(_host(got.logp) - want["logp"])
                <= ref.logp_tol(want["logp"], want["lse"])).all()
    if K:
        assert (got.top_token.cpu().numpy() == want["top_token"]).all()
        assert (np.abs(_host(got.top_logp) - want["top_logp"])
                <= ref.logp_tol(want["top_logp"], want["lse"])).all()


@pytest.mark.parametrize("V,d,B,K,T,dtype", [
    (1, 8, 1, 1, 1.0, "bf16"), (3, 8, 2, 3, 1.0, "bf16"), (32, 16, 5, 32, 0.5, "fp16"),
    (33, 64, 130, 32, 1.0, "bf16"), (127, 64, 17, 4, 1.0, "bf16"), (129, 72, 128, 8, 1.0, "fp16"),
    (257, 136, 129, 8, 2.0, "bf16"), (1000, 520, 64, 5, 1.0, "bf16"),
    (5001, 264, 1, 20, 0.7, "bf16"), (5001, 264, 300, 20, 0.7, "fp16"),
    (32000, 128, 3, 32, 1.0, "bf16"), (32000, 128, 513, 32, 1.0, "bf16"),
    (50001, 64, 260, 1, 1.3, "fp16"), (70000, 8, 129, 13, 1.0, "bf16"),
    (1352, 384, 1300, 5, 1.0, "bf16"), (20000, 64, 1100, 32, 1.0, "bf16"),
    (60000, 24, 1050, 8, 1.0, "fp16"), (9000, 40, 1500, 0, 0.8, "bf16"),
    (151936, 16, 450, 8, 1.0, "bf16"), (20000, 64, 2100, 32, 1.0, "bf16"),
    (1352, 64, 4400, 5, 1.0, "fp16"),
])
def test_score(V, d, B, K, T, dtype):
    torch = _torch()
    W, h, t = ref.grid_inputs(11 + V + B, V, d, B, masked=0.2)
    head = _head(W, dtype)
    got = head.score(ref.to_dev(h, dtype), torch.from_numpy(t).cuda(), top_k=K, temperature=T)
    assert head.check() == 0
    _check_score(got, ref.score(W, h, t, K, T), K, T)


@pytest.mark.parametrize("B", [2, 200])
def test_score_without_targets_or_alternatives(B):
    W, h, t = ref.grid_inputs(3, 700, 64, B)
    head = _head(W, "bf16")
    got = head.score(ref.to_dev(h, "bf16"))
    assert got.logp is None and got.top_token is None
    _check_score(got, ref.score(W, h, t, 0, 1.0), 0, 1.0)
    empty = head.score(ref.to_dev(h[:0], "bf16"), top_k=3)
    assert empty.entropy.shape == (0,) and empty.top_token.shape == (0, 3)
    assert head.check() == 0


def test_row_bits_do_not_depend_on_the_batch():
    torch = _torch()
    W, h, t = ref.grid_inputs(5, 9001, 328, 5200)
    head = _head(W, "bf16")
    # off-grid values too: the sums' rounding must not depend on B either
    noise = torch.randn(5200, 328, generator=torch.Generator().manual_seed(1)).cuda()
    hd = (ref.to_dev(h, "bf16").float() + noise).bfloat16()
    td = torch.from_numpy(t).cuda()
    full = head.score(hd, td, top_k=9, temperature=0.9)
    for rows in ([0], [5, 699], list(range(100, 117)), list(range(31, 159)),
                 list(range(300, 429)), list(range(690, 100, -1)), list(range(5000, 900, -2))):
        i = torch.tensor(rows, device="cuda")
        part = head.score(hd[i].contiguous(), td[i].contiguous(), top_k=9, temperature=0.9)
        for a, b in zip(full, part):
            assert torch.equal(a[i], b)
    assert head.check() == 0


@pytest.mark.parametrize("B", [4, 300, 1100, 1500])
def test_equal_and_ordered_logits(B):
    """Rows that admit every block as a candidate: all logits equal (a zero
    row), rising, and falling along the vocabulary."""
    torch = _torch()
    V, d, K = 40000, 16, 32
    W = np.zeros((V, d))
    v = np.arange(V)
    W[:, 0] = v // 200            # up to 199: exact in bf16, 200 entries share each value
    W[:, 1] = 1.0
    h = np.zeros((B, d))
    h[1::3, 0] = 0.0625
    h[2::3, 0] = -0.0625
    h[:, 1] = 0.5
    t = (v[:B] * 97 % V).astype(np.int32)
    head = _head(W, "bf16")
    got = head.score(ref.to_dev(h, "bf16"), torch.from_numpy(t).cuda(), top_k=K)
    assert head.check() == 0
    _check_score(got, ref.score(W, h, t, K, 1.0), K, 1.0)


@pytest.mark.parametrize("B", [3, 290])
def test_infinite_and_nan_logits(B):
    torch = _torch()
    V, d = 3000, 64
    W, h, t = ref.grid_inputs(8, V, d, B)
    hd = ref.to_dev(h, "bf16")
    hd[1, 3] = float("nan")
    head = _head(W, "bf16")
    td = torch.from_numpy(t).cuda()
    got = head.score(hd, td, top_k=4)
    want = ref.score(W, h, t, 4, 1.0)
    ok = np.arange(B) != 1
    for name in ("logp", "entropy", "lse"):
        x = _host(getattr(got, name))
        assert np.isnan(x[1]) and np.isfinite(x[ok]).all()
    assert (got.top_token.cpu().numpy()[ok] == want["top_token"][ok]).all()
    assert (got.top_token.cpu().numpy()[1] == -1).all()
    assert torch.isnan(got.top_logp[1]).all()
    # very large logits, one of them far above the rest: a distribution on it
    hd = torch.zeros((B, d), dtype=torch.bfloat16, device="cuda")
    hd[:, 0] = 2.0 ** 100
    Wb = torch.zeros((V, d), dtype=torch.bfloat16, device="cuda")
    Wb[:, 0] = -(2.0 ** 20)
    Wb[V - 1, 0] = 2.0 ** 20
    from invariant_output_head_gb300 import Head
    got = Head(Wb).score(hd, torch.full((B,), V - 1, dtype=torch.int32, device="cuda"), top_k=2)
    assert (got.logp == 0).all() and (got.entropy == 0).all()
    assert (got.top_token[:, 0] == V - 1).all() and (got.top_token[:, 1] == 0).all()


def test_bad_targets_are_reported():
    torch = _torch()
    W, h, t = ref.grid_inputs(9, 500, 64, 140)
    for B in (5, 140):
        tb = t[:B].copy()
        tb[2], tb[3], tb[4] = 500, -2, -1
        head = _head(W, "fp16")
        got = _host(head.score(ref.to_dev(h[:B], "fp16"), torch.from_numpy(tb).cuda()).logp)
        from invariant_output_head_gb300 import DETLM_ETARGET
        assert head.check() == DETLM_ETARGET
        assert np.isnan(got[2]) and np.isnan(got[3]) and got[4] == 0.0


# ---------------------------------------------------------------- gradient
def _gradient_case(V, d, B, dtype, T, with_entropy, seed=21):
    W, h, t = ref.grid_inputs(seed + V + B, V, d, B, masked=0.2)
    rng = np.random.Generator(np.random.PCG64(seed))
    scale = 64.0 if dtype == "fp16" else 1.0 / B
    dlogp = (rng.standard_normal(B) * scale).astype(np.float32)
    dent = (rng.standard_normal(B) * 0.05 * scale).astype(np.float32) if with_entropy else None
    return W, h, t, dlogp, dent


def _p_terms(W, h, t, dlogp, dent, T):
    logp, _ = ref.logsoftmax((h @ W.T) / T)
    p = np.exp(logp)
    H = -(p * logp).sum(axis=1, keepdims=True)
    out = p * np.where(t >= 0, np.abs(dlogp), 0.0)[:, None]
    if dent is not None:
        out = out + p * np.abs(dent)[:, None] * (np.abs(logp) + H)
    return out / T


@pytest.mark.parametrize("V,d,B,dtype,T,with_entropy", [
    (1, 8, 1, "bf16", 1.0, True), (5, 8, 1, "bf16", 1.0, False), (64, 16, 3, "fp16", 0.5, True),
    (257, 264, 65, "bf16", 1.0, True), (1000, 520, 7, "fp16", 1.0, False),
    (2049, 72, 129, "bf16", 2.0, True), (5001, 256, 300, "bf16", 1.0, True),
    (16385, 64, 257, "fp16", 0.9, True), (40000, 136, 20, "bf16", 1.0, False),
    (300, 72, 2500, "bf16", 1.0, True),
])
def test_gradient(V, d, B, dtype, T, with_entropy):
    torch = _torch()
    W, h, t, dlogp, dent = _gradient_case(V, d, B, dtype, T, with_entropy)
    head = _head(W, dtype)
    hd, td = ref.to_dev(h, dtype), torch.from_numpy(t).cuda()
    s = head.score(hd, td, temperature=T)
    dl = torch.from_numpy(dlogp).cuda()
    de = None if dent is None else torch.from_numpy(dent).cuda()
    dh, dW = head.score_backward(hd, td, s.lse, s.entropy, dl, de, temperature=T)
    assert head.check() == 0
    want = ref.gradient(W, h, t, dlogp, dent, T)
    tol_h, tol_W = ref.gradient_tol(want, W, h, _p_terms(W, h, t, dlogp, dent, T), dtype)
    assert (np.abs(_host(dh) - want["dh"]) <= tol_h).all()
    assert (np.abs(_host(dW) - want["dW"]) <= tol_W).all()
    # one of the two alone is the same; a second call is the same bits
    a, none = head.score_backward(hd, td, s.lse, s.entropy, dl, de, temperature=T, need_dW=False)
    assert none is None and torch.equal(a, dh)
    none, b = head.score_backward(hd, td, s.lse, s.entropy, dl, de, temperature=T, need_dh=False)
    assert none is None and torch.equal(b, dW)


def test_gradient_against_differences():
    """Central differences of the 64-bit loss along random directions."""
    torch = _torch()
    V, d, B, T = 700, 64, 40, 0.8
    W, h, t, dlogp, dent = _gradient_case(V, d, B, "bf16", T, True)
    head = _head(W, "bf16")
    hd, td = ref.to_dev(h, "bf16"), torch.from_numpy(t).cuda()
    s = head.score(hd, td, temperature=T)
    dh, dW = head.score_backward(hd, td, s.lse, s.entropy, torch.from_numpy(dlogp).cuda(),
                                 torch.from_numpy(dent).cuda(), temperature=T)
    want = ref.gradient(W, h, t, dlogp, dent, T)
    tol_h, tol_W = ref.gradient_tol(want, W, h, _p_terms(W, h, t, dlogp, dent, T), "bf16")
    rng = np.random.Generator(np.random.PCG64(4))
    eps = 1e-5
    for _ in range(5):
        u, w = rng.standard_normal(h.shape), rng.standard_normal(W.shape)
        num_h = (ref.loss(W, h + eps * u, t, dlogp, dent, T)
                 - ref.loss(W, h - eps * u, t, dlogp, dent, T)) / (2 * eps)
        num_W = (ref.loss(W + eps * w, h, t, dlogp, dent, T)
                 - ref.loss(W - eps * w, h, t, dlogp, dent, T)) / (2 * eps)
        # elementwise bounds along the direction, and 1e-7 of the magnitudes
        # for the difference quotient (eps^2 and rounding / eps)
        assert abs((_host(dh) * u).sum() - num_h) <= (tol_h * np.abs(u)).sum() + 1e-7
        assert abs((_host(dW) * w).sum() - num_W) <= (tol_W * np.abs(w)).sum() + 1e-7


def test_gradient_rows_do_not_depend_on_the_batch():
    torch = _torch()
    V, d, B = 36000, 136, 1400
    W, h, t, dlogp, dent = _gradient_case(V, d, B, "bf16", 1.0, True)
    head = _head(W, "bf16")
    hd, td = ref.to_dev(h, "bf16"), torch.from_numpy(t).cuda()
    s = head.score(hd, td)
    dl, de = torch.from_numpy(dlogp).cuda(), torch.from_numpy(dent).cuda()
    full, _ = head.score_backward(hd, td, s.lse, s.entropy, dl, de, need_dW=False)
    for rows in ([7], list(range(40, 300)), list(range(1399, 500, -1))):
        i = torch.tensor(rows, device="cuda")
        part, _ = head.score_backward(*(x[i].contiguous() for x in (hd, td, s.lse, s.entropy, dl, de)),
                                      need_dW=False)
        assert torch.equal(full[i], part)


def test_gradient_of_masked_and_shared_targets():
    """No target anywhere: only the entropy term; every row the same target."""
    torch = _torch()
    V, d, B = 3000, 64, 600
    W, h, t, dlogp, dent = _gradient_case(V, d, B, "bf16", 1.0, True)
    head = _head(W, "bf16")
    hd = ref.to_dev(h, "bf16")
    dl, de = torch.from_numpy(dlogp).cuda(), torch.from_numpy(dent).cuda()
    for same in (-1, 1234, V + 5):
        t[:] = same
        td = torch.from_numpy(t).cuda()
        s = head.score(hd)
        dh, dW = head.score_backward(hd, td, s.lse, s.entropy, dl, de)
        want = ref.gradient(W, h, t, dlogp, dent, 1.0)
        tol_h, tol_W = ref.gradient_tol(want, W, h, _p_terms(W, h, t, dlogp, dent, 1.0), "bf16")
        assert (np.abs(_host(dh) - want["dh"]) <= tol_h).all()
        assert (np.abs(_host(dW) - want["dW"]) <= tol_W).all()
    zero = torch.zeros_like(dl)
    dh, dW = head.score_backward(hd, td, s.lse, s.entropy, zero, zero)
    assert (dh == 0).all() and (dW == 0).all()
    dh, dW = head.score_backward(hd[:0], td[:0], s.lse[:0], s.entropy[:0], dl[:0], de[:0])
    assert dh.shape == (0, d) and (dW == 0).all()


def test_gradient_in_several_passes_over_the_vocabulary():
    """More rows than one pass's dz holds (about 8 GB): a row's dh is the bits
    of a call of few rows, and dW is that of two half batches added."""
    torch = _torch()
    from invariant_output_head_gb300 import Head
    V, d, B = 140001, 16, 40000
    g = torch.Generator(device="cuda").manual_seed(3)
    W = torch.randn(V, d, generator=g, device="cuda").bfloat16()
    h = torch.randn(B, d, generator=g, device="cuda").bfloat16()
    t = torch.randint(0, V, (B,), generator=g, device="cuda", dtype=torch.int32)
    t[::7] = 139999                               # a frequent token, in the last pass
    dl = torch.randn(B, generator=g, device="cuda") / B
    head = Head(W)
    s = head.score(h, t)
    dh, dW = head.score_backward(h, t, s.lse, s.entropy, dl)
    halves = []
    for i in (slice(0, B // 2), slice(B // 2, B)):
        part = head.score_backward(h[i].contiguous(), t[i].contiguous(), s.lse[i].contiguous(),
                                   s.entropy[i].contiguous(), dl[i].contiguous())
        assert torch.equal(part[0], dh[i])
        halves.append(part[1].float())
    few = head.score_backward(h[:3].contiguous(), t[:3].contiguous(), s.lse[:3].contiguous(),
                              s.entropy[:3].contiguous(), dl[:3].contiguous())
    assert torch.equal(few[0], dh[:3])
    # each half and the whole are rounded once to bf16 (2^-8 of themselves at
    # most), and their fp32 sums differ by 1e-5 of the halves' magnitudes
    a, b = halves
    tol = 2.0 ** -8 * (a.abs() + b.abs() + dW.float().abs()) * 1.01 + 1e-9
    assert ((dW.float() - (a + b)).abs() <= tol).all()
    assert head.check() == 0


# ------------------------------------------------------------ scaled logits
@pytest.mark.parametrize("V,d,B", [(1, 16, 1), (130, 32, 5), (3, 2048, 8), (5001, 4112, 7),
                                   (1000, 16384, 6), (1001, 16384, 4), (257, 528, 3), (2000, 64, 2), (1000, 1040, 33), (1001, 272, 64),
                                   (5001, 512, 200), (5000, 512, 256), (5001, 2064, 300),
                                   (4996, 512, 700)])
@pytest.mark.parametrize("out", ["float32", "bfloat16", "float16"])
def test_scaled_logits(V, d, B, out):
    torch = _torch()
    from invariant_output_head_gb300 import Head
    rng = np.random.Generator(np.random.PCG64(V + d + B))
    W = rng.integers(-128, 128, (V, d), dtype=np.int8)
    q = rng.integers(-128, 128, (B, d), dtype=np.int8)
    sx = (rng.random(B) * 0.02 + 1e-4).astype(np.float32)
    sw = (rng.random(V) * 1e-3 + 1e-5).astype(np.float32)
    sw[::7] = 0.0
    head = Head(torch.from_numpy(W).cuda())
    got = head.scaled_logits(torch.from_numpy(q).cuda(), torch.from_numpy(sx).cuda(),
                             torch.from_numpy(sw).cuda(), out_dtype=getattr(torch, out))
    assert head.check() == 0 and got.dtype == getattr(torch, out)
    acc = (q.astype(np.float64) @ W.astype(np.float64).T).astype(np.float32)   # one rounding
    y = acc * (sx[:, None] * sw[None, :])                                      # fp32, one each
    want = torch.from_numpy(y).to(getattr(torch, out))
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("B", [1, 3, 8, 20, 70, 300])
def test_scaled_logits_of_the_largest_sums(B):
    """All values -128 at the largest d: partial sums reach 2^24 in every
    kernel's chunks, the whole sum 2^28."""
    torch = _torch()
    from invariant_output_head_gb300 import Head
    V, d = 300, 16384
    W = torch.full((V, d), -128, dtype=torch.int8, device="cuda")
    W[1::3] = 127
    W[2::3, ::2] = 127
    q = torch.full((B, d), -128, dtype=torch.int8, device="cuda")
    got = Head(W).scaled_logits(q, torch.ones(B, device="cuda"), torch.ones(V, device="cuda"))
    want = (q.double() @ W.double().t()).float()
    assert torch.equal(got, want)


def test_scaled_logits_with_the_integer_front_end():
    """Float rows through quantize_rows: the scale of a row is 2^S / M."""
    torch = _torch()
    from invariant_output_head_gb300 import Head, quantize_rows
    g = torch.Generator().manual_seed(2)
    x = torch.randn(9, 256, generator=g).bfloat16().cuda()
    W = torch.randint(-127, 128, (800, 256), generator=g, dtype=torch.int8).cuda()
    sw = (torch.rand(800, generator=g) * 1e-3).cuda()
    q, M, S = quantize_rows(x)
    sx = torch.ldexp(torch.ones_like(M, dtype=torch.float32), S) / M.float()
    got = Head(W).scaled_logits(q, sx, sw)
    want = x.double() @ (W.double() * sw.double()[:, None]).t()
    # |x - q 2^S / M| <= half a step (a step is 2^S / M)
    tol = 0.5 * sx.double()[:, None] * (W.double().abs().sum(1) * sw.double())[None, :] * 1.001
    assert ((got.double() - want).abs() <= tol + 1e-6 * want.abs()).all()


# ---------------------------------------------------------------- refusals
def test_refusals():
    torch = _torch()
    from invariant_output_head_gb300 import (DETLM_EINVAL, DETLM_EUNSUPPORTED, DetlmError, Head)
    W, h, t = ref.grid_inputs(2, 40, 16, 3)
    head = _head(W, "bf16")
    hd, td = ref.to_dev(h, "bf16"), torch.from_numpy(t).cuda()
    s = head.score(hd, td)

    def refused(status, call):
        with pytest.raises(DetlmError) as e:
            call()
        assert e.value.status == status

    for T in (0.0, -1.0, float("nan"), float("inf"), 1e-45):
        refused(DETLM_EINVAL, lambda: head.score(hd, td, temperature=T))
        refused(DETLM_EINVAL, lambda: head.score_backward(hd, td, s.lse, s.entropy, s.logp,
                                                          temperature=T))
    refused(DETLM_EINVAL, lambda: head.score(hd, td, top_k=33))
    refused(DETLM_EINVAL, lambda: _head(W[:4], "bf16").score(hd, td, top_k=5))
    for bad in (td.long(), td[:2], td.cpu()):
        with pytest.raises(ValueError):
            head.score(hd, bad)
    with pytest.raises(ValueError):
        head.score(hd.t(), td)
    with pytest.raises(ValueError):
        head.score(hd, td, top_k=2, out=head.score_buffers(3, 1))
    with pytest.raises(ValueError):
        head.score(hd, None, out=head.score_buffers(3))
    with pytest.raises(ValueError):
        head.score_backward(hd, td, s.lse.double(), s.entropy, s.logp)
    with pytest.raises(ValueError):
        head.score_backward(hd.half(), td, s.lse, s.entropy, s.logp)
    with pytest.raises(ValueError):
        head.score_backward(hd, td, s.lse, s.entropy, s.logp, out=(hd, hd))
    with pytest.raises(DetlmError):
        head.scaled_logits(hd, s.lse, s.lse)

    W8 = torch.zeros((40, 16), dtype=torch.int8, device="cuda")
    q = torch.zeros((3, 16), dtype=torch.int8, device="cuda")
    sw = torch.ones(40, device="cuda")
    h8 = Head(W8)
    refused(DETLM_EUNSUPPORTED, lambda: h8.score(q))
    refused(DETLM_EUNSUPPORTED, lambda: h8.reserve_score(3))
    refused(DETLM_EUNSUPPORTED, lambda: h8.reserve_backward(3))
    with pytest.raises(ValueError):
        h8.scaled_logits(q, s.lse, sw[:39])
    with pytest.raises(ValueError):
        h8.scaled_logits(q, s.lse, sw, out_dtype=torch.int32)
    with pytest.raises(ValueError):
        h8.scaled_logits(q, s.lse, sw, out=torch.empty(3, 41, device="cuda"))
    assert head.check() == 0 and h8.check() == 0


# ------------------------------------------------- workspaces, streams, graphs
def test_reserved_calls_on_another_stream_and_in_a_graph():
    torch = _torch()
    W, h, t = ref.grid_inputs(31, 4000, 128, 300)
    head = _head(W, "bf16")
    head.reserve_score(300, 8)
    head.reserve_backward(300)
    hd, td = ref.to_dev(h, "bf16"), torch.from_numpy(t).cuda()
    dl = torch.linspace(-1, 1, 300, device="cuda")
    free = torch.cuda.mem_get_info()[0]
    s = head.score(hd, td, top_k=8)
    dh, dW = head.score_backward(hd, td, s.lse, s.entropy, dl)
    few = head.score(hd[:9].contiguous(), td[:9].contiguous(), top_k=8)
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] >= free - (64 << 20)    # torch's own outputs
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s2 = head.score(hd, td, top_k=8)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(s, s2))
    out = head.score_buffers(300, 8)
    grads = (torch.empty_like(hd), torch.empty_like(head.W))
    few_out = head.score_buffers(9, 8)
    h9, t9 = hd[:9].contiguous(), td[:9].contiguous()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        head.score(hd, td, top_k=8, out=out)
        head.score_backward(hd, td, out.lse, out.entropy, dl, out=grads)
        head.score(h9, t9, top_k=8, out=few_out)
    for _ in range(2):
        for x in (*out, *grads, *few_out):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(s, out))
        assert all(torch.equal(a, b) for a, b in zip(few, few_out))
        assert torch.equal(grads[0], dh) and torch.equal(grads[1], dW)
    assert head.check() == 0


def test_a_wait_that_runs_out_is_reported():
    torch = _torch()
    from invariant_output_head_gb300 import (DETLM_DEBUG_STALL, DETLM_ETIMEOUT, Head,
                                             detlm_head_debug)
    W, h, t = ref.grid_inputs(6, 2000, 128, 300)
    head = _head(W, "bf16")
    hd, td = ref.to_dev(h, "bf16"), torch.from_numpy(t).cuda()
    dl = torch.ones(300, device="cuda")
    want = head.score(hd, td, top_k=4)
    grad = head.score_backward(hd, td, want.lse, want.entropy, dl)
    torch.cuda.synchronize()
    q = torch.randint(-127, 128, (300, 128), dtype=torch.int8, device="cuda")
    W8 = torch.randint(-127, 128, (2000, 128), dtype=torch.int8, device="cuda")
    h8 = Head(W8)
    sx, sw = torch.ones(300, device="cuda"), torch.ones(2000, device="cuda")
    y = h8.scaled_logits(q, sx, sw)
    for hh, call in ((head, lambda: head.score(hd, td, top_k=4)),
                     (head, lambda: head.score(hd[:5].contiguous(), td[:5].contiguous(), top_k=4)),
                     (head, lambda: head.score_backward(hd, td, want.lse, want.entropy, dl)),
                     (h8, lambda: h8.scaled_logits(q, sx, sw)),
                     # (calls of up to 8 rows have no wait that could run out)
                     (h8, lambda: h8.scaled_logits(q[:40].contiguous(), sx[:40].contiguous(), sw))):
        detlm_head_debug(hh.handle, DETLM_DEBUG_STALL, 20_000_000)
        call()
        assert hh.check() == DETLM_ETIMEOUT
        detlm_head_debug(hh.handle, 0, 0)
    again = head.score(hd, td, top_k=4)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    back = head.score_backward(hd, td, want.lse, want.entropy, dl)
    assert torch.equal(back[0], grad[0]) and torch.equal(back[1], grad[1])
    assert torch.equal(h8.scaled_logits(q, sx, sw), y)
    assert head.check() == 0 and h8.check() == 0


def test_weights_changed():
    torch = _torch()
    from invariant_output_head_gb300 import Head
    W8 = torch.randint(-127, 128, (600, 64), dtype=torch.int8, device="cuda")
    q = torch.randint(-127, 128, (300, 64), dtype=torch.int8, device="cuda")
    sx, sw = torch.ones(300, device="cuda"), torch.ones(600, device="cuda")
    head = Head(W8)
    head.scaled_logits(q, sx, sw)
    W8.neg_()
    head.weights_changed()
    want = (q.float() @ W8.float().t())
    assert torch.equal(head.scaled_logits(q, sx, sw), want)
    assert torch.equal(head.scaled_logits(q[:4].contiguous(), sx[:4].contiguous(), sw), want[:4])
    # a 16-bit head whose rows are padded (d % 16 == 8)
    W, h, t = ref.grid_inputs(41, 900, 24, 200)
    Wd, hd, td = ref.to_dev(W, "bf16"), ref.to_dev(h, "bf16"), torch.from_numpy(t).cuda()
    head = Head(Wd)
    for B in (5, 200):
        head.score(hd[:B].contiguous(), td[:B].contiguous(), top_k=3)
    Wd.neg_()
    head.weights_changed()
    for B in (5, 200):
        got = head.score(hd[:B].contiguous(), td[:B].contiguous(), top_k=3)
        _check_score(got, ref.score(-W, h[:B], t[:B], 3, 1.0), 3, 1.0)


def test_differentiable_score():
    """The autograd function against the call it is made of, and the example
    that runs the operators together."""
    torch = _torch()
    from invariant_output_head_gb300 import Head
    from invariant_output_head_gb300.training import scored_logprobs
    W, h, t = ref.grid_inputs(12, 800, 72, 60, masked=0.1)
    Wd = ref.to_dev(W, "bf16").requires_grad_()
    hd = ref.to_dev(h, "bf16").requires_grad_()
    td = torch.from_numpy(t).cuda()
    head = Head(Wd)
    logp, entropy = scored_logprobs(head, hd, td, 0.9)
    a, b = torch.randn(60, device="cuda"), torch.randn(60, device="cuda")
    ((a * logp).sum() + (b * entropy).sum()).backward()
    s = head.score(hd.detach(), td, temperature=0.9)
    assert torch.equal(s.logp, logp.detach()) and torch.equal(s.entropy, entropy.detach())
    dh, dW = head.score_backward(hd.detach(), td, s.lse, s.entropy, a, b, temperature=0.9)
    assert torch.equal(hd.grad, dh) and torch.equal(Wd.grad, dW)
    hd.grad = None
    logp, _ = scored_logprobs(head, hd, td)                  # only logp, only h
    (dh_only,) = torch.autograd.grad(logp.sum(), hd)
    s = head.score(hd.detach(), td)
    dh, _ = head.score_backward(hd.detach(), td, s.lse, s.entropy, torch.ones(60, device="cuda"),
                                torch.zeros(60, device="cuda"), need_dW=False)
    assert torch.equal(dh_only, dh)
    from examples.policy_step import main
    band, values = main(rows=200, vocab=3000, dim=256, say=lambda *_: None)
    assert band <= 0.2 and values[1] > values[0]
