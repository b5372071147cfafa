"""Heads that keep a copy of W (padded rows of a 16-bit head with d % 16 == 8,
fp16 values for an int8 head's wide calls) after W was changed in place: on
another stream, around CUDA graphs, and with reserved workspaces."""
import pytest

pytestmark = pytest.mark.gpu


class _Scored:
    """A 16-bit head with padded rows; its calls are the score and gradient."""

    def __init__(self, B):
        import torch
        from invariant_output_head_gb300 import Head
        g = torch.Generator(device="cuda").manual_seed(5 + B)
        self.B = B
        self.W = (torch.randn(900, 24, generator=g, device="cuda") * 0.3).bfloat16()
        self.h = torch.randn(B, 24, generator=g, device="cuda").bfloat16()
        self.t = torch.randint(0, 900, (B,), generator=g, device="cuda", dtype=torch.int32)
        self.dl = torch.randn(B, generator=g, device="cuda")
        self.head = Head(self.W)
        self.out = self.head.score_buffers(B, 3)
        self.grads = (torch.empty_like(self.h), torch.empty_like(self.W))

    def reserve(self):
        self.head.reserve_score(self.B, 3)
        self.head.reserve_backward(self.B)

    def run(self):
        s = self.head.score(self.h, self.t, top_k=3, out=self.out)
        self.head.score_backward(self.h, self.t, s.lse, s.entropy, self.dl, out=self.grads)
        return [*self.out, *self.grads]


class _Scaled:
    """An int8 head; its calls are scaled logits and the greedy decision."""

    def __init__(self, B):
        import torch
        from invariant_output_head_gb300 import Head
        g = torch.Generator(device="cuda").manual_seed(7 + B)
        self.B = B
        self.W = torch.randint(-127, 128, (600, 64), generator=g, device="cuda").to(torch.int8)
        self.q = torch.randint(-127, 128, (B, 64), generator=g, device="cuda").to(torch.int8)
        self.sx = torch.rand(B, generator=g, device="cuda")
        self.sw = torch.rand(600, generator=g, device="cuda")
        self.head = Head(self.W)
        self.out = torch.empty(B, 600, device="cuda")
        self.best = (torch.empty(B, dtype=torch.int32, device="cuda"),
                     torch.empty(B, dtype=torch.int32, device="cuda"), None)

    def reserve(self):
        self.head.reserve(self.B)

    def run(self):
        self.head.scaled_logits(self.q, self.sx, self.sw, out=self.out)
        self.head.greedy(self.q, out=self.best)
        return [self.out, *self.best[:2]]


# rows for every path that reads the copies
_CASES = [(_Scored, 5), (_Scored, 200), (_Scaled, 100), (_Scaled, 300)]


def _check(c, got):
    """`got` against the same calls on a head that has seen no other W."""
    import torch
    fresh = type(c)(c.B)
    fresh.W.copy_(c.W)
    torch.cuda.synchronize()
    want = fresh.run()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert c.head.check() == 0 and fresh.head.check() == 0


@pytest.mark.parametrize("kind,B", _CASES)
def test_capture_after_a_change_does_not_stand_in_for_a_call(kind, B):
    """W changed, a call captured but not replayed: the next eager call still
    uses the new W, and so do the replays afterwards."""
    import torch
    c = kind(B)
    c.run()
    c.W.neg_()
    c.head.weights_changed()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    _check(c, c.run())
    for x in (*c.out, *c.grads) if kind is _Scored else (c.out, *c.best[:2]):
        x.zero_()
    graph.replay()
    _check(c, [*c.out, *c.grads] if kind is _Scored else [c.out, *c.best[:2]])


@pytest.mark.parametrize("kind,B", _CASES)
def test_replays_use_the_changed_weights(kind, B):
    """A graph captured before a change of W, replayed after it."""
    import torch
    c = kind(B)
    got = c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for _ in range(2):
        c.W.neg_()
        c.W[::3] = 1
        c.head.weights_changed()
        graph.replay()
        _check(c, got)


@pytest.mark.parametrize("kind,B", _CASES)
def test_a_change_captured_with_the_calls(kind, B):
    """The update, its announcement and the calls in one graph."""
    import torch
    c = kind(B)
    got = c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.W.neg_()
        c.head.weights_changed()
        c.run()
    _check(c, c.run())                     # nothing has run: W is the old one
    graph.replay()
    _check(c, got)
    graph.replay()
    _check(c, got)
    _check(c, c.run())


@pytest.mark.parametrize("kind,B", _CASES)
def test_first_call_captured(kind, B):
    """Reserved, then captured before any eager call."""
    import torch
    c = kind(B)
    c.reserve()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.run()
    c.W.neg_()
    c.head.weights_changed()
    _check(c, c.run())
    graph.replay()
    _check(c, got)


@pytest.mark.parametrize("kind,B", _CASES)
@pytest.mark.parametrize("seen", [False, True])
def test_reserve_after_a_change_on_another_stream(kind, B, seen):
    """W is still being written on a side stream when a workspace is reserved
    (with `seen`: after the head's first calls, and announced)."""
    import torch
    c = kind(B)
    if seen:
        c.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)      # some 20 ms ahead of the write
        c.W.neg_()
        if seen:
            c.head.weights_changed()
    c.reserve()
    side.synchronize()
    _check(c, c.run())


@pytest.mark.parametrize("kind,B", [(_Scaled, 65), (_Scaled, 100), (_Scaled, 255), (_Scaled, 300),
                                    (_Scored, 5), (_Scored, 200)])
def test_reserved_calls_allocate_nothing(kind, B):
    """After a reserve the first calls leave the free memory as it is and can
    be captured, for every number of rows up to the reserved one."""
    import torch
    kind(B).run()                          # (kernels are loaded by their first launch)
    c = kind(B)
    c.reserve()
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    got = c.run()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free
    d = kind(B)
    d.reserve()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.run()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, [*d.out, *d.grads] if kind is _Scored else [d.out, *d.best[:2]]):
        assert torch.equal(a, b)
    assert c.head.check() == 0 and d.head.check() == 0
