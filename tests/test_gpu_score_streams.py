"""Outputs of the score call, its gradient, the scaled logits and the greedy
call when they run on a stream that is not the current one."""
import pytest

pytestmark = pytest.mark.gpu


def _calls(side):
    """name -> (the call on the side stream, bytes of its largest output)."""
    import torch
    from invariant_output_head_gb300 import Head
    g = torch.Generator(device="cuda").manual_seed(2)
    W = torch.randn(40000, 256, generator=g, device="cuda").bfloat16()
    h = torch.randn(40000, 256, generator=g, device="cuda").bfloat16()
    t = torch.randint(0, 40000, (40000,), generator=g, device="cuda", dtype=torch.int32)
    dl = torch.randn(40000, generator=g, device="cuda")
    few = [x[:40].contiguous() for x in (h, t, dl)]
    head, head8 = Head(W), Head((W * 20).round().clamp(-127, 127).to(torch.int8))
    q = (h[:40] * 20).round().clamp(-127, 127).to(torch.int8)
    sx, sw = torch.rand(40, device="cuda"), torch.rand(40000, device="cuda")
    s = head.score(few[0], few[1])
    head.reserve_score(40000, 32)
    head.reserve_backward(40)
    torch.cuda.synchronize()
    return {
        "score": (lambda: head.score(h, t, top_k=32, stream=side), 40000 * 32 * 4),
        "gradient": (lambda: head.score_backward(few[0], few[1], s.lse, s.entropy, few[2],
                                                 stream=side), 40000 * 256 * 2),
        "scaled": (lambda: head8.scaled_logits(q, sx, sw, stream=side), 40 * 40000 * 4),
        "greedy": (lambda: head.greedy(few[0], with_logits=True, stream=side), 40 * 40000 * 4),
    }


@pytest.mark.parametrize("name", ["score", "gradient", "scaled", "greedy"])
def test_outputs_do_not_take_memory_that_the_current_stream_still_uses(name):
    """A tensor of the size of the call's output is read by work that waits on
    the current stream, and freed: its memory is free for that stream's later
    work only, not for a call on another stream, which runs before."""
    import torch
    side = torch.cuda.Stream()
    call, size = _calls(side)[name]
    call()                                      # (what the first call loads is loaded)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    xs = [torch.full((size,), 5, dtype=torch.uint8, device="cuda") for _ in range(4)]
    ys = [torch.empty_like(x) for x in xs]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)              # some 50 ms
    for x, y in zip(xs, ys):
        y.copy_(x)
    del x, xs
    out = call()                                # does not wait for the copies
    side.synchronize()
    torch.cuda.synchronize()
    assert all(bool((y == 5).all()) for y in ys)
    del out
