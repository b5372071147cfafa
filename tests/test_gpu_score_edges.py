"""The score call, its gradient and the scaled logits at the ends of their
ranges: workspaces of many rows."""
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
    head = Head(W)
    head.reserve_score(B)
    head.reserve_backward(max_B)
    out = head.score_buffers(B)
    grads = (torch.empty_like(h), torch.empty_like(W))
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    s = head.score(h, t, out=out)
    head.score_backward(h, t, s.lse, s.entropy, dl, out=grads)
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free
    assert head.check() == 0
    head.close()
