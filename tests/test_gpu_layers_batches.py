"""Batches of one token a sequence that are slices of longer ones."""
import pytest

from gpu_util import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


@pytest.mark.parametrize("at", [0, 4, 9])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_one_token_of_each_sequence(at, dt):
    import torch
    import laplace_prefix_scans_amd as lp
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(at)
    q, k, v, go = (torch.randn(3, 10, h, d, generator=g).to(dtype).cuda()[:, at:at + 1] for h, d in ((4, 16), (2, 16), (2, 24), (4, 24)))
    rate = torch.tensor([0.1, 0.5, 0.0, 2.0]).cuda()
    s0, gs = (torch.randn(3, 4, 16, 24, generator=g).cuda() for _ in range(2))
    assert not q.is_contiguous()
    c = [t.contiguous() for t in (q, k, v, go)]
    assert torch.equal(lp.laplex_decay_attn(q, k, v, rate, state_in=s0), lp.laplex_decay_attn(c[0], c[1], c[2], rate, state_in=s0))
    a = lp.laplex_decay_attn_backward(q, k, v, rate, c[3], state_in=s0, dstate_out=gs)
    b = lp.laplex_decay_attn_backward(c[0], c[1], c[2], rate, c[3], state_in=s0, dstate_out=gs)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
