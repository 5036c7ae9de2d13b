"""The example's autograd functions: a second derivative is refused instead of being silently incomplete, and what no
parameter needs is not formed."""
import os
import sys

import pytest

from gpu_util import have_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


def inputs():
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(40, 2, 16, device="cuda", generator=g).requires_grad_() for _ in range(3))
    rate = torch.tensor([0.1, 0.3], device="cuda").requires_grad_()
    return q, k, v, rate, torch.tensor([0, 15, 40], dtype=torch.int32, device="cuda")


def test_second_derivatives_are_refused():
    import torch
    import decay_lm
    q, k, v, rate, off = inputs()
    x = torch.randn(8, 32, device="cuda").requires_grad_()
    w, b = torch.ones(32, device="cuda").requires_grad_(), torch.zeros(32, device="cuda").requires_grad_()
    table = torch.randn(9, 16, device="cuda").requires_grad_()
    ids = torch.arange(8, device="cuda")
    for y, leaf in ((decay_lm.DecayAttention.apply(q, k, v, rate, off, 1.0), q), (decay_lm.LayerNorm.apply(x, w, b), x),
                    (decay_lm.Embedding.apply(ids, table, 1.0), table)):
        (grad,) = torch.autograd.grad((y * y).sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (grad * leaf).sum().backward()


@pytest.mark.parametrize("learned", [False, True])
def test_the_rates_gradient_is_formed_where_the_rates_are_learned(learned):
    import torch
    import decay_lm
    import laplace_prefix_scans_amd as lp
    q, k, v, rate, off = inputs()
    rate.requires_grad_(learned)
    y = decay_lm.DecayAttention.apply(q, k, v, rate, off, 1.0)
    g = torch.randn_like(y)
    with lp.profile_launches(64) as prof:
        y.backward(g)
        torch.cuda.synchronize()
    names = [r[0] for r in prof.records]
    assert "k_attn_chunk" in names and ("k_attn_drate" in names) == learned
    assert (rate.grad is not None) == learned
    want = lp.laplex_decay_attn_backward(q.detach(), k.detach(), v.detach(), rate.detach(), g, offsets=off, rate_grad=learned)
    for p, x in zip((q, k, v, rate), want):
        assert x is None or torch.equal(p.grad, x)


def test_norm_without_learned_weights():
    import torch
    import decay_lm
    x, w, b = torch.randn(8, 32, device="cuda").requires_grad_(), torch.ones(32, device="cuda"), torch.zeros(32, device="cuda")
    y = decay_lm.LayerNorm.apply(x, w, b)
    (dx,) = torch.autograd.grad(y, x, torch.ones_like(y) * x.detach())
    w2 = w.clone().requires_grad_()
    y2 = decay_lm.LayerNorm.apply(x, w2, b)
    dx2, _ = torch.autograd.grad(y2, (x, w2), torch.ones_like(y) * x.detach())
    assert torch.equal(dx, dx2)
