"""The example model: its loss falls, every parameter gets a gradient, and generation from
the recurrent states gives the logits of the packed forward pass."""
import os
import sys

import pytest

from gpu_util import have_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_example_trains_and_generates(dt):
    import torch
    import decay_lm
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    torch.manual_seed(0)
    model = decay_lm.DecayLM(vocab=64, width=128, heads=4, layers=2, dtype=dtype)
    losses = decay_lm.train(model, 60, docs=24, lr=3e-3)
    assert losses[-1] < 0.75 * losses[0], losses[::10]
    for name, p in model.p.items():
        assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.abs().max() > 0, name
    # the logits of a document token by token from its first half's states, and of the packed pass
    ids, offsets = decay_lm.documents(5, 64, torch.Generator().manual_seed(7))
    with torch.no_grad():
        whole = model.forward(ids, offsets)
    ends = offsets.tolist()
    half = [a + (b - a) // 2 for a, b in zip(ends[:-1], ends[1:])]
    first = torch.cat([ids[a:h] for a, h in zip(ends[:-1], half)])
    cut = torch.tensor([0] + [h - a for a, h in zip(ends[:-1], half)]).cumsum(0).to(torch.int32).cuda()
    _, states = model.prefill(first, cut)
    slots = torch.tensor([3, 0, 4, 1, 2], dtype=torch.int32).cuda()  # the pool's order is not the batch's
    pool = []
    for s in states:
        t = torch.empty_like(s)
        t[slots.long()] = s
        pool.append(t)
    steps = min(b - h for h, b in zip(half, ends[1:]))
    scale = float(whole.abs().max())
    for t in range(steps):
        now = torch.stack([ids[h + t] for h in half])
        got = model.step(now, pool, slots=slots)
        want = torch.stack([whole[h + t] for h in half])
        # float32: rounding of the two orders of summation over two layers; bfloat16: a few of its roundings (2^-8) per layer
        assert float((got - want).abs().max()) <= (2e-4 if dt == "f32" else 0.06) * scale, t


def test_gradients_of_the_whole_model_against_differences():
    """The loss's change along one random direction of all parameters, central difference in float32:
    truncation estimated from the difference at twice the step, rounding from the loss's own last bits."""
    import torch
    import decay_lm
    model = decay_lm.DecayLM(vocab=32, width=64, heads=2, layers=1, dtype=torch.float32)
    ids, offsets = decay_lm.documents(6, 32, torch.Generator().manual_seed(3))
    weight = torch.randn(ids.shape[0], 32, generator=torch.Generator().manual_seed(4)).cuda().double()

    def loss():
        return (model.forward(ids, offsets).double() * weight).sum()

    loss().backward()
    g = torch.Generator().manual_seed(5)
    d = {n: (torch.randn(p.shape, generator=g)).to(p.device) * p.detach().abs().mean() for n, p in model.p.items()}
    want = sum(float((p.grad.double() * d[n].double()).sum()) for n, p in model.p.items())

    def at(h):
        with torch.no_grad():
            for n, p in model.p.items():
                p += h * d[n]
            v = float(loss())
            for n, p in model.p.items():
                p -= h * d[n]
        return v

    h = 2.0 ** -9
    one = (at(h) - at(-h)) / (2 * h)
    two = (at(2 * h) - at(-2 * h)) / (4 * h)
    with torch.no_grad():
        size = float((model.forward(ids, offsets).double() * weight).square().sum().sqrt())
    assert abs(one - want) <= abs(two - one) + 2e-6 * size / h, (one, two, want)
