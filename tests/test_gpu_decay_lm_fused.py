"""The example model with the gated recurrence, the loss without logits and one call for all parameters: that it runs, its
gradients, and that its token by token form follows the packed one."""
import os
import sys

import pytest

from gpu_util import have_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("mixer", ["attention", "gated"])
@pytest.mark.parametrize("moments", [32, 8])
def test_fused_training_runs(dt, mixer, moments):
    import torch
    import decay_lm
    model = decay_lm.DecayLM(vocab=64, width=128, heads=4, layers=2, dtype=torch.float32 if dt == "f32" else torch.bfloat16, mixer=mixer)
    before = {n: p.detach().clone() for n, p in model.p.items()}
    losses = decay_lm.train(model, 6, docs=12, lr=3e-3, fused=True, moments=moments)
    assert all(0 < v < 20 for v in losses), losses
    for name, p in model.p.items():
        assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.abs().max() > 0, name
        assert torch.isfinite(p).all() and not torch.equal(p.detach(), before[name]), name


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_tokens_one_by_one_follow_the_packed_pass(dt):
    import torch
    import decay_lm
    model = decay_lm.DecayLM(vocab=64, width=128, layers=2, dtype=torch.float32 if dt == "f32" else torch.bfloat16, mixer="gated")
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
    scale = float(whole.abs().max())
    for t in range(min(b - h for h, b in zip(half, ends[1:]))):
        now = torch.stack([ids[h + t] for h in half])
        got = model.step(now, pool, slots=slots)
        want = torch.stack([whole[h + t] for h in half])
        # float32: rounding of the two orders of summation over two layers; bfloat16: a few of its roundings (2^-8) per layer
        assert float((got - want).abs().max()) <= (2e-4 if dt == "f32" else 0.06) * scale, t


@pytest.mark.parametrize("mixer", ["attention", "gated"])
def test_gradients_of_the_fused_loss_against_differences(mixer):
    """The loss's change along one random direction of all parameters, central difference in float32: truncation
    estimated from the difference at twice the step, rounding from the losses' own last bits."""
    import torch
    import decay_lm
    model = decay_lm.DecayLM(vocab=32, width=64, heads=2, layers=1, dtype=torch.float32, mixer=mixer)
    ids, offsets = decay_lm.documents(6, 32, torch.Generator().manual_seed(3))
    g = torch.Generator().manual_seed(4)
    target = torch.roll(ids, -1)
    target[::5] = -1
    weight = torch.randn(ids.shape[0], generator=g).cuda().double()

    def loss():
        return (model.losses(ids, offsets, target).double() * weight).sum()

    loss().backward()
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
        # a loss is a difference of an lse and a logit: of about its size and the largest logit's
        size = float(((model.losses(ids, offsets, target).double() + model.forward(ids, offsets).abs().max()) * weight).square().sum().sqrt())
    assert abs(one - want) <= abs(two - one) + 2e-6 * size / h, (one, two, want)


def test_the_fused_loss_is_the_losses():
    """The same model's losses and gradients, with the logits in memory and without: in float32 a logit is off by
    at most 64 roundings (4 10^-6) of its terms' magnitudes on either side, a gradient by those of every layer's products."""
    import torch
    import decay_lm
    model = decay_lm.DecayLM(vocab=32, width=64, heads=2, layers=1, dtype=torch.float32, mixer="gated")
    ids, offsets = decay_lm.documents(6, 32, torch.Generator().manual_seed(3))
    target = torch.roll(ids, -1)
    target[::5] = -1
    fused = model.losses(ids, offsets, target)
    got = torch.autograd.grad(fused.sum(), list(model.p.values()))
    logits = model.forward(ids, offsets)
    plain = torch.nn.functional.cross_entropy(logits, target, ignore_index=-1, reduction="none")
    want = torch.autograd.grad(plain.sum(), list(model.p.values()))
    assert float((fused - plain).detach().abs().max()) <= 1e-5 * float(logits.detach().abs().max())
    for name, a, b in zip(model.p, got, want):
        assert float((a - b).abs().max()) <= 1e-4 * float(b.abs().max()) + 1e-7, name


def test_second_derivatives_of_the_new_ones_are_refused():
    import torch
    import decay_lm
    model = decay_lm.DecayLM(vocab=32, width=64, heads=2, layers=1, dtype=torch.float32, mixer="gated")
    ids, offsets = decay_lm.documents(3, 32, torch.Generator().manual_seed(3))
    target = torch.roll(ids, -1)
    first = torch.autograd.grad(model.losses(ids, offsets, target).sum(), model.p["0.gx"], create_graph=True)[0]
    with pytest.raises(RuntimeError):
        first.sum().backward()
