"""Thousands of single-token steps against float64 and against one pass over the same tokens.

A step multiplies the state by exp(-rate), adds a token and rounds: n steps add roundings of either sign (each
token's bits shift what the next is), about sqrt(n) 2^-24 of the state's size, taken eightfold for the largest of
many elements.  A decay that is itself off by up to 2^-25 or more, the same way each time, would add up to n 2^-25."""
import numpy as np
import pytest

import layers_ref as ref
from gpu_util import have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

STEPS = 6000


def test_steps_and_a_pass_over_the_same_tokens():
    import torch
    import laplace_prefix_scans_amd as lp
    rates = [0.0, 1e-4, 3e-4, 2e-3]
    heads, dk, dv = len(rates), 24, 20
    g = torch.Generator().manual_seed(2)
    # values of one sign: what a wrong decay does to old tokens does not average out
    q, k, v = (torch.rand(STEPS, heads, d, generator=g) for d in (dk, dk, dv))
    rate = torch.tensor(rates)
    d = [t.cuda() for t in (q, k, v, rate)]
    whole, state = torch.empty(1, heads, dk, dv, device="cuda"), torch.zeros(1, heads, dk, dv, device="cuda")
    o = lp.laplex_decay_attn(*d, state_out=whole)
    last = None
    for t in range(STEPS):
        last = lp.laplex_decay_attn_step(d[0][t:t + 1], d[1][t:t + 1], d[2][t:t + 1], d[3], state)
    want, final = ref.attn_scan(*[t.numpy() for t in (q, k, v, rate)], [0, STEPS], 1.0)
    tol = (8 * np.sqrt(STEPS + dk) + 20) * 2.0 ** -24  # every term is positive: the results are their own magnitudes
    for name, got, exact in (("steps' state", host(state), final), ("pass's state", host(whole), final),
                             ("last step", host(last)[0], want[-1]), ("pass's last token", host(o)[-1], want[-1])):
        assert np.abs(got / exact - 1).max() <= tol, (name, np.abs(got / exact - 1).max(), tol)
