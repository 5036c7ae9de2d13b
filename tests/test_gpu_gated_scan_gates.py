"""The gated linear recurrence at gates that are easy to get wrong: rates of minus zero and of zero, gates that are NaN, and
decays far from 1, whose exponentials have to keep their bits."""
import numpy as np
import pytest

import train_ref as ref
from gpu_util import have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


def dtype_of(name):
    import torch
    return torch.float32 if name == "f32" else torch.bfloat16


def inputs(lengths, channels, dtype, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    n, tokens = len(lengths), sum(lengths)
    normal = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x = {"x": normal(tokens, channels).to(dtype), "dh": normal(tokens, channels).to(dtype), "state_in": normal(n, channels),
         "dstate_out": normal(n, channels), "gate": (torch.exp(normal(tokens, channels) - 3)).to(dtype)}
    x["where"] = torch.rand(tokens, channels, generator=g)
    x["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)
    return {k: v.cuda() for k, v in x.items()}


def both(x, kind, gate=None):
    """Everything that the forward and the backward return."""
    import torch
    import laplace_prefix_scans_amd as lp
    gate = x["gate"] if gate is None else gate
    out = torch.empty_like(x["state_in"])
    h, carries = lp.laplex_gated_scan(gate, x["x"], kind, offsets=x["offsets"], state_in=x["state_in"], state_out=out, keep=True)
    dgate, dx, dstate = lp.laplex_gated_scan_backward(gate, x["x"], carries, x["dh"], kind, offsets=x["offsets"], state_in=x["state_in"],
                                                      dstate_out=x["dstate_out"])
    return {"h": h, "state_out": out, "carries": carries, "dgate": dgate, "dx": dx, "dstate_in": dstate}


# one token, a last tile, whole tiles with boundaries inside and at their ends, tiles without any, several segments
LENGTHS = [[1], [5], [16], [48], [7, 1, 0, 30], [16, 32], [400], [100, 0, 700, 1, 333], [3000]]


@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda v: "-".join(map(str, v)))
@pytest.mark.parametrize("part", [1.0, 0.3])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_a_rate_of_minus_zero_is_a_rate_of_zero(dt, part, lengths):
    """-0.0 is not below zero: the decay is 1, as for 0.0, bit for bit; and both are what the definition gives."""
    import torch
    x = inputs(lengths, 70, dtype_of(dt), len(lengths) + lengths[0])
    some = x["where"] < part
    plus, minus = torch.where(some, 0.0, x["gate"]).to(x["gate"].dtype), torch.where(some, -0.0, x["gate"]).to(x["gate"].dtype)
    assert torch.signbit(minus[some]).all() and not torch.signbit(plus).any()
    want, got = both(x, "rate", plus), both(x, "rate", minus)
    npf = lambda t: t.float().cpu().numpy()  # noqa: E731
    exact = ref.scan(npf(plus), npf(x["x"]), "rate", x["offsets"].tolist(), npf(x["state_in"]), npf(x["dh"]), npf(x["dstate_out"]))
    for name in want:
        assert torch.equal(got[name], want[name]), name
        if name == "carries":
            continue
        half = 2.0 ** -8 if dt == "bf16" and name in ("h", "dgate", "dx") else 2.0 ** -24
        e = exact[name]
        assert (np.abs(host(got[name].float()) - e) <= exact["~" + name] + np.abs(e) * half + 1e-37).all(), name


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_steps_with_rates_of_minus_zero_follow_the_whole_pass(dt):
    import torch
    import laplace_prefix_scans_amd as lp
    x = inputs([40], 70, dtype_of(dt), 1)
    gate = torch.where(x["where"] < 0.5, -0.0, x["gate"]).to(x["gate"].dtype)
    state = x["state_in"].clone()
    h = lp.laplex_gated_scan(gate, x["x"], "rate", state_in=x["state_in"])
    steps = torch.cat([lp.laplex_gated_scan_step(gate[t:t + 1], x["x"][t:t + 1], state, "rate") for t in range(40)])
    assert torch.equal(h, steps)  # one segment of tokens: the same operations in the same order


@pytest.mark.parametrize("kind", ["rate", "sigmoid"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gates_that_are_nan_stay_in_their_sequence_and_channel(kind, dt):
    """A NaN gate takes its token and, forward, those behind it; backward those before it; nothing else."""
    import torch
    lengths = [100, 1, 300, 0, 500]
    bounds = np.concatenate([[0], np.cumsum(lengths)])
    x = inputs(lengths, 70, dtype_of(dt), 8)
    clean = both(x, kind)
    bad = [(0, 3), (150, 3), (99, 10), (100, 11), (101, 12), (400, 0), (401, 1), (450, 20), (900, 69), (640, 33)]
    gate = x["gate"].clone()
    after, before, there, last = (torch.zeros(901, 70, dtype=torch.bool, device="cuda") for _ in range(4))
    ends = torch.zeros(5, 70, dtype=torch.bool, device="cuda")
    for t, ch in bad:
        gate[t, ch] = float("nan")
        s = int(np.searchsorted(bounds, t, side="right")) - 1
        after[t:bounds[s + 1], ch] = True
        before[bounds[s]:t, ch] = True
        there[t, ch] = True
        ends[s, ch] = True
    got = both(x, kind, gate)
    # the weight of an input of the kind "sigmoid" is the gate's too
    for name, hit in (("h", after), ("state_out", ends), ("dx", before | there if kind == "sigmoid" else before), ("dgate", before | after),
                      ("dstate_in", ends)):
        assert torch.isnan(got[name][hit]).all(), name
        assert torch.isfinite(clean[name]).all() and torch.equal(got[name][~hit], clean[name][~hit]), name


@pytest.mark.parametrize("kind", ["rate", "sigmoid"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_decays_and_weights_keep_their_bits_however_small(dt, kind):
    """A step from a state of 1 without an input leaves the decay as the state, one of an input of 1 from zero its weight, in
    float32: the hardware's exponential and reciprocal are off by a step (2 U) each, the factor for what the product with
    log2 e leaves out, the product by it, the sum 1 + e and the last product by U each, and the one sum that a decay near 1 takes
    by U: 9 U of the value, whatever the gate.  In bfloat16 the factor is 1 - 80 ln 2 7.1e-6 at least, in which the square of what is
    taken from 1 is left out: half of (3.9e-4)^2, less than 2 U."""
    import torch
    import laplace_prefix_scans_amd as lp
    g = torch.Generator().manual_seed(5)
    z = torch.cat([torch.linspace(-80, 80, 6401), 3 * torch.randn(4000, generator=g), 30 * torch.randn(4000, generator=g).clamp(-2.5, 2.5)])
    if kind == "rate":
        z = z.abs()
    z = z.to(dtype_of(dt)).cuda()[None]
    most = 9 if dt == "f32" else 11
    one, none = torch.ones_like(z), torch.zeros_like(z)
    e = z.double().cpu().numpy()
    cases = [(none, one, np.exp(-e) if kind == "rate" else 1 / (1 + np.exp(-e)))]
    if kind == "sigmoid":
        cases.append((one, none, 1 / (1 + np.exp(e))))
    for x, before, want in cases:
        state = before.float().clone()
        lp.laplex_gated_scan_step(z, x, state, kind)
        off = np.abs(host(state).astype(np.float64) - want) / want / ref.U
        print("off by %.2f U" % off.max())
        assert off.max() <= most


@pytest.mark.parametrize("kind", ["rate", "sigmoid"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gates_too_large_for_an_exponential(kind, dt):
    """Decays and weights that are too small for a float are zeros, not NaN: gates up to infinity."""
    import torch
    import laplace_prefix_scans_amd as lp
    inf = float("inf")
    z = torch.tensor([200.0, 1e4, 2.5e38, 3.3e38, inf, 104.0, 88.0], device="cuda").to(dtype_of(dt))[None]
    assert torch.isfinite(z[0, 3])
    x, state = torch.full_like(z, 3.0), torch.full(z.shape, 2.0, device="cuda")
    # (e^-88 is next to the smallest normal float: lost beside 2 and 3, as all the others are)
    if kind == "rate":
        cases = [(z, 3.0)]  # the decay is 0
    else:
        cases = [(z, 2.0), (-z, 3.0)]  # the state stays, the weight is 0; the other way round
    for gate, want in cases:
        h = lp.laplex_gated_scan(gate, x, kind, state_in=state)
        assert (h == want).all()
        assert torch.equal(h, lp.laplex_gated_scan_step(gate, x, state.clone(), kind))
