"""Decayed attention on integers: every sum is exact in float32, so every result is known to the last bit.

With a rate of 0 and a scale of 1 all weights are 1.  Where the magnitudes of an output's terms add up to less
than 2^24, each partial sum of them is an integer that float32 holds, whatever the order; a result of the
library is then the exact one, rounded once to its type.  The operands are chosen so that the factors formed
on the way (pair products, carries, lag-weighted pairs) need more than the 17 bits of two bfloat16 values."""
import numpy as np
import pytest

import layers_ref as ref
from gpu_util import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

# (heads, key/value heads, dk, dv); 32 heads and more of 65 to 128 columns are many blocks
HEADS = [(2, 2, 64, 64), (2, 1, 40, 24), (3, 3, 33, 17), (32, 32, 128, 128), (64, 64, 64, 128), (40, 20, 100, 96), (48, 48, 127, 121),
         (2, 2, 256, 256), (4, 2, 129, 200)]
LENGTHS = [150, 0, 131, 1]


def integers(g, top, shape, keep=1.0):
    """Integers of magnitude up to top; all but a share `keep` of them zero."""
    import torch
    x = torch.randint(-top, top + 1, shape, generator=g).float()
    return x if keep >= 1.0 else x * (torch.rand(shape, generator=g) < keep)


def inputs(kind, heads, dtype):
    import torch
    h, kv, dk, dv = heads
    t = sum(LENGTHS)
    g = torch.Generator().manual_seed(dk * dv + h)

    def tokens(keep):  # whole tokens are kept or not, signs and zeros otherwise
        return lambda n, d: torch.randint(-1, 2, (t, n, d), generator=g).float() * (torch.rand(t, n, 1, generator=g) < keep)

    wide = int(200 * min(1.0, (64 / max(dk, dv)) ** 0.5))
    if kind == "pairs":  # q.k and go.v of up to 20 bits, met by few tokens
        q, k = integers(g, wide, (t, h, dk)), integers(g, wide, (t, kv, dk))
        v, go = tokens(1 / 24)(kv, dv), tokens(1 / 24)(h, dv)
    elif kind == "carry":  # k v^T and q go^T add up to 20 bits, read by few channels
        q, go = integers(g, 1, (t, h, dk), 2 / dk), integers(g, 1, (t, h, dv), 2 / dv)
        k, v = integers(g, 180, (t, kv, dk)), integers(g, 180, (t, kv, dv))
    else:  # go.v times the lag
        go, v = integers(g, 24, (t, h, dv), min(1.0, 64 / dv)), integers(g, 24, (t, kv, dv))
        q, k = tokens(1 / 24)(h, dk), tokens(1 / 24)(kv, dk)
    x = {"q": q, "k": k, "v": v, "go": go}
    return {n: y.to(dtype) for n, y in x.items()}


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("kind", ["pairs", "carry", "lags"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_integers_are_exact(heads, kind, dt):
    import torch
    import laplace_prefix_scans_amd as lp
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    print("attention of integers", heads, kind, dt, flush=True)
    h, kv, dk, dv = heads
    x = inputs(kind, heads, dtype)
    bounds = [0] + [int(c) for c in np.cumsum(LENGTHS)]
    rate = torch.zeros(h)
    f = {n: y.float().numpy() for n, y in x.items()}
    args = (f["q"], f["k"], f["v"], rate.numpy(), f["go"], bounds, 1.0)
    want, env = ref.attn_pairs(*args), ref.attn_pairs(*args, absolute=True)
    d = {n: y.cuda() for n, y in x.items()}
    off = torch.tensor(bounds, dtype=torch.int32).cuda()
    state = torch.empty(len(LENGTHS), h, dk, dv, device="cuda")
    got = {"o": lp.laplex_decay_attn(d["q"], d["k"], d["v"], rate.cuda(), offsets=off, state_out=state), "state_out": state}
    grads = lp.laplex_decay_attn_backward(d["q"], d["k"], d["v"], rate.cuda(), d["go"], offsets=off)
    got.update(zip(("dq", "dk", "dv", "drate"), grads))
    checked = []
    for name, y in got.items():
        # the rate's gradient adds, in doubles, float32 products of q and of lag-weighted sums as large as the ones below
        size = env[name].max() if name != "drate" else (lag_sums(f, bounds, h // kv) * np.maximum(np.abs(f["q"]), 1)).max()
        if size >= 2.0 ** 24:
            continue
        checked.append(name)
        exact = torch.from_numpy(want[name]).to(torch.float32).to(y.dtype)
        bad = y.cpu() != exact
        assert not bad.any(), "%s: %d of %d are not the exact value rounded once" % (name, int(bad.sum()), bad.numel())
    assert {"pairs": {"o", "dv"}, "carry": {"o", "state_out"}, "lags": {"dq", "drate"}}[kind] <= set(checked), checked


def lag_sums(f, bounds, group):
    """The magnitudes of sum_j (i - j) (go_i . v_j) k_j, added up."""
    go, v, k = np.abs(f["go"]), np.repeat(np.abs(f["v"]), group, 1), np.repeat(np.abs(f["k"]), group, 1)
    out = np.zeros(f["q"].shape)
    for a, b in zip(bounds[:-1], bounds[1:]):
        i = np.arange(b - a)
        lag = np.maximum(i[:, None] - i[None, :], 0)
        for h in range(out.shape[1]):
            out[a:b, h] = (lag * (go[a:b, h] @ v[a:b, h].T)) @ k[a:b, h]
    return out


@pytest.mark.parametrize("heads", [(2, 2, 64, 64), (32, 8, 128, 128), (40, 40, 100, 96), (2, 1, 256, 130)], ids=str)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_outputs_do_not_depend_on_what_else_is_asked_for(heads, dt):
    """o with and without the final states, and the gradients with and without the rate's and the initial state's, have the same bits
    (where the segments are the same: the rate's gradient takes others)."""
    import torch
    import laplace_prefix_scans_amd as lp
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    h, kv, dk, dv = heads
    g = torch.Generator().manual_seed(3)
    off = torch.tensor([0, 700, 701, 1500], dtype=torch.int32).cuda()

    def normal(*shape):
        return torch.randn(shape, generator=g).to(dtype).cuda()

    q, k, v, go = normal(1500, h, dk), normal(1500, kv, dk), normal(1500, kv, dv), normal(1500, h, dv)
    rate = torch.linspace(0.0, 0.2, h).cuda()
    zero = torch.zeros(3, h, dk, dv, device="cuda")
    state = torch.empty_like(zero)
    alone = lp.laplex_decay_attn(q, k, v, rate, offsets=off)
    assert torch.equal(alone, lp.laplex_decay_attn(q, k, v, rate, offsets=off, state_out=state))
    assert torch.equal(alone, lp.laplex_decay_attn(q, k, v, rate, offsets=off, state_in=zero))
    plain = lp.laplex_decay_attn_backward(q, k, v, rate, go, offsets=off, rate_grad=False)
    with_state = lp.laplex_decay_attn_backward(q, k, v, rate, go, offsets=off, rate_grad=False, state_in=zero)
    with_rate = lp.laplex_decay_attn_backward(q, k, v, rate, go, offsets=off, state_in=zero)
    for a, b, c in zip(plain[:3], with_state[:3], with_rate[:3]):
        assert torch.equal(a, b)
        if a.shape != q.shape or a is not plain[0]:
            assert torch.equal(a, c)
