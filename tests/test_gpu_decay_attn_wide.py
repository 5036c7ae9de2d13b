"""Decayed attention on the GPU at the shapes that take blocks of eight waves: 65 to 128 columns of the
output (or 129 and more on at most 128 rows of the carry) and more than 160 blocks, cut into segments or not,
aligned and not; and what reaches over several segments.  References and tolerances as in test_gpu_decay_attn."""
import numpy as np
import pytest

import layers_ref as ref
import test_gpu_decay_attn as base
from gpu_util import have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

# lengths, heads, key/value heads, dk, dv
CASES = [([700, 700], 32, 32, 128, 128), ([700, 0, 699], 32, 8, 100, 127), ([333, 64, 1], 60, 60, 64, 96), ([50, 140], 41, 41, 33, 130),
         ([129, 0, 200], 40, 20, 127, 129), ([90, 31], 90, 30, 65, 70), ([2000], 24, 24, 96, 96)]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_against_pairs(case, dt):
    lengths, heads, kv, dk, dv = case
    base.run_case(lengths, heads, kv, dk, dv, base.dtypes()[dt], True, seed=dk + dv)


@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_many_short_sequences(dt):
    r = np.random.default_rng(12)
    base.run_case([int(x) for x in r.integers(0, 70, 40)], 16, 4, 72, 104, base.dtypes()[dt], True, seed=12, lead=3, tail=2)


@pytest.mark.parametrize("dims", [(128, 128), (100, 66)], ids=str)
@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_one_long_prompt(dims, dt):
    """47 segments of one sequence, forward, with the states that come in and go out."""
    import torch
    import laplace_prefix_scans_amd as lp
    tokens, heads = 6000, 8
    dk, dv = dims
    x = base.make(21, tokens, heads, heads, dk, dv, 1, base.dtypes()[dt], True)
    x["rate"] = torch.tensor([0.0, 1e-4, 0.3, 7.0, 0.02, 2e-3, 1e-3, 0.1])
    d = base.cuda(x)
    state = torch.empty(1, heads, dk, dv, device="cuda")
    o = lp.laplex_decay_attn(d["q"], d["k"], d["v"], d["rate"], scale=0.3, state_in=d["state_in"], state_out=state)
    args = [base.npf(x[n]) for n in ("q", "k", "v", "rate")]
    s0 = base.npf(x["state_in"])
    want, final = ref.attn_scan(*args, [0, tokens], 0.3, s0)
    env, env_final = ref.attn_scan(*[np.abs(a) for a in args], [0, tokens], 0.3, np.abs(s0))
    n = dk + dv + tokens + 64
    base.check("o", host(o.float()), want, env, n, dt == 1)
    base.check("state_out", host(state), final, env_final, n)


@pytest.mark.parametrize("dims", [(128, 128), (100, 66)], ids=str)
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_a_nonfinite_token_segments_before_the_end(dims, which, dt):
    import torch
    import laplace_prefix_scans_amd as lp
    dk, dv = dims
    x = base.cuda(base.make(22, 3200, 16, 16, dk, dv, 2, base.dtypes()[dt], False))
    x["rate"] = torch.full((16,), 1e-3, device="cuda")
    off = torch.tensor([0, 3000, 3200], dtype=torch.int32).cuda()
    want = lp.laplex_decay_attn(x["q"], x["k"], x["v"], x["rate"], offsets=off)
    for j in (0, 127, 1000):
        for value in (float("nan"), float("inf")):
            y = dict(x)
            y[which] = x[which].clone()
            y[which][j, 5, 3] = value
            got = lp.laplex_decay_attn(y["q"], y["k"], y["v"], y["rate"], offsets=off)
            keep = [h for h in range(16) if h != 5]
            assert torch.equal(got[:j], want[:j]) and torch.equal(got[3000:], want[3000:]) and torch.equal(got[:, keep], want[:, keep])
            for t in (j, j + 1, 1900, 2999):
                assert not torch.isfinite(got[t, 5]).all(), t


@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("dims", [(128, 128), (72, 96), (101, 77)], ids=str)
def test_strided_and_unaligned_inputs_give_the_same_bits(dt, dims):
    """q, k, v as slices of one projection, at element offsets that keep or break 16-byte alignment."""
    import torch
    import laplace_prefix_scans_amd as lp
    dk, dv = dims
    heads, tokens = 48, 600
    x = base.cuda(base.make(23, tokens, heads, heads, dk, dv, 1, base.dtypes()[dt], False))
    want = lp.laplex_decay_attn(x["q"], x["k"], x["v"], x["rate"])
    grads = lp.laplex_decay_attn_backward(x["q"], x["k"], x["v"], x["rate"], x["go"])
    for pad in (0, 1, 8):
        width = heads * (2 * dk + dv) + pad
        buf = torch.full((tokens * width + pad,), float("nan"), dtype=x["q"].dtype).cuda()
        rows = buf[pad:].view(tokens, width)
        q, k, v = (r.unflatten(1, (heads, -1)) for r in rows[:, :heads * (2 * dk + dv)].split([heads * dk, heads * dk, heads * dv], 1))
        q.copy_(x["q"]), k.copy_(x["k"]), v.copy_(x["v"])
        assert torch.equal(lp.laplex_decay_attn(q, k, v, x["rate"]), want)
        for a, b in zip(lp.laplex_decay_attn_backward(q, k, v, x["rate"], x["go"])[:4], grads[:4]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("heads", [2, 48])
@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_offsets_that_run_out_of_the_buffer(heads, dt):
    """Offsets below 0 and above the token count are taken as 0 and the count: the same bits as with those."""
    import torch
    import laplace_prefix_scans_amd as lp
    x = base.cuda(base.make(24, 500, heads, heads, 80, 96, 4, base.dtypes()[dt], True))

    def go(*bounds):
        off = torch.tensor(bounds, dtype=torch.int32).cuda()
        state = torch.empty_like(x["state_in"])
        o = lp.laplex_decay_attn(x["q"], x["k"], x["v"], x["rate"], offsets=off, state_in=x["state_in"], state_out=state)
        return (o, state) + lp.laplex_decay_attn_backward(x["q"], x["k"], x["v"], x["rate"], x["go"], offsets=off,
                                                          state_in=x["state_in"], dstate_out=x["dstate_out"])

    for bad, good in (((-7, -3, 200, 450, 600), (0, 0, 200, 450, 500)), ((-2 ** 31, 0, 500, 501, 2 ** 31 - 1), (0, 0, 500, 500, 500))):
        for a, b in zip(go(*bad), go(*good)):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ one token
@pytest.mark.parametrize("dims", [(128, 128), (128, 127)], ids=str)
@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_step_on_states_larger_than_the_caches(dims, dt):
    """314 MB of states, which a step loads and stores past the caches."""
    import torch
    import laplace_prefix_scans_amd as lp
    dk, dv = dims
    n, heads, kv = 300, 16, 4
    x = base.cuda(base.make(25, n, heads, kv, dk, dv, 1, base.dtypes()[dt], False))
    g = torch.Generator(device="cuda").manual_seed(25)
    state = torch.randn(n + 1, heads, dk, dv, device="cuda", generator=g)
    slots = torch.randperm(n + 1, device="cuda", generator=g)[:n].to(torch.int32)
    slots[7] = -1
    old = state.clone()
    o = lp.laplex_decay_attn_step(x["q"], x["k"], x["v"], x["rate"], state, slots=slots, scale=0.5)
    w = torch.from_numpy(ref.weight_per_head(host(x["rate"]), 1)).cuda()[:, None, None]
    untouched = torch.ones(n + 1, dtype=torch.bool)
    for r, s in enumerate(slots.tolist()):
        if s < 0:
            assert not o[r].any()
            continue
        untouched[s] = False
        k, v = (x[m][r].double().repeat_interleave(heads // kv, 0) for m in ("k", "v"))
        q = x["q"][r].double()[:, :, None]
        kv_ = k[:, :, None] * v[:, None, :]
        new, env = w * old[s].double() + kv_, w * old[s].double().abs() + kv_.abs()
        if r % 10 and r < n - 3:  # states all over, outputs of every row
            assert ((state[s].double() - new).abs() <= env * (8 * 2 ** 0.5 + 40) * 2.0 ** -24).all(), r
        want, size = 0.5 * (q * new).sum(1), 0.5 * (q.abs() * env).sum(1)
        tol = size * (8 * dk ** 0.5 + 40) * 2.0 ** -24 + (want.abs() * 2.0 ** -8 if dt == 1 else 0.0) + 1e-30
        assert ((o[r].double() - want).abs() <= tol).all(), r
    assert torch.equal(state[untouched.cuda()], old[untouched.cuda()])
