"""Decayed linear attention on the GPU against float64 sums over pairs.

Tolerances.  An output is a sum of n = (channels + tokens + chunk joins) float32
terms whose magnitudes add up to `env` (the same sum of absolute values): its
rounding error behaves like sqrt(n) 2^-24 env, with a factor of 8 for the
largest of many elements, and the weights exp(-rate n) add 20 ulp (the
exponent's rounding, for arguments up to about 20).  bfloat16 results add their own
rounding, 2^-9 of the value (2^-8 allowed), and 3 * 2^-17 env where a float32
factor enters a product as a sum of two bfloat16 values."""
import numpy as np
import pytest

import layers_ref as ref
from gpu_util import have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

RATES = [0.0, 1e-4, 0.3, 7.0, float("inf"), 0.02, 1.0, 1e-3]


def bound(env, value, n, bf16):
    t = env * (8 * np.sqrt(n) * 2.0 ** -24 + 20 * 2.0 ** -23) + 1e-30
    return t + (np.abs(value) * 2.0 ** -8 + env * 3 * 2.0 ** -17 if bf16 else 0.0)


def check(name, got, want, env, n, bf16=False):
    assert got.shape == want.shape, name
    assert np.isfinite(got).all(), "%s: non-finite" % name
    bad = np.abs(got - want) > bound(env, want, n, bf16)
    assert not bad.any(), "%s: %d of %d off, worst %.3e of env, first at %s" % (
        name, bad.sum(), bad.size, (np.abs(got - want) / np.maximum(env, 1e-30)).max(), np.argwhere(bad)[:3].tolist())


def make(seed, tokens, heads, kv, dk, dv, seqs, dtype, states):
    import torch
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, dt):
        return torch.randn(shape, generator=g).to(dt)

    x = {"q": normal(tokens, heads, dk, dt=dtype), "k": normal(tokens, kv, dk, dt=dtype), "v": normal(tokens, kv, dv, dt=dtype),
         "go": normal(tokens, heads, dv, dt=dtype), "rate": torch.tensor([RATES[(i + seed) % len(RATES)] for i in range(heads)])}
    x["state_in"] = normal(seqs, heads, dk, dv, dt=torch.float32) if states else None
    x["dstate_out"] = normal(seqs, heads, dk, dv, dt=torch.float32) if states else None
    return x


def cuda(x):
    return {k: None if v is None else v.cuda() for k, v in x.items()}


def npf(t):
    return None if t is None else t.float().numpy()


def run_case(lengths, heads, kv, dk, dv, dtype, states, seed=0, lead=0, tail=0, use_offsets=True):
    """Forward and backward against the references; lead/tail: tokens outside every sequence."""
    import torch
    import laplace_prefix_scans_amd as lp
    bf16 = dtype == torch.bfloat16
    bounds = [lead + int(c) for c in np.concatenate([[0], np.cumsum(lengths)])]
    tokens = bounds[-1] + tail
    x = make(seed, tokens, heads, kv, dk, dv, len(lengths), dtype, states)
    d = cuda(x)
    scale = 0.37
    off = torch.tensor(bounds, dtype=torch.int32).cuda() if use_offsets else None
    print("attn lengths=%s heads=%d/%d dk=%d dv=%d %s states=%s" % (lengths[:8], heads, kv, dk, dv, dtype, states), flush=True)
    state_out = torch.full((len(lengths), heads, dk, dv), float("nan")).cuda() if states else None
    o = lp.laplex_decay_attn(d["q"], d["k"], d["v"], d["rate"], offsets=off, scale=scale, state_in=d["state_in"],
                             state_out=state_out)
    dq, dk_, dv_, drate, dsi = lp.laplex_decay_attn_backward(d["q"], d["k"], d["v"], d["rate"], d["go"], offsets=off, scale=scale,
                                                             state_in=d["state_in"], dstate_out=d["dstate_out"])
    args = [npf(x[n]) for n in ("q", "k", "v", "rate", "go")] + [bounds, scale, npf(x["state_in"]), npf(x["dstate_out"])]
    want, env = ref.attn_pairs(*args), ref.attn_pairs(*args, absolute=True)
    scanned, final = ref.attn_scan(npf(x["q"]), npf(x["k"]), npf(x["v"]), npf(x["rate"]), bounds, scale, npf(x["state_in"]))
    assert np.allclose(scanned, want["o"], rtol=1e-9, atol=1e-9) and np.allclose(final, want["state_out"], rtol=1e-9, atol=1e-9)
    longest = max(list(lengths) + [1])
    n = dk + dv + longest + 64
    got = {"o": o, "dq": dq, "dk": dk_, "dv": dv_}
    for name, t in got.items():
        assert t.dtype == dtype
        check(name, host(t.float()), want[name], env[name], n * (heads // kv if name in ("dk", "dv") else 1), bf16)
    check("drate", host(drate), want["drate"], env["drate"], n + tokens)
    if states:
        check("state_out", host(state_out), want["state_out"], env["state_out"], n)
        check("dstate_in", host(dsi), want["dstate_in"], env["dstate_in"], n)
    else:
        assert dsi is None


def dtypes():
    import torch
    return [torch.float32, torch.bfloat16]


LENGTHS = [[1], [2], [0], [16, 17], [63, 64, 65], [0, 1, 0, 129, 0], [200], [31, 32, 33, 0, 127, 128, 1], [513], [1100, 3]]


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_lengths(lengths, states, dt):
    run_case(lengths, 4, 2, 64, 64, dtypes()[dt], states, seed=len(lengths))


@pytest.mark.parametrize("dims", [(1, 1), (3, 5), (16, 24), (33, 130), (64, 128), (80, 96), (128, 64), (128, 128), (127, 129),
                                  (256, 256), (256, 8), (7, 250)], ids=str)
@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_channels(dims, dt):
    run_case([130, 0, 67], 3, 3, *dims, dtypes()[dt], True, seed=dims[0])


@pytest.mark.parametrize("heads", [(1, 1), (8, 1), (8, 4), (5, 5)], ids=str)
@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_heads(heads, dt):
    run_case([70, 300], *heads, 32, 48, dtypes()[dt], True, seed=heads[0])


@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_tokens_outside_every_sequence_are_zero(dt):
    run_case([40, 0, 100], 2, 1, 64, 32, dtypes()[dt], True, seed=3, lead=5, tail=130)
    run_case([0], 2, 2, 16, 16, dtypes()[dt], True, seed=4, lead=70, tail=0)


@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_many_sequences(dt):
    r = np.random.default_rng(5)
    run_case([int(x) for x in r.integers(0, 90, 61)], 2, 2, 32, 32, dtypes()[dt], True, seed=5)


@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_long_sequences_over_several_segments(dt):
    run_case([5003, 20, 3001], 2, 1, 24, 40, dtypes()[dt], True, seed=6)
    run_case([9000], 1, 1, 64, 64, dtypes()[dt], False, seed=7, use_offsets=False)


@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_batch_axis_equals_packed(dt):
    import torch
    import laplace_prefix_scans_amd as lp
    x = cuda(make(1, 3 * 150, 2, 2, 64, 64, 3, dtypes()[dt], True))
    off = torch.tensor([0, 150, 300, 450], dtype=torch.int32).cuda()
    b = {n: x[n].view(3, 150, *x[n].shape[1:]) for n in ("q", "k", "v", "go")}
    for packed, batched in (
            (lp.laplex_decay_attn(x["q"], x["k"], x["v"], x["rate"], offsets=off, state_in=x["state_in"]),
             lp.laplex_decay_attn(b["q"], b["k"], b["v"], x["rate"], state_in=x["state_in"])),):
        assert torch.equal(packed, batched.view(packed.shape))
    gp = lp.laplex_decay_attn_backward(x["q"], x["k"], x["v"], x["rate"], x["go"], offsets=off, dstate_out=x["dstate_out"])
    gb = lp.laplex_decay_attn_backward(b["q"], b["k"], b["v"], x["rate"], b["go"], dstate_out=x["dstate_out"])
    for p, q in zip(gp[:4], gb[:4]):
        assert torch.equal(p, q.view(p.shape))


@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("dims", [(64, 64), (40, 24), (33, 17)], ids=str)
def test_strided_and_unaligned_inputs_give_the_same_bits(dt, dims):
    """q, k, v as slices of one projection, at an element offset that breaks 16-byte alignment."""
    import torch
    import laplace_prefix_scans_amd as lp
    dk, dv = dims
    H, T = 3, 200
    x = cuda(make(2, T, H, H, dk, dv, 1, dtypes()[dt], False))
    want = lp.laplex_decay_attn(x["q"], x["k"], x["v"], x["rate"])
    grads = lp.laplex_decay_attn_backward(x["q"], x["k"], x["v"], x["rate"], x["go"])
    for pad in (0, 1, 8):
        width = H * (2 * dk + dv) + pad
        buf = torch.full((T * width + pad,), float("nan"), dtype=x["q"].dtype).cuda()
        rows = buf[pad:].view(T, width)
        q = rows[:, :H * dk].unflatten(1, (H, dk))
        k = rows[:, H * dk:2 * H * dk].unflatten(1, (H, dk))
        v = rows[:, 2 * H * dk:H * (2 * dk + dv)].unflatten(1, (H, dv))
        q.copy_(x["q"]), k.copy_(x["k"]), v.copy_(x["v"])
        assert torch.equal(lp.laplex_decay_attn(q, k, v, x["rate"]), want)
        for a, b in zip(lp.laplex_decay_attn_backward(q, k, v, x["rate"], x["go"])[:4], grads[:4]):
            assert torch.equal(a, b)
    # heads before tokens, and one key/value head broadcast by a stride of zero
    qt = x["q"].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(lp.laplex_decay_attn(qt, x["k"], x["v"], x["rate"]), want)
    k1, v1 = x["k"][:, :1], x["v"][:, :1]
    assert torch.equal(lp.laplex_decay_attn(x["q"], k1.expand(T, H, dk), v1.expand(T, H, dv), x["rate"]),
                       lp.laplex_decay_attn(x["q"], k1.contiguous(), v1.contiguous(), x["rate"]))


@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_token_offsets_past_32_bits(dt):
    import torch
    import laplace_prefix_scans_amd as lp
    T, stride = 70, 1 << 26  # 4.5e9 elements apart
    x = cuda(make(3, T, 2, 2, 32, 32, 1, dtypes()[dt], False))
    buf = torch.empty(T * stride, dtype=x["q"].dtype, device="cuda")
    rows = torch.as_strided(buf, (T, 2, 96), (stride, 96, 1))
    q, k, v = rows[..., :32], rows[..., 32:64], rows[..., 64:]
    q.copy_(x["q"]), k.copy_(x["k"]), v.copy_(x["v"])
    assert torch.equal(lp.laplex_decay_attn(q, k, v, x["rate"]), lp.laplex_decay_attn(x["q"], x["k"], x["v"], x["rate"]))
    for a, b in zip(lp.laplex_decay_attn_backward(q, k, v, x["rate"], x["go"])[:4],
                    lp.laplex_decay_attn_backward(x["q"], x["k"], x["v"], x["rate"], x["go"])[:4]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")], ids=str)
@pytest.mark.parametrize("which", ["q", "k", "v"])
@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_nonfinite_tokens_stay_behind_the_mask(value, which, dt):
    """A bad value in token j of one sequence: earlier tokens, other sequences and other heads keep their bits,
    the token's own output is non-finite."""
    import torch
    import laplace_prefix_scans_amd as lp
    for j in (0, 5, 70, 149):
        x = cuda(make(4, 300, 2, 2, 64, 64, 2, dtypes()[dt], False))
        x["rate"] = torch.tensor([0.01, 0.2]).cuda()
        off = torch.tensor([0, 150, 300], dtype=torch.int32).cuda()
        want = lp.laplex_decay_attn(x["q"], x["k"], x["v"], x["rate"], offsets=off)
        x[which][j, 1, 3] = value
        got = lp.laplex_decay_attn(x["q"], x["k"], x["v"], x["rate"], offsets=off)
        assert torch.equal(got[:j], want[:j]) and torch.equal(got[150:], want[150:]) and torch.equal(got[:, 0], want[:, 0])
        assert not torch.isfinite(got[j, 1]).all()
        if which == "q":
            assert torch.equal(got[j + 1:], want[j + 1:])
    # backward: dk_j, dv_j see the tokens i >= j only, dq_i those j <= i
    x = cuda(make(5, 150, 2, 2, 64, 64, 1, dtypes()[dt], False))
    x["rate"] = torch.tensor([0.01, 0.2]).cuda()
    want = lp.laplex_decay_attn_backward(x["q"], x["k"], x["v"], x["rate"], x["go"])
    x["go"][70, 1, 3] = value
    got = lp.laplex_decay_attn_backward(x["q"], x["k"], x["v"], x["rate"], x["go"])
    assert torch.equal(got[0][:70], want[0][:70]) and torch.equal(got[0][71:], want[0][71:])
    for a, b in ((got[1], want[1]), (got[2], want[2])):
        assert torch.equal(a[71:], b[71:]) and torch.equal(a[:, 0], b[:, 0])
    assert torch.equal(got[3][:1], want[3][:1])


def test_gradients_against_differences():
    """The loss <go, o> + <dstate_out, state_out> is linear in q, in k (given q and v), in v and in the
    initial state, so a central difference with a step of 1 has no truncation error: only the rounding of
    two float32 passes, about 1e-6 of the sum of the products' magnitudes.  In the rate, h = 2^-9 leaves
    h^2 / 6 of the third derivative, estimated from a second difference at twice the step."""
    import torch
    import laplace_prefix_scans_amd as lp
    x = make(6, 333, 4, 2, 40, 56, 2, torch.float32, True)
    x["rate"] = torch.tensor([0.05, 0.3, 0.01, 0.9])
    d = cuda(x)
    off = torch.tensor([0, 133, 333], dtype=torch.int32).cuda()

    def loss(**over):
        y = {**d, **over}
        so = torch.empty_like(d["state_in"])
        o = lp.laplex_decay_attn(y["q"], y["k"], y["v"], y["rate"], offsets=off, scale=0.2, state_in=y["state_in"], state_out=so)
        return (o.double() * d["go"].double()).sum() + (so.double() * d["dstate_out"].double()).sum(), \
            ((o.double() * d["go"].double()) ** 2).sum().sqrt() + ((so.double() * d["dstate_out"].double()) ** 2).sum().sqrt()

    dq, dk, dv, drate, dsi = lp.laplex_decay_attn_backward(d["q"], d["k"], d["v"], d["rate"], d["go"], offsets=off, scale=0.2,
                                                           state_in=d["state_in"], dstate_out=d["dstate_out"])
    g = torch.Generator().manual_seed(9)
    for name, grad in (("q", dq), ("k", dk), ("v", dv), ("state_in", dsi)):
        e = torch.randn(d[name].shape, generator=g).cuda()
        (up, nu), (down, nd) = loss(**{name: d[name] + e}), loss(**{name: d[name] - e})
        # the rounding of the outputs (1e-5 of their root sum of squares) and of the perturbed inputs (one part in 2^24)
        assert abs(float((up - down) / 2 - (grad.double() * e.double()).sum())) <= 1e-5 * float(nu + nd), name
    for h in range(4):
        def at(step):
            r = d["rate"].clone()
            r[h] += step
            return loss(rate=r)
        (u1, n1), (d1, _) = at(2.0 ** -9), at(-2.0 ** -9)
        (u2, _), (d2, _) = at(2.0 ** -8), at(-2.0 ** -8)
        one, two = float(u1 - d1) * 2 ** 8, float(u2 - d2) * 2 ** 7
        # one - truth = (two - one) / 3 to fourth order; twice that, and rounding over the step
        assert abs(one - float(drate[h])) <= abs(two - one) + 1e-5 * float(n1) * 2 ** 8, h


def test_repeats_streams_and_workspaces_give_the_same_bits():
    import torch
    import laplace_prefix_scans_amd as lp
    for dt in dtypes():
        x = cuda(make(7, 2000, 4, 2, 64, 64, 3, dt, True))
        off = torch.tensor([0, 900, 901, 2000], dtype=torch.int32).cuda()

        def go(ws_f=None, ws_b=None):
            so = torch.empty_like(x["state_in"])
            o = lp.laplex_decay_attn(x["q"], x["k"], x["v"], x["rate"], offsets=off, state_in=x["state_in"], state_out=so, ws=ws_f)
            return (o, so) + lp.laplex_decay_attn_backward(x["q"], x["k"], x["v"], x["rate"], x["go"], offsets=off,
                                                           state_in=x["state_in"], dstate_out=x["dstate_out"], ws=ws_b)
        want = go()
        dirty = [torch.full((max(256, lp.laplex_decay_attn_workspace_bytes(b, x["q"], x["k"], x["v"], x["rate"], off)),), 255,
                            dtype=torch.uint8).cuda() for b in (False, True)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = go(*dirty)
        side.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ one token
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1), (1, 8, 8, 64, 64), (5, 4, 2, 80, 96), (17, 3, 1, 128, 128), (4, 2, 2, 256, 256),
                                   (3, 2, 2, 33, 7), (300, 1, 1, 64, 66)], ids=str)
@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_step(shape, dt):
    import torch
    import laplace_prefix_scans_amd as lp
    n, heads, kv, dk, dv = shape
    dtype = dtypes()[dt]
    x = make(n, n, heads, kv, dk, dv, n + 3, dtype, True)
    d = cuda(x)
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(n + 3, generator=g)[:n].to(torch.int32)
    if n > 2:
        slots[1], slots[2] = -1, n + 3  # outside the pool
    pool = d["state_in"].clone()
    o = lp.laplex_decay_attn_step(d["q"], d["k"], d["v"], d["rate"], pool, slots=slots.cuda(), scale=0.5)
    want_pool, env_pool = npf(x["state_in"]).astype(np.float64), np.abs(npf(x["state_in"])).astype(np.float64)
    want, env = np.zeros((n, heads, dv)), np.zeros((n, heads, dv))
    w = ref.weight_per_head(npf(x["rate"]), 1)[:, None, None]
    for r, s in enumerate(slots.tolist()):
        if not 0 <= s < n + 3:
            continue
        q, k, v = (npf(x[m])[r].astype(np.float64) for m in ("q", "k", "v"))
        k, v = np.repeat(k, heads // kv, 0)[:, :, None], np.repeat(v, heads // kv, 0)[:, None, :]
        want_pool[s] = w * want_pool[s] + k * v
        env_pool[s] = w * env_pool[s] + np.abs(k * v)
        want[r] = 0.5 * np.einsum("hk,hkv->hv", q, want_pool[s])
        env[r] = 0.5 * np.einsum("hk,hkv->hv", np.abs(q), env_pool[s])
    check("state", host(pool), want_pool, env_pool, 2)
    check("o", host(o.float()), want, env, dk, dt == 1)
    dead = [r for r, s in enumerate(slots.tolist()) if not 0 <= s < n + 3]
    assert not host(o.float())[dead].any()


def test_steps_continue_a_prompt():
    """A prompt's final state carried on token by token gives what one pass over both gives."""
    import torch
    import laplace_prefix_scans_amd as lp
    x = cuda(make(8, 100, 4, 2, 64, 48, 1, torch.float32, False))
    x["rate"] = torch.tensor([0.0, 0.01, 0.4, 3.0]).cuda()
    whole = lp.laplex_decay_attn(x["q"], x["k"], x["v"], x["rate"])
    state = torch.empty(1, 4, 64, 48, device="cuda")
    first = lp.laplex_decay_attn(x["q"][:90], x["k"][:90], x["v"][:90], x["rate"], state_out=state)
    rest = [lp.laplex_decay_attn_step(x["q"][t:t + 1], x["k"][t:t + 1], x["v"][t:t + 1], x["rate"], state) for t in range(90, 100)]
    got = host(torch.cat([first] + rest))
    env = np.abs(host(whole)).max()
    assert np.abs(got - host(whole)).max() <= 1e-5 * env


def test_step_state_offsets_past_32_bits():
    import torch
    import laplace_prefix_scans_amd as lp
    pool = 140000  # 2.3e9 floats
    state = torch.empty(pool, 1, 128, 128, device="cuda")
    slots = torch.tensor([pool - 1, 0, 131072], dtype=torch.int32).cuda()
    x = cuda(make(9, 3, 1, 1, 128, 128, 3, torch.float32, True))
    state[slots.long()] = x["state_in"]
    small = x["state_in"].clone()
    a = lp.laplex_decay_attn_step(x["q"], x["k"], x["v"], x["rate"], state, slots=slots)
    b = lp.laplex_decay_attn_step(x["q"], x["k"], x["v"], x["rate"], small)
    assert torch.equal(a, b) and torch.equal(state[slots.long()], small)
