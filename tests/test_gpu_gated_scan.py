"""The gated linear recurrence on the GPU against a token-by-token recurrence in float64.  Tolerances: train_ref.scan
follows each operation's rounding through the recurrence; bfloat16 results add half a step, 2^-8 of the value."""
import numpy as np
import pytest

import train_ref as ref
from gpu_util import have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]
KINDS = ["rate", "sigmoid"]


def dtype_of(name):
    import torch
    return torch.float32 if name == "f32" else torch.bfloat16


def check(name, got, want, bound, bf16):
    got = host(got.float())
    assert got.shape == want.shape, name
    assert np.isfinite(got).all(), "%s: non-finite" % name
    tol = bound + np.abs(want) * (2.0 ** -8 if bf16 else 2.0 ** -24) + 1e-37
    bad = np.abs(got - want) > tol
    assert not bad.any(), "%s: %d of %d off, worst %.2f of the bound, first at %s" % (
        name, bad.sum(), bad.size, (np.abs(got - want) / tol).max(), np.argwhere(bad)[:3].tolist())


def make(seed, tokens, channels, seqs, dtype, kind, slow=False):
    import torch
    g = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    if kind == "rate":
        z = torch.exp(1.5 * normal(tokens, channels) - (7 if slow else 1))
        if tokens and not slow:
            z[0, 0], z[-1, -1], z[tokens // 2, channels // 2] = 0.0, float("inf"), 25.0
    else:
        z = 2 * normal(tokens, channels) + (8 if slow else 0)
        if tokens and not slow:
            z[0, 0], z[-1, -1], z[tokens // 2, channels // 2] = 0.0, float("-inf"), 30.0
    return {"gate": z.to(dtype), "x": normal(tokens, channels).to(dtype), "dh": normal(tokens, channels).to(dtype),
            "state_in": normal(seqs, channels), "dstate_out": normal(seqs, channels)}


def run_case(lengths, channels, dt, kind, states=True, seed=0, lead=0, tail=0, use_offsets=True, slow=False):
    import torch
    import laplace_prefix_scans_amd as lp
    dtype = dtype_of(dt)
    bounds = [lead + int(c) for c in np.concatenate([[0], np.cumsum(lengths)])]
    tokens, n = bounds[-1] + tail, len(lengths)
    print("scan lengths=%s channels=%d %s %s states=%s" % (lengths[:8], channels, dt, kind, states), flush=True)
    x = make(seed, tokens, channels, n, dtype, kind, slow)
    if not states:
        x["state_in"] = x["dstate_out"] = None
    c = {k: None if v is None else v.cuda() for k, v in x.items()}
    off = torch.tensor(bounds, dtype=torch.int32).cuda() if use_offsets else None
    nan = lambda: torch.full((n, channels), float("nan")).cuda()  # noqa: E731
    state_out = nan() if states else None
    h, carries = lp.laplex_gated_scan(c["gate"], c["x"], kind, offsets=off, state_in=c["state_in"], state_out=state_out, keep=True)
    dgate, dx, dsi = lp.laplex_gated_scan_backward(c["gate"], c["x"], carries, c["dh"], kind, offsets=off, state_in=c["state_in"],
                                                   dstate_out=c["dstate_out"])
    npf = lambda t: None if t is None else t.float().numpy()  # noqa: E731
    want = ref.scan(npf(x["gate"]), npf(x["x"]), kind, bounds, npf(x["state_in"]), npf(x["dh"]), npf(x["dstate_out"]))
    for name, t in (("h", h), ("dgate", dgate), ("dx", dx)):
        assert t.dtype == dtype
        check(name, t, want[name], want["~" + name], dt == "bf16")
    if states:
        check("state_out", state_out, want["state_out"], want["~state_out"], False)
        check("dstate_in", dsi, want["dstate_in"], want["~dstate_in"], False)
    else:
        assert dsi is None
    # the same without what training needs
    assert torch.equal(h, lp.laplex_gated_scan(c["gate"], c["x"], kind, offsets=off, state_in=c["state_in"]))


LENGTHS = [[1], [2], [0], [15, 16, 17], [16, 16], [0, 1, 0, 0, 33, 0], [64], [65], [127, 1, 128], [1] * 70, [300], [0] * 90 + [40, 0, 3]]


@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda v: "-".join(map(str, v[:6])))
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_lengths(lengths, kind, dt):
    run_case(lengths, 70, dt, kind, states=len(lengths) % 2 == 1, seed=len(lengths))


@pytest.mark.parametrize("channels", [1, 2, 3, 63, 64, 65, 127, 128, 129, 1001])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_channels(channels, dt):
    run_case([37, 0, 90], channels, dt, KINDS[channels % 2], seed=channels)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_many_segments_and_slow_decays(kind, dt):
    run_case([4099, 1, 0, 700, 3000], 40, dt, kind, seed=3, slow=True)


def test_a_long_sequence_in_as_many_segments_as_there_are():
    run_case([40000], 6, "f32", "rate", seed=4, slow=True)
    run_case([20000, 20001], 5, "bf16", "sigmoid", seed=5, slow=True)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_tokens_outside_every_sequence_are_zero(dt):
    for lead, tail in ((5, 0), (0, 9), (16, 16), (100, 77)):
        run_case([30, 50], 20, dt, KINDS[lead % 2], lead=lead, tail=tail, seed=lead)


@pytest.mark.parametrize("kind", KINDS)
def test_batches_and_strides(kind):
    import torch
    import laplace_prefix_scans_amd as lp
    torch.manual_seed(1)
    wide = torch.rand(3, 50, 2, 90, device="cuda")
    gate, x = wide[:, :, 0, 3:80], wide[:, :, 1, 1:78]
    dh, si, so = torch.randn(3, 50, 77, device="cuda"), torch.randn(3, 77, device="cuda"), torch.empty(3, 77, device="cuda")
    h, c = lp.laplex_gated_scan(gate, x, kind, state_in=si, state_out=so, keep=True)
    g = lp.laplex_gated_scan_backward(gate, x, c, dh, kind, state_in=si)
    off = torch.tensor([0, 50, 100, 150], dtype=torch.int32, device="cuda")
    flat = lambda t: t.reshape(150, 77).contiguous()  # noqa: E731
    h2, c2 = lp.laplex_gated_scan(flat(gate), flat(x), kind, offsets=off, state_in=si, keep=True)
    g2 = lp.laplex_gated_scan_backward(flat(gate), flat(x), c2, flat(dh), kind, offsets=off, state_in=si)
    assert torch.equal(flat(h), h2) and torch.equal(c, c2)
    assert torch.equal(flat(g[0]), flat(g2[0])) and torch.equal(flat(g[1]), flat(g2[1])) and torch.equal(g[2], g2[2])
    assert torch.equal(so, h[:, -1])  # float32: the last output is the state
    one = lp.laplex_gated_scan(gate[:, 7:8], x[:, 7:8], kind, state_in=si)  # single tokens of longer sequences
    assert torch.equal(one, lp.laplex_gated_scan(gate[:, 7:8].contiguous(), x[:, 7:8].contiguous(), kind, state_in=si))


@pytest.mark.parametrize("kind", KINDS)
def test_a_broadcast_gate(kind):
    """A gate that does not depend on the token: a token stride of zero."""
    import torch
    import laplace_prefix_scans_amd as lp
    gate, x = torch.rand(1, 33, device="cuda").expand(200, 33), torch.randn(200, 33, device="cuda")
    assert torch.equal(lp.laplex_gated_scan(gate, x, kind), lp.laplex_gated_scan(gate.contiguous(), x, kind))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_non_finite_tokens_stay_in_their_sequence_and_channel(kind, dt):
    import torch
    import laplace_prefix_scans_amd as lp
    lengths = [100, 1, 300, 0, 500]
    bounds = np.concatenate([[0], np.cumsum(lengths)])
    x = {k: v.cuda() for k, v in make(8, 901, 70, 5, dtype_of(dt), kind, slow=True).items()}
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")

    def both():
        h, c = lp.laplex_gated_scan(x["gate"], x["x"], kind, offsets=off, state_in=x["state_in"], keep=True)
        return (h,) + lp.laplex_gated_scan_backward(x["gate"], x["x"], c, x["dh"], kind, offsets=off, state_in=x["state_in"])[:2]
    clean = both()
    bad = {(150, 3): float("nan"), (150, 4): float("inf"), (99, 10): float("nan"), (450, 20): float("-inf"), (400, 0): float("nan")}
    for (t, ch), value in bad.items():
        x["x"][t, ch] = value
    h, dgate, dx = both()
    hit = torch.zeros(901, 70, dtype=torch.bool, device="cuda")
    for t, ch in bad:
        end = int(bounds[np.searchsorted(bounds, t, side="right")])
        hit[t:end, ch] = True
    assert torch.isfinite(h[~hit]).all() and not torch.isfinite(h[hit]).any()
    assert torch.equal(h[~hit], clean[0][~hit])
    assert torch.equal(dx, clean[2])  # no input enters it
    assert torch.equal(dgate[~hit], clean[1][~hit])
    x["dh"][200, 33] = float("nan")
    for t, ch in bad:
        x["x"][t, ch] = 0.0
    h, dgate, dx = both()
    hit[:] = False
    hit[101:201, 33] = True
    assert torch.isfinite(h).all() and torch.isfinite(dx[~hit]).all() and torch.isnan(dx[hit]).all()
    assert torch.isfinite(dgate[~hit]).all()


@pytest.mark.parametrize("kind", KINDS)
def test_gradients_against_differences(kind):
    import torch
    import laplace_prefix_scans_amd as lp
    bounds = [0, 7, 7, 20]
    x = {k: v.numpy().astype(np.float64) for k, v in make(6, 20, 3, 3, torch.float32, kind, slow=False).items()}
    x["gate"] = np.clip(x["gate"], -3, 3) + (0.1 if kind == "rate" else 0.0)
    c = {k: torch.from_numpy(v).float().cuda() for k, v in x.items()}
    x = {k: v.cpu().numpy().astype(np.float64) for k, v in c.items()}
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    _, carries = lp.laplex_gated_scan(c["gate"], c["x"], kind, offsets=off, state_in=c["state_in"], keep=True)
    got = lp.laplex_gated_scan_backward(c["gate"], c["x"], carries, c["dh"], kind, offsets=off, state_in=c["state_in"],
                                        dstate_out=c["dstate_out"])

    def loss():
        r = ref.scan(x["gate"], x["x"], kind, bounds, x["state_in"])
        return (r["h"] * x["dh"]).sum() + (r["state_out"] * x["dstate_out"]).sum()
    for name, g in zip(("gate", "x", "state_in"), got):
        for at in np.ndindex(x[name].shape):
            keep, step = x[name][at], 1e-5
            x[name][at] = keep + step
            up = loss()
            x[name][at] = keep - step
            down = loss()
            x[name][at] = keep
            # central differences: third derivatives of order 10 times step^2, cancellation of 20 2^-53 / step
            assert abs(float(g[at]) - (up - down) / (2 * step)) < 2e-5 * (1 + abs(float(g[at]))), (name, at)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("channels", [1, 64, 513])
def test_steps_follow_the_whole_pass(kind, dt, channels):
    import torch
    import laplace_prefix_scans_amd as lp
    x = {k: v.cuda() for k, v in make(9, 60, channels, 2, dtype_of(dt), kind).items()}
    state = torch.full((5, channels), 7.0, device="cuda")
    state[3], state[1] = x["state_in"][0], x["state_in"][1]
    slots = torch.tensor([3, -1, 1, 5, -(2 ** 31)], dtype=torch.int32, device="cuda")
    outs = []
    for t in range(30):
        rows = torch.tensor([t, 0, 30 + t, 0, 0], device="cuda")
        outs.append(lp.laplex_gated_scan_step(x["gate"][rows], x["x"][rows], state, kind, slots=slots))
    outs = torch.stack(outs)
    assert (outs[:, [1, 3, 4]] == 0).all() and (state[[0, 2, 4]] == 7.0).all()
    off = torch.tensor([0, 30, 60], dtype=torch.int32, device="cuda")
    so = torch.empty(2, channels, device="cuda")
    h = lp.laplex_gated_scan(x["gate"], x["x"], kind, offsets=off, state_in=x["state_in"], state_out=so)
    # one segment of tokens: the same operations in the same order
    assert torch.equal(outs[:, 0], h[:30]) and torch.equal(outs[:, 2], h[30:])
    assert torch.equal(state[3], so[0]) and torch.equal(state[1], so[1])


def test_steps_without_slots_and_past_2_32_elements():
    import torch
    import laplace_prefix_scans_amd as lp
    gate, x = torch.rand(3, 40, device="cuda"), torch.randn(3, 40, device="cuda")
    state = torch.randn(4, 40, device="cuda")
    want = torch.exp(-gate.double()) * state[:3].double() + x.double()
    keep = state[3].clone()
    h = lp.laplex_gated_scan_step(gate, x, state)
    assert torch.equal(h, state[:3]) and torch.equal(state[3], keep)
    assert ((h - want).abs() < 1e-5).all()
    pool = torch.zeros((1 << 16) + 3, 1 << 16, device="cuda")  # 17 GB: the last rows begin past 2^32 elements
    slots = torch.tensor([(1 << 16) + 2, 0], dtype=torch.int32, device="cuda")
    gate, x = torch.zeros(2, 1 << 16, device="cuda"), torch.randn(2, 1 << 16, device="cuda")
    h = lp.laplex_gated_scan_step(gate, x, pool, slots=slots)
    assert torch.equal(h, x) and torch.equal(pool[-1], x[0]) and torch.equal(pool[0], x[1]) and not pool[1].any()


def test_a_repeated_call_gives_the_same_bits_also_in_a_used_workspace():
    import torch
    import laplace_prefix_scans_amd as lp
    x = {k: v.cuda() for k, v in make(2, 5000, 200, 1, torch.bfloat16, "sigmoid").items()}
    need = max(lp.laplex_gated_scan_workspace_bytes(x["gate"][:t], x["x"][:t]) for t in (5000, 4999, 3000))
    assert need == lp.laplex_gated_scan_workspace_bytes(x["gate"], x["x"]) > 0
    for t in (5000, 4999, 4990, 100):
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        a = (x["gate"][:t], x["x"][:t])
        h, c = lp.laplex_gated_scan(*a, "sigmoid", keep=True)
        h2, c2 = lp.laplex_gated_scan(*a, "sigmoid", keep=True, ws=ws)
        assert torch.equal(h, h2) and torch.equal(c, c2)
        for p, q in zip(lp.laplex_gated_scan_backward(*a, c, x["dh"][:t], "sigmoid")[:2],
                        lp.laplex_gated_scan_backward(*a, c, x["dh"][:t], "sigmoid", ws=ws.fill_(255))[:2]):
            assert torch.equal(p, q)


def test_no_tokens_and_no_sequences():
    import torch
    import laplace_prefix_scans_amd as lp
    e = torch.empty(0, 9, device="cuda")
    si = torch.randn(2, 9, device="cuda")
    so = torch.empty(2, 9, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    h, c = lp.laplex_gated_scan(e, e, offsets=off, state_in=si, state_out=so, keep=True)
    assert h.shape == (0, 9) and c.shape == (0, 9) and torch.equal(so, si)
    dg, dx, ds = lp.laplex_gated_scan_backward(e, e, c, e, offsets=off, state_in=si, dstate_out=so * 2)
    assert dg.shape == dx.shape == (0, 9) and torch.equal(ds, so * 2)
    assert (lp.laplex_gated_scan_backward(e, e, c, e, offsets=off, state_in=si)[2] == 0).all()
    x = torch.empty(2, 0, 9, device="cuda")  # a batch of no tokens
    lp.laplex_gated_scan(x, x, state_in=si, state_out=so.zero_())
    assert torch.equal(so, si)
    assert lp.laplex_gated_scan(e, e, offsets=off[:1]).shape == (0, 9)
    assert lp.laplex_gated_scan_step(e, e, si).shape == (0, 9)


def test_another_stream():
    import torch
    import laplace_prefix_scans_amd as lp
    x = {k: v.cuda() for k, v in make(2, 3000, 300, 1, torch.float32, "rate").items()}
    want = lp.laplex_gated_scan(x["gate"], x["x"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = lp.laplex_gated_scan(x["gate"], x["x"])
        got.record_stream(s)
    s.synchronize()
    assert torch.equal(got, want)


def test_as_many_tokens_as_offsets_can_name():
    """2^31 - 1 tokens of one channel: constant inputs, whose states and gradients settle to those of an endless sequence."""
    import torch
    import laplace_prefix_scans_amd as lp
    n = 2 ** 31 - 1
    gate, x = torch.full((1, 1), 1.0, device="cuda").expand(n, 1), torch.ones(n, 1, device="cuda")
    h, carries = lp.laplex_gated_scan(gate, x, keep=True)
    a = float(np.exp(-1.0))
    want = 1 / (1 - a)
    # the decay is off by 14 roundings, and what it multiplies is 1 / (1 - a) times as much; each token adds two
    tol = 16 * ref.U * want / (1 - a)
    settled = h[40:]  # (e^-40 of the beginning is left)
    assert abs(float(settled.max()) - want) <= tol and abs(float(settled.min()) - want) <= tol and abs(float(h[0]) - 1) <= ref.U
    dgate, dx, _ = lp.laplex_gated_scan_backward(gate, x, carries, h.fill_(1.0))
    del h
    assert abs(float(dx[:-40].max()) - want) <= tol and abs(float(dx[:-40].min()) - want) <= tol and float(dx[-1]) == 1.0
    del dx
    settled = dgate[41:-41]
    want = -a * want * want
    tol = 3 * tol * abs(want)
    assert abs(float(settled.max()) - want) <= tol and abs(float(settled.min()) - want) <= tol and float(dgate[0]) == 0.0


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_offsets_outside_the_tokens_touch_nothing_else(dt):
    """Offsets that are not ascending, negative or past the tokens: whatever they give, it stays inside the call's tensors."""
    import torch
    import laplace_prefix_scans_amd as lp
    dtype = dtype_of(dt)
    tokens, channels, guard = 300, 70, 1 << 16
    g = torch.Generator().manual_seed(0)
    gate, x, dh = (torch.randn(tokens, channels, generator=g).to(dtype).cuda() for _ in range(3))
    for bad in ([0, 100, 50, 300], [-40, 20, 20, 290], [0, 10, 400, 70000], [2 ** 31 - 1, 0, 5, 300], [300, 200, 100, 0], [-5, -4, -3, -2]):
        offsets = torch.tensor(bad, dtype=torch.int32).cuda()
        whole = torch.full((guard + 3 * channels + guard,), 7.0, device="cuda")
        state_out = whole[guard:guard + 3 * channels].view(3, channels)
        buf = torch.full((guard + tokens * channels + guard,), 7.0, dtype=dtype, device="cuda")
        state_in = torch.ones(3, channels, device="cuda")
        h, carries = lp.laplex_gated_scan(gate, x, "sigmoid", offsets=offsets, state_in=state_in, state_out=state_out, keep=True,
                                          h=buf[guard:guard + tokens * channels].view(tokens, channels))
        lp.laplex_gated_scan_backward(gate, x, carries, dh, "sigmoid", offsets=offsets, state_in=state_in)
        torch.cuda.synchronize()
        for t, n in ((whole, 3 * channels), (buf, tokens * channels)):
            assert (t[:guard] == 7).all() and (t[guard + n:] == 7).all(), bad
