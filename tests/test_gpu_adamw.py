"""The AdamW step on the GPU against float64, and its 8-bit moments against the format's definition."""
import math

import numpy as np
import pytest

import train_ref as ref
from gpu_util import have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]
SIZES = [1, 2, 7, 8, 9, 255, 256, 257, 2047, 2048, 2049, 5000, 0, 40000]
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8)


def make(sizes, pd, gd, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    normal = lambda n: torch.randn(n, generator=g)  # noqa: E731
    return {"p": [normal(n).to(pd) for n in sizes], "g": [(1e-2 * normal(n)).to(gd) for n in sizes], "m": [1e-3 * normal(n) for n in sizes],
            "v": [(1e-3 * normal(n)) ** 2 for n in sizes]}


def cuda(x):
    return {k: [t.cuda() for t in v] for k, v in x.items()}


def dtypes(name):
    import torch
    return {"f": torch.float32, "b": torch.bfloat16}[name]


@pytest.mark.parametrize("types", ["ff", "fb", "bf", "bb"])
@pytest.mark.parametrize("step", [1, 1000])
def test_float_moments(types, step):
    import laplace_prefix_scans_amd as lp
    x = make(SIZES, dtypes(types[0]), dtypes(types[1]), step)
    decays = [0.1 * (i % 3) for i in range(len(SIZES))]
    c = cuda(x)
    lp.laplex_adamw(c["p"], c["g"], c["m"], c["v"], step=step, weight_decay=decays, **HYPER)
    for i, n in enumerate(SIZES):
        a = [x[k][i].float().numpy() for k in ("p", "g", "m", "v")]
        p, m, v, err = ref.adamw(*a, HYPER["lr"], *HYPER["betas"], HYPER["eps"], decays[i], step)
        assert (np.abs(host(c["p"][i].float()) - p) <= err + (np.abs(p) * 2.0 ** -8 if types[0] == "b" else 0)).all()
        # betas and their complements rounded, three operations
        assert (np.abs(host(c["m"][i]) - m) <= 4 * ref.U * (0.9 * np.abs(a[2]) + 0.1 * np.abs(a[1]))).all()
        assert (np.abs(host(c["v"][i]) - v) <= 5 * ref.U * v).all()


def test_master_copies():
    import torch
    import laplace_prefix_scans_amd as lp
    x = make(SIZES, torch.bfloat16, torch.bfloat16)
    c = cuda(x)
    master = [t.float() + 1e-4 for t in c["p"]]
    plain = [t.clone() for t in master]
    m, v = [t.clone() for t in c["m"]], [t.clone() for t in c["v"]]
    lp.laplex_adamw(c["p"], c["g"], c["m"], c["v"], step=3, master=master, **HYPER)
    lp.laplex_adamw(plain, c["g"], m, v, step=3, **HYPER)
    for a, b, p in zip(master, plain, c["p"]):
        assert torch.equal(a, b) and torch.equal(p, a.bfloat16())


def test_many_tensors_are_the_same_as_one_at_a_time():
    import torch
    import laplace_prefix_scans_amd as lp
    sizes = [(i * 37) % 700 + (3000 if i % 50 == 0 else 0) for i in range(150)]
    c = cuda(make(sizes, torch.float32, torch.float32))
    d = {k: [t.clone() for t in v] for k, v in c.items()}
    lp.laplex_adamw(c["p"], c["g"], c["m"], c["v"], step=2, weight_decay=0.1, **HYPER)
    for i in range(len(sizes)):
        lp.laplex_adamw(*[d[k][i:i + 1] for k in ("p", "g", "m", "v")], step=2, weight_decay=0.1, **HYPER)
    for k in ("p", "m", "v"):
        for a, b in zip(c[k], d[k]):
            assert torch.equal(a, b)


def test_neighbours_are_left_alone():
    """Tensors that are slices, at every alignment: what lies between them stays."""
    import torch
    import laplace_prefix_scans_amd as lp
    for types in ("ff", "bb"):
        flat = {k: torch.full((9000,), 3.0, dtype=d, device="cuda") for k, d in (("p", dtypes(types[0])), ("g", dtypes(types[1])), ("m", torch.float32), ("v", torch.float32))}
        cut, at = [], 1
        for n in (5, 300, 2048, 1, 4001):
            cut.append((at, at + n))
            at += n + 3
        views = {k: [t[a:b] for a, b in cut] for k, t in flat.items()}
        lp.laplex_adamw(views["p"], views["g"], views["m"], views["v"], step=1, **HYPER)
        inside = torch.zeros(9000, dtype=torch.bool, device="cuda")
        for a, b in cut:
            inside[a:b] = True
        for k in ("p", "m", "v"):
            assert (flat[k][~inside] == 3.0).all()
            changed = flat[k][inside]
            assert (changed == changed[0]).all() and (changed[0] != 3.0 or k == "m")
        assert (flat["g"] == 3.0).all()


def test_step_rate_and_scale_on_the_device():
    import torch
    import laplace_prefix_scans_amd as lp
    sizes = [300, 5000]
    x = make(sizes, torch.float32, torch.float32)
    a, b = cuda(x), cuda(x)
    lr = float(np.float32(HYPER["lr"]))
    lp.laplex_adamw(a["p"], [g * 0.25 for g in a["g"]], a["m"], a["v"], step=7, lr=lr, betas=(0.9, 0.95), weight_decay=0.1)
    lp.laplex_adamw(b["p"], b["g"], b["m"], b["v"], step=torch.tensor([7], dtype=torch.int32, device="cuda"),
                    lr=torch.tensor(lr, device="cuda"), betas=(0.9, 0.95), weight_decay=0.1, grad_scale=torch.tensor(0.25, device="cuda"))
    for k in ("m", "v"):
        for s, t in zip(a[k], b[k]):
            assert torch.equal(s, t)
    for s, t, p in zip(a["p"], b["p"], x["p"]):
        # the host's and the device's powers may round differently: a step of the corrections, and of 1 - lr weight_decay
        assert ((s - t).abs() <= 4 * ref.U * (s.abs() + (s - p.cuda()).abs() * 4)).all()
    # a scale that is not finite: nothing changes
    for bad in (float("nan"), float("inf")):
        keep = {k: [t.clone() for t in v] for k, v in b.items()}
        lp.laplex_adamw(b["p"], b["g"], b["m"], b["v"], step=8, lr=lr, grad_scale=torch.tensor(bad, device="cuda"))
        assert all(torch.equal(s, t) for k in b for s, t in zip(b[k], keep[k]))


# ------------------------------------------------------------------ 8 bits
def e4m3_values():
    """The value of each of the 127 finite magnitudes."""
    c = np.arange(127)
    e, f = c >> 3, c & 7
    return np.where(e == 0, f * 2.0 ** -9, (1 + f / 8.0) * 2.0 ** (e - 7.0))


def eight(sizes, seed=0, gd=None):
    import torch
    x = cuda(make(sizes, torch.float32, gd or torch.float32, seed))
    x["m"] = [torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda") for n in sizes]
    x["v"] = [torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda") for n in sizes]
    x["ms"] = [torch.zeros(-(-n // 256), device="cuda") for n in sizes]
    x["vs"] = [torch.zeros(-(-n // 256), device="cuda") for n in sizes]
    return x


def step8(x, **over):
    import laplace_prefix_scans_amd as lp
    lp.laplex_adamw(x["p"], x["g"], x["m"], x["v"], m_scale=x["ms"], v_scale=x["vs"], **{**HYPER, "step": 1, **over})


def values(x):
    import laplace_prefix_scans_amd as lp
    return lp.laplex_adamw_moments(x["m"], x["v"], x["ms"], x["vs"])


@pytest.mark.parametrize("seed", [None, 5])
def test_eight_bit_moments_are_neighbouring_codes(seed):
    """After one step from zero the moments are (1 - b1) g and (1 - b2) g^2: each code is one of the two next to the value
    over the scale (to nearest: the nearer), and the values that come back are the codes'."""
    import torch
    x = eight(SIZES)
    step8(x, seed=seed)
    mv, vv = values(x)
    grid = np.append(e4m3_values(), np.inf)
    for i, n in enumerate(SIZES):
        g = host(x["g"][i])
        for name, value in (("m", np.float32(0.1) * g), ("v", np.sqrt(np.float32(0.05) * (g * g)))):
            codes, scales = host(x[name][i].view(torch.uint8)), host(x[name + "s"][i])
            assert ((codes & 128) == (128 if name == "m" else 0) * (value < 0)).all()
            at = np.repeat(scales, 256)[:n].astype(np.float64)
            for b in range(len(scales)):
                most = np.abs(value[256 * b:256 * b + 256]).max()
                assert abs(scales[b] - most / 448) <= 4 * ref.U * scales[b]
            y = np.abs(value.astype(np.float64)) / at
            mag = (codes & 127).astype(int)
            lo, hi = grid[np.maximum(mag - 1, 0)], grid[mag + 1]
            slack = 8 * ref.U * y + 2.0 ** -24  # float32 quotients; random bits end 2^-16 of a step below it
            assert ((y >= lo - slack) & (y <= hi + slack)).all()
            if seed is None:
                half_lo, half_hi = (grid[mag] + lo) / 2, (grid[mag] + np.minimum(hi, 480)) / 2
                small = (mag == 1) & (name == "v")  # what is not zero stays so
                assert (((y >= half_lo - slack) | small) & (y <= half_hi + slack)).all()
            got = host(mv[i] if name == "m" else vv[i])
            want = grid[mag] * at * np.where(codes & 128, -1, 1)
            want = want if name == "m" else want * want
            assert (np.abs(got - want) <= 3 * ref.U * np.abs(want)).all()


def test_the_step_is_made_of_moments_before_their_rounding():
    import torch
    import laplace_prefix_scans_amd as lp
    x, y = eight(SIZES, 3), cuda(make(SIZES, torch.float32, torch.float32, 3))
    y["m"], y["v"] = [torch.zeros_like(t) for t in y["p"]], [torch.zeros_like(t) for t in y["p"]]
    step8(x, seed=1, weight_decay=0.1)
    lp.laplex_adamw(y["p"], y["g"], y["m"], y["v"], step=1, weight_decay=0.1, **HYPER)
    assert all(torch.equal(a, b) for a, b in zip(x["p"], y["p"]))
    # and the next one of what the codes stand for
    mv, vv = values(x)
    q = [t.clone() for t in x["p"]]
    step8(x, seed=1, step=2)
    lp.laplex_adamw(q, x["g"], mv, vv, step=2, **HYPER)
    assert all(torch.equal(a, b) for a, b in zip(x["p"], q))


def test_random_rounding_is_fair_and_reproducible():
    import torch
    n, runs = 4096, 200
    first = eight([n], 7)
    g = host(first["g"][0])
    total = np.zeros(n)
    for r in range(runs):
        x = eight([n], 7)
        step8(x, seed=r)
        total += host(values(x)[0][0])
    want = np.float32(0.1) * g
    scale = np.repeat(host(x["ms"][0]), 256)[:n]
    gap = np.maximum(2.0 ** -9, 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want / scale), 2.0 ** -6))) - 3)) * scale
    # a fair choice between two codes has a deviation of at most half their distance; over 200 runs the mean's is 1/28 of
    # it, and the largest of 4096 stays below 5.5 of those; the mean over the elements is 64 times sharper
    dev = (total / runs - want) / gap
    assert np.abs(dev).max() < 5.5 * 0.5 / math.sqrt(runs)
    assert abs(dev.mean()) < 5 * 0.5 / math.sqrt(runs * n)
    a, b, c, d = (eight([n, n], 7) for _ in range(4))
    step8(a, seed=9)
    step8(b, seed=9)
    step8(c, seed=10)
    assert torch.equal(a["m"][0].view(torch.uint8), b["m"][0].view(torch.uint8))
    assert not torch.equal(a["m"][0].view(torch.uint8), c["m"][0].view(torch.uint8))
    for k in ("g", "p"):
        d[k][1].copy_(d[k][0])
    step8(d, seed=9)  # two tensors with the same values draw different bits
    assert not torch.equal(d["m"][0].view(torch.uint8), d["m"][1].view(torch.uint8))


def test_second_moments_follow_a_change_that_nearest_codes_would_miss():
    """Gradients fall to a tenth: with b2 = 0.999 sqrt(v) moves by 5e-4 a step, a code's width is 2^-4 or more.  Rounded at
    random the mean follows sqrt(b2^t 1 + (1 - b2^t) 0.01) to within 2 %, over 4096 elements."""
    import torch
    n = 4096
    x = eight([n])
    x["p"] = [torch.zeros(n, device="cuda")]
    v = 0.0
    for t in range(1, 401):
        size = 1.0 if t <= 100 else 0.1
        x["g"] = [torch.full((n,), size, device="cuda")]
        x["g"][0][::256] = 3.0  # an element of each block that keeps the scale where it is
        step8(x, step=t, betas=(0.9, 0.999), seed=0)
        v = 0.999 * v + 0.001 * size * size
    rest = torch.arange(n, device="cuda") % 256 != 0
    got = float(values(x)[1][0][rest].sqrt().mean())
    assert abs(got - math.sqrt(v)) < 0.02 * math.sqrt(v), (got, math.sqrt(v))


def test_moments_that_are_not_finite_or_tiny():
    import torch
    x = eight([600])
    keep = [t.clone() for t in x["p"]]
    g = x["g"][0]
    g[3], g[300], g[301] = float("nan"), float("inf"), 0.0
    g[512:] = 0.0
    step8(x, seed=1)
    m, v = values(x)
    bad = torch.zeros(600, dtype=torch.bool, device="cuda")
    bad[3] = bad[300] = True
    assert torch.isnan(m[0][bad]).all() and torch.isnan(v[0][bad]).all()
    assert torch.isfinite(m[0][~bad]).all() and torch.isfinite(v[0][~bad]).all() and torch.isfinite(x["p"][0][~bad]).all()
    assert not m[0][512:].any() and not v[0][512:].any() and torch.equal(x["p"][0][512:], keep[0][512:])
    assert (v[0][:512][(g[:512] != 0) & ~bad[:512]] > 0).all()
    x = eight([256])
    x["g"] = [torch.full((256,), 1e-40, device="cuda")]
    step8(x, seed=1)
    m, v = values(x)
    assert torch.isfinite(m[0]).all() and torch.isfinite(v[0]).all() and torch.isfinite(x["p"][0]).all()


def test_the_same_tensor_twice_is_refused():
    import torch
    import laplace_prefix_scans_amd as lp
    x = cuda(make([100, 100], torch.float32, torch.float32))
    for k in ("p", "m", "v"):
        twice = {**x, k: [x[k][0], x[k][0]]}
        with pytest.raises(lp.LaplexError) as e:
            lp.laplex_adamw(twice["p"], twice["g"], twice["m"], twice["v"], step=1, **HYPER)
        assert e.value.code == 7
    with pytest.raises(lp.LaplexError):
        lp.laplex_adamw(x["p"], x["p"], x["m"], x["v"], step=1, **HYPER)
    lp.laplex_adamw(x["p"], [x["g"][0], x["g"][0]], x["m"], x["v"], step=1, **HYPER)  # a gradient may be shared


def test_a_tensor_past_2_32_bytes():
    import torch
    import laplace_prefix_scans_amd as lp
    n = (1 << 30) + 11
    p, g = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    lp.laplex_adamw([p], [g], [m], [v], step=1, lr=0.5)
    assert bool((p == p[0]).all()) and abs(float(p[0]) + 0.5) < 1e-6 and bool((m == m[0]).all()) and bool((v == v[0]).all())


@pytest.mark.parametrize("types", ["ff", "bb", "fb"])
@pytest.mark.parametrize("bits", [32, 8])
def test_parameters_larger_than_the_caches_as_in_parts(types, bits):
    """A step's result does not depend on how many bytes it moves: one call for all, and one for each part."""
    import torch
    import laplace_prefix_scans_amd as lp
    part, count = 5_000_192, 16 if types == "ff" else 24  # more than 288 MiB together, each part less
    g = torch.Generator(device="cuda").manual_seed(1)
    n = part * count - 100
    p = torch.randn(n, generator=g, device="cuda").to(dtypes(types[0]))
    grad = (1e-2 * torch.randn(n, generator=g, device="cuda")).to(dtypes(types[1]))
    kind = torch.float32 if bits == 32 else torch.uint8
    state = {k: torch.zeros(n, dtype=kind, device="cuda") for k in ("m", "v")}
    if bits == 8:
        state.update({k: torch.zeros(-(-n // 256), device="cuda") for k in ("m_scale", "v_scale")})
    else:
        state["m"].copy_(1e-3 * grad.float())
        state["v"].copy_(1e-3 * grad.float() ** 2)
    if types == "bb":
        state["master"] = p.float()
    q, other = p.clone(), {k: v.clone() for k, v in state.items()}
    for step in (1, 2):
        lp.laplex_adamw([p], [grad], step=step, weight_decay=0.1, **{k: [v] for k, v in state.items()}, **HYPER)
        for i in range(0, n, part):
            cut = {k: [v[i // 256:(i + part) // 256] if k.endswith("scale") and i + part < n else v[i // 256:] if k.endswith("scale") else v[i:i + part]]
                   for k, v in other.items()}
            lp.laplex_adamw([q[i:i + part]], [grad[i:i + part]], step=step, weight_decay=0.1, **cut, **HYPER)
        assert torch.equal(p, q) and all(torch.equal(v, other[k]) for k, v in state.items())
    if bits == 8:
        m, v = lp.laplex_adamw_moments(*[[state[k]] for k in ("m", "v", "m_scale", "v_scale")])
        small = lp.laplex_adamw_moments(*[[state[k][:1000]] for k in ("m", "v")], *[[state[k][:4]] for k in ("m_scale", "v_scale")])
        assert torch.equal(m[0][:1000], small[0][0]) and torch.equal(v[0][:1000], small[1][0])
