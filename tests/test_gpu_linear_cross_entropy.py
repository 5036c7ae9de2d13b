"""Linear softmax cross entropy on the GPU against float64.  Tolerances: train_ref.cross_entropy follows the errors of the
logits through the softmax and the products; bfloat16 results add half a step, 2^-8 of the value."""
import numpy as np
import pytest

import train_ref as ref
from gpu_util import have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


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


def make(tokens, vocab, width, dtype, seed=0, ids=None, spread=2.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    ids = torch.int64 if ids is None else ids
    y = torch.randint(0, vocab, (tokens,), generator=g)
    table = (spread * width ** -0.5 * normal(vocab, width)).to(dtype)
    # some rows lean towards their targets, so that some are nearly certain
    x = (normal(tokens, width) + torch.rand(tokens, 1, generator=g) * 5 * table[y].float()).to(dtype)
    y = y.to(ids)
    if tokens > 2:  # left out: padding, the end of the vocabulary, far outside
        y[1] = -1
        y[tokens // 2] = vocab
        y[-1] = torch.iinfo(ids).min
    return {"x": x, "table": table, "y": y, "dloss": normal(tokens), "dlse": normal(tokens)}


def run_case(tokens, vocab, width, dt, seed=0, ids=None, scale=1.0, dlse=False, table_dtype=None, spread=2.0):
    import torch
    import laplace_prefix_scans_amd as lp
    print("cross entropy tokens=%d vocab=%d width=%d %s" % (tokens, vocab, width, dt), flush=True)
    dtype = dtype_of(dt)
    x = make(tokens, vocab, width, dtype, seed, ids, spread)
    c = {k: v.cuda() for k, v in x.items()}
    loss, lse = lp.laplex_linear_cross_entropy(c["x"], c["table"], c["y"], scale=scale)
    dx, dt_ = lp.laplex_linear_cross_entropy_backward(c["x"], c["table"], c["y"], lse, c["dloss"], c["dlse"] if dlse else None, scale=scale,
                                                      dtype=table_dtype)
    npf = {k: v.float().numpy() if v.is_floating_point() else v.numpy() for k, v in x.items()}
    want = ref.cross_entropy(npf["x"], npf["table"], npf["y"], scale, npf["dloss"], npf["dlse"] if dlse else None, dt == "bf16")
    assert loss.dtype == lse.dtype == torch.float32 and dx.dtype == dtype and dt_.dtype == (table_dtype or dtype)
    check("lse", lse, want["lse"], want["~lse"], False)
    check("loss", loss, want["loss"], want["~loss"], False)
    check("dx", dx, want["dx"], want["~dx"], dt == "bf16")
    check("dtable", dt_, want["dtable"], want["~dtable"], dt == "bf16")
    return c, lse, dx, dt_


@pytest.mark.parametrize("tokens", [1, 2, 3, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 300])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_tokens(tokens, dt):
    run_case(tokens, 200, 96, dt, seed=tokens)


@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 32, 63, 64, 65, 128, 129, 255, 256, 257, 1000, 4099])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_vocabularies(vocab, dt):
    run_case(70, vocab, 64, dt, seed=vocab)


@pytest.mark.parametrize("width", [1, 2, 7, 8, 31, 32, 33, 64, 100, 128, 129, 200, 256, 513, 1024])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_widths(width, dt):
    run_case(80, 150, width, dt, seed=width)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_many_tiles_of_everything(dt):
    run_case(700, 3001, 320, dt, seed=5)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("ids", ["int32", "int64"])
def test_types_scale_and_the_gradient_of_lse(dt, ids):
    import torch
    run_case(90, 300, 72, dt, ids=getattr(torch, ids), scale=0.3, dlse=True, table_dtype=torch.float32)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_wide_logits(dt):
    run_case(100, 500, 128, dt, scale=-1.7, spread=20.0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_one_gradient_alone(dt):
    import torch
    import laplace_prefix_scans_amd as lp
    c, lse, dx, dtable = run_case(130, 260, 64, dt)
    a = (c["x"], c["table"], c["y"], lse, c["dloss"])
    p, q = lp.laplex_linear_cross_entropy_backward(*a, table_grad=False)
    assert torch.equal(p, dx) and q is None
    p, q = lp.laplex_linear_cross_entropy_backward(*a, x_grad=False)
    assert p is None and torch.equal(q, dtable)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_tokens_left_out_take_no_part_whatever_they_hold(dt):
    import torch
    import laplace_prefix_scans_amd as lp
    c, lse, dx, dtable = run_case(200, 300, 80, dt, seed=3)
    out = (c["y"] < 0) | (c["y"] >= 300)
    assert out.sum() == 3
    for bad in (float("nan"), float("inf"), 3e38):
        x, w = c["x"].clone(), c["dloss"].clone()
        x[out] = bad
        w[out] = float("nan")
        loss2, lse2 = lp.laplex_linear_cross_entropy(x, c["table"], c["y"])
        assert (loss2[out] == 0).all() and (lse2[out] == 0).all() and torch.equal(lse2, lse)
        lse2[out] = float("nan")
        dx2, dt2 = lp.laplex_linear_cross_entropy_backward(x, c["table"], c["y"], lse2, w)
        assert torch.equal(dx2, dx) and torch.equal(dt2, dtable) and (dx2[out] == 0).all()
    # none is left
    y = torch.full_like(c["y"], -1)
    loss, lse = lp.laplex_linear_cross_entropy(c["x"], c["table"], y)
    dx, dtable = lp.laplex_linear_cross_entropy_backward(c["x"], c["table"], y, lse, c["dloss"])
    assert not loss.any() and not lse.any() and not dx.any() and not dtable.any()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_a_table_row_of_infinities_leaves_tokens_left_out_alone(dt):
    import torch
    import laplace_prefix_scans_amd as lp
    x = {k: v.cuda() for k, v in make(40, 70, 64, dtype_of(dt)).items()}
    x["table"][5] = float("inf")
    loss, lse = lp.laplex_linear_cross_entropy(x["x"], x["table"], x["y"])
    out = (x["y"] < 0) | (x["y"] >= 70)
    dx, _ = lp.laplex_linear_cross_entropy_backward(x["x"], x["table"], x["y"], lse, x["dloss"])
    assert (loss[out] == 0).all() and (dx[out] == 0).all()


def test_infinite_and_undefined_logits():
    import torch
    import laplace_prefix_scans_amd as lp
    inf, nan = float("inf"), float("nan")
    table = torch.ones(3, 1, device="cuda")
    table[:, 0] = torch.tensor([1.0, 2.0, -3.0])
    x = torch.tensor([[inf], [-inf], [nan], [0.0], [1e38], [-1e38]], device="cuda")
    for y in (0, 1, 2):
        t = torch.full((6,), y, device="cuda")
        loss, lse = lp.laplex_linear_cross_entropy(x, table, t)
        logits = x.double() @ table.double().t()
        want_lse = torch.logsumexp(logits.float(), 1)  # in float the last rows' logits still are finite
        want = want_lse - logits.float()[:, y]
        assert torch.equal(torch.isnan(lse), torch.isnan(want_lse)) and torch.equal(torch.isnan(loss), torch.isnan(want))
        fine = ~torch.isnan(want_lse)
        assert torch.allclose(lse[fine], want_lse[fine], rtol=1e-6)
        fine = ~torch.isnan(want)
        assert torch.allclose(loss[fine], want[fine], rtol=1e-6)
    # logits of minus infinity alone
    table = torch.full((200, 1), -inf, device="cuda")
    loss, lse = lp.laplex_linear_cross_entropy(torch.ones(2, 1, device="cuda"), table, torch.tensor([0, 150], device="cuda"))
    assert (lse == -inf).all() and torch.isnan(loss).all()
    table[133] = 2.0
    loss, lse = lp.laplex_linear_cross_entropy(torch.ones(2, 1, device="cuda"), table, torch.tensor([133, 150], device="cuda"))
    assert (lse == 2.0).all() and loss[0] == 0.0 and loss[1] == inf


def test_gradients_against_differences():
    import torch
    import laplace_prefix_scans_amd as lp
    x = make(6, 9, 4, torch.float32, seed=2)
    c = {k: v.cuda() for k, v in x.items()}
    _, lse = lp.laplex_linear_cross_entropy(c["x"], c["table"], c["y"], scale=0.7)
    got = lp.laplex_linear_cross_entropy_backward(c["x"], c["table"], c["y"], lse, c["dloss"], c["dlse"], scale=0.7)
    n = {k: v.numpy().astype(np.float64) if v.is_floating_point() else v.numpy() for k, v in x.items()}

    def value():
        r = ref.cross_entropy(n["x"], n["table"], n["y"], 0.7)
        return (r["loss"] * n["dloss"]).sum() + (r["lse"] * n["dlse"]).sum()
    for name, g in zip(("x", "table"), got):
        for at in np.ndindex(n[name].shape):
            keep, step = n[name][at], 1e-5
            n[name][at] = keep + step
            up = value()
            n[name][at] = keep - step
            down = value()
            n[name][at] = keep
            # central differences: third derivatives of order 100 times step^2, cancellation of 100 2^-53 / step
            assert abs(float(g[at]) - (up - down) / (2 * step)) < 1e-5 * (1 + abs(float(g[at]))), (name, at)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_alignment(dt):
    """Rows that begin anywhere: the same bits."""
    import torch
    import laplace_prefix_scans_amd as lp
    c = {k: v.cuda() for k, v in make(70, 90, 128, dtype_of(dt)).items()}
    _, lse = lp.laplex_linear_cross_entropy(c["x"], c["table"], c["y"])
    want = lp.laplex_linear_cross_entropy_backward(c["x"], c["table"], c["y"], lse, c["dloss"])

    def moved(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:]
        return flat.copy_(t.reshape(-1)).view(t.shape)
    x, table = moved(c["x"]), moved(c["table"])
    _, lse2 = lp.laplex_linear_cross_entropy(x, table, c["y"])
    got = lp.laplex_linear_cross_entropy_backward(x, table, c["y"], lse2, c["dloss"])
    assert torch.equal(lse, lse2) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_workspaces_serve_fewer_tokens(dt):
    import torch
    import laplace_prefix_scans_amd as lp
    c = {k: v.cuda() for k, v in make(400, 333, 96, dtype_of(dt)).items()}
    a = lambda t: (c["x"][:t], c["table"], c["y"][:t])  # noqa: E731
    size = lambda b, t: lp.laplex_linear_cross_entropy_workspace_bytes(b, *a(t))  # noqa: E731
    assert size(False, 1) <= size(False, 399) <= size(False, 400) and size(True, 1) <= size(True, 399) <= size(True, 400)
    for t in (400, 399, 130, 1):
        ws = [torch.full((size(b, 400),), 255, dtype=torch.uint8, device="cuda") for b in (False, True)]
        loss, lse = lp.laplex_linear_cross_entropy(*a(t))
        loss2, lse2 = lp.laplex_linear_cross_entropy(*a(t), ws=ws[0])
        assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
        for p, q in zip(lp.laplex_linear_cross_entropy_backward(*a(t), lse, c["dloss"][:t]),
                        lp.laplex_linear_cross_entropy_backward(*a(t), lse, c["dloss"][:t], ws=ws[1])):
            assert torch.equal(p, q)


def test_several_pieces_of_the_vocabulary():
    """Tokens and vocabulary whose gradient of the logits is formed in pieces: against float64 on the GPU."""
    import torch
    import laplace_prefix_scans_amd as lp
    tokens, vocab, width = 6000, 50001, 72
    x = {k: v.cuda() for k, v in make(tokens, vocab, width, torch.bfloat16, seed=1).items()}
    _, lse = lp.laplex_linear_cross_entropy(x["x"], x["table"], x["y"])
    dx, dtable = lp.laplex_linear_cross_entropy_backward(x["x"], x["table"], x["y"], lse, x["dloss"], dtype=torch.float32)
    inside = (x["y"] >= 0) & (x["y"] < vocab)
    logits = x["x"].double() @ x["table"].double().t()
    want = torch.logsumexp(logits, 1)
    assert ((lse.double() - want)[inside].abs() < 2e-5).all()
    d = torch.where(inside, x["dloss"], 0.0).double()[:, None]
    p = torch.softmax(logits, 1) * d
    # p exp's factors are off by the errors of a logit (train_ref.cross_entropy) and of the lse (2e-5, above): where a target is
    # nearly certain, p - 1 is a difference of nearly equal numbers, and this is many times 2^-8 of it
    e = p.abs() * (72.0 ** 0.5 * 8 + 4) * ref.U * (x["x"].double().abs() @ x["table"].double().abs().t())
    e += p.abs() * (2e-5 + 3 * ref.U * (logits - want[:, None]).abs() + 8 * ref.U)
    p[torch.arange(tokens, device="cuda"), x["y"].clamp(0, vocab - 1)] -= d[:, 0]
    # rounding of the factor (2^-8 of each term), of float32 sums (8 sqrt(n) roundings) and of the result
    e += 2.0 ** -8 * p.abs()
    for got, w, off, size, n in ((dx, p @ x["table"].double(), e @ x["table"].double().abs(), p.abs() @ x["table"].double().abs(), vocab),
                                 (dtable, p.t() @ x["x"].double(), e.t() @ x["x"].double().abs(), p.abs().t() @ x["x"].double().abs(), tokens)):
        assert ((got.double() - w).abs() <= 2.0 ** -8 * w.abs() + off + 8 * n ** 0.5 * ref.U * size + 1e-30).all()


def test_shapes_no_tokens_and_streams():
    import torch
    import laplace_prefix_scans_amd as lp
    x = {k: v.cuda() for k, v in make(60, 90, 32, torch.float32).items()}
    loss, lse = lp.laplex_linear_cross_entropy(x["x"], x["table"], x["y"])
    y3, x3 = x["y"].view(3, 4, 5), x["x"].view(3, 4, 5, 32)
    loss3, lse3 = lp.laplex_linear_cross_entropy(x3, x["table"], y3)
    assert loss3.shape == (3, 4, 5) and torch.equal(loss3.view(-1), loss)
    dx3, dt3 = lp.laplex_linear_cross_entropy_backward(x3, x["table"], y3, lse3, x["dloss"].view(3, 4, 5))
    dx, dt = lp.laplex_linear_cross_entropy_backward(x["x"], x["table"], x["y"], lse, x["dloss"])
    assert torch.equal(dx3.view(-1, 32), dx) and torch.equal(dt3, dt)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        l2, _ = lp.laplex_linear_cross_entropy(x["x"], x["table"], x["y"])
        l2.record_stream(s)
    s.synchronize()
    assert torch.equal(l2, loss)
    e, ye, f = x["x"][:0], x["y"][:0], torch.empty(0, device="cuda")
    assert lp.laplex_linear_cross_entropy(e, x["table"], ye)[0].shape == (0,)
    dx, dt = lp.laplex_linear_cross_entropy_backward(e, x["table"], ye, f, f)
    assert dx.shape == (0, 32) and dt.shape == (90, 32) and not dt.any()


# ------------------------------------------------------------------ a few tokens
@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 5, 7, 8, 9])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_few_tokens(tokens, dt):
    run_case(tokens, 2003, 520, dt, seed=tokens)


# rows of less than a load of a wave, of whole loads, with ends of every kind; tokens that fill 128 KB, and one element more
@pytest.mark.parametrize("tokens,width", [(t, w) for t in (2, 4) for w in (1, 3, 64, 255, 256, 257, 511, 512, 513, 4096, 4097, 8191, 8193, 16383, 16384, 16385)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_few_tokens_of_any_width(tokens, width, dt):
    run_case(tokens, 77, width, dt, seed=width)


@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 63, 65, 33000])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_few_tokens_of_any_vocabulary(vocab, dt):
    import torch
    run_case(4, vocab, 40, dt, seed=vocab, ids=torch.int32, scale=-0.7, dlse=True)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_few_tokens_that_begin_anywhere(dt):
    import torch
    import laplace_prefix_scans_amd as lp
    for tokens, width in ((2, 128), (2, 1024), (4, 1024), (4, 1001)):
        c = {k: v.cuda() for k, v in make(tokens, 90, width, dtype_of(dt)).items()}
        loss, lse = lp.laplex_linear_cross_entropy(c["x"], c["table"], c["y"])

        def moved(t):
            flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:]
            return flat.copy_(t.reshape(-1)).view(t.shape)
        loss2, lse2 = lp.laplex_linear_cross_entropy(moved(c["x"]), moved(c["table"]), c["y"])
        assert torch.equal(lse, lse2) and torch.equal(loss, loss2)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [4, 20])
def test_a_token_has_nothing_of_its_neighbours(tokens, dt):
    """A token's loss and lse have the same bits whatever the others hold, infinities and huge logits among them."""
    import torch
    import laplace_prefix_scans_amd as lp
    c = {k: v.cuda() for k, v in make(tokens, 300, 200, dtype_of(dt)).items()}
    y = c["y"].clamp(0, 299)
    loss, lse = lp.laplex_linear_cross_entropy(c["x"], c["table"], y)
    for bad in (float("inf"), float("nan"), 1e30):
        x = c["x"].clone()
        x[1::2] = bad
        loss2, lse2 = lp.laplex_linear_cross_entropy(x, c["table"], y)
        assert torch.equal(loss2[::2], loss[::2]) and torch.equal(lse2[::2], lse[::2]), bad


# ------------------------------------------------------------------ more tiles than run at once
# Each tile shape of each product, with a second round of tiles for its blocks, and split sums among them
@pytest.mark.parametrize("dims", [(33, 3001, 1500), (33, 9001, 640), (33, 20001, 1500), (33, 40001, 640), (100, 40001, 33), (200, 20001, 40),
                                  (500, 40001, 72), (700, 40001, 32), (700, 3001, 1500), (3001, 100, 1500)], ids=str)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_more_tiles_than_run_at_once(dims, dt):
    run_case(*dims, dt, seed=2)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dims", [(3, 1000, 256), (300, 9001, 640)], ids=str)
def test_a_repeated_call_gives_the_same_bits(dims, dt):
    import torch
    import laplace_prefix_scans_amd as lp
    c = {k: v.cuda() for k, v in make(*dims, dtype_of(dt)).items()}

    def both():
        loss, lse = lp.laplex_linear_cross_entropy(c["x"], c["table"], c["y"])
        return (loss, lse, *lp.laplex_linear_cross_entropy_backward(c["x"], c["table"], c["y"], lse, c["dloss"], c["dlse"]))
    first = both()
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(both(), first))


# ------------------------------------------------------------------ the gradient's factor in two parts
@pytest.mark.parametrize("dims", [(1, 300, 100), (11, 227, 2696), (64, 65, 64), (100, 9001, 72), (512, 700, 130), (2048, 300, 72)], ids=str)
def test_gradients_of_few_tokens_are_off_by_their_own_rounding(dims):
    """In bfloat16: the factor G is held in two parts, whose second is off by half a step (2^-8) of what the first left
    out (2^-8 of G at most): 2^-16 of G, 2^-8 of what train_ref.cross_entropy allows for one part."""
    import torch
    import laplace_prefix_scans_amd as lp
    x = make(*dims, torch.bfloat16, seed=7)
    c = {k: v.cuda() for k, v in x.items()}
    _, lse = lp.laplex_linear_cross_entropy(c["x"], c["table"], c["y"])
    dx, dtable = lp.laplex_linear_cross_entropy_backward(c["x"], c["table"], c["y"], lse, c["dloss"], c["dlse"])
    npf = {k: v.float().numpy() if v.is_floating_point() else v.numpy() for k, v in x.items()}
    one, none = (ref.cross_entropy(npf["x"], npf["table"], npf["y"], 1.0, npf["dloss"], npf["dlse"], b) for b in (True, False))
    for name, got in (("dx", dx), ("dtable", dtable)):
        exact = none["~" + name]
        check(name, got, none[name], exact + 2.0 ** -8 * (one["~" + name] - exact), True)


def test_two_parts_of_a_vocabulary_in_pieces():
    """Two parts, and a vocabulary of two pieces: against float64 on the GPU."""
    import torch
    import laplace_prefix_scans_amd as lp
    tokens, vocab, width = 512, 270001, 8
    x = {k: v.cuda() for k, v in make(tokens, vocab, width, torch.bfloat16, seed=1).items()}
    _, lse = lp.laplex_linear_cross_entropy(x["x"], x["table"], x["y"])
    dx, dtable = lp.laplex_linear_cross_entropy_backward(x["x"], x["table"], x["y"], lse, x["dloss"], dtype=torch.float32)
    inside = (x["y"] >= 0) & (x["y"] < vocab)
    logits = x["x"].double() @ x["table"].double().t()
    want = torch.logsumexp(logits, 1)
    assert ((lse.double() - want)[inside].abs() < 2e-5).all()
    d = torch.where(inside, x["dloss"], 0.0).double()[:, None]
    p = torch.softmax(logits, 1) * d
    # errors of a logit, of the lse (2e-5, above) and of the exponential, as in train_ref.cross_entropy
    e = p.abs() * ((8.0 ** 0.5 * 8 + 4) * ref.U * (x["x"].double().abs() @ x["table"].double().abs().t()) + 2e-5 + 8 * ref.U
                   + 3 * ref.U * (logits - want[:, None]).abs())
    p[torch.arange(tokens, device="cuda"), x["y"].clamp(0, vocab - 1)] -= d[:, 0]
    e += (2.0 ** -16 + 2 * ref.U) * p.abs()
    for got, half, w, off, size, n in ((dx, 2.0 ** -8, p @ x["table"].double(), e @ x["table"].double().abs(), p.abs() @ x["table"].double().abs(), vocab),
                                       (dtable, 2.0 ** -24, p.t() @ x["x"].double(), e.t() @ x["x"].double().abs(), p.abs().t() @ x["x"].double().abs(), tokens)):
        assert ((got.double() - w).abs() <= half * w.abs() + off + 8 * n ** 0.5 * ref.U * size + 1e-30).all()
