"""Layer norm and embedding on the GPU against float64.

Tolerances.  A sum of n float32 terms is off by about sqrt(n) 2^-24 of the
terms' magnitudes, taken eightfold for the largest of many elements; a result
formed from a few rounded factors adds 8 ulp; a bfloat16 result its rounding,
2^-9 (2^-8 allowed)."""
import numpy as np
import pytest

import layers_ref as ref
from gpu_util import have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

U = 2.0 ** -24


def dtypes():
    import torch
    return [torch.float32, torch.bfloat16]


def near(name, got, want, env, n, bf16=False):
    assert got.shape == want.shape and np.isfinite(got).all(), name
    tol = env * (8 * np.sqrt(n) + 16) * U + (np.abs(want) * 2.0 ** -8 if bf16 else 0.0) + 1e-30
    bad = np.abs(got - want) > tol
    assert not bad.any(), "%s: %d of %d off, worst %.3e of the tolerance" % (name, bad.sum(), bad.size,
                                                                           (np.abs(got - want) / tol).max())


# ------------------------------------------------------------------ layer norm
SHAPES = [(1, 1), (3, 2), (5, 63), (4, 64), (7, 65), (130, 256), (17, 1000), (8, 2048), (3, 4097), (2, 8192), (1, 20001), (700, 33),
          (2050, 8), (5, 16384), (1, 100003)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_layer_norm(shape, affine, dt):
    import torch
    import laplace_prefix_scans_amd as lp
    print("norm", shape, affine, dt, flush=True)
    rows, width = shape
    g = torch.Generator().manual_seed(rows + width)
    dtype = dtypes()[dt]
    x = (torch.randn(rows, width, generator=g) * 2 + 3).to(dtype)
    dy = torch.randn(rows, width, generator=g).to(dtype)
    w = (1 + 0.3 * torch.randn(width, generator=g)).to(dtype) if affine else None
    b = torch.randn(width, generator=g).to(dtype) if affine else None
    eps = 1e-5
    dev = [None if t is None else t.cuda() for t in (x, dy, w, b)]
    y, mean, rstd = lp.laplex_layer_norm(dev[0], dev[2], dev[3], eps=eps)
    f = [None if t is None else t.float().numpy() for t in (x, dy, w, b)]
    want_y, want_mean, want_rstd = ref.layer_norm(f[0], f[2], f[3], eps)
    big = np.abs(f[0]).astype(np.float64).max(1)  # the mean's error scales with it, and (over the row's deviation) everything after
    near("mean", host(mean), want_mean, big, width)
    sens = big * want_rstd  # how much a mean off by one part in `big` moves z
    near("rstd", host(rstd), want_rstd, want_rstd * (1 + sens), width)
    wmag = 1.0 if w is None else np.abs(f[2])
    z = np.abs((f[0].astype(np.float64) - want_mean[:, None]) * want_rstd[:, None])
    near("y", host(y.float()), want_y, wmag * (z + sens[:, None]) * (1 + z.max(1, keepdims=True)) + (0 if b is None else np.abs(f[3])),
         width, dt == 1)
    dx, dw, db = lp.laplex_layer_norm_backward(dev[0], dev[1], mean, rstd, dev[2])
    want_dx, want_dw, want_db, _ = ref.layer_norm_backward(f[0], f[1], f[2], eps)
    u = np.abs(f[1].astype(np.float64) * wmag)
    zz = z + sens[:, None]
    env = want_rstd[:, None] * (u + u.mean(1, keepdims=True) + zz * (u * zz).mean(1, keepdims=True)) * (1 + sens[:, None])
    near("dx", host(dx.float()), want_dx, env, width, dt == 1)
    near("dw", host(dw), want_dw, (np.abs(f[1]) * zz * (1 + sens[:, None])).sum(0), rows + width)
    near("db", host(db), want_db, np.abs(f[1]).astype(np.float64).sum(0), rows)


def test_layer_norm_gradient_against_differences():
    """<dy, y> along one direction of x, step h: central difference; truncation h^2/6 of the third derivative,
    estimated from the difference at twice the step."""
    import torch
    import laplace_prefix_scans_amd as lp
    g = torch.Generator().manual_seed(1)
    x, dy, e = (torch.randn(40, 200, generator=g).cuda() for _ in range(3))
    w, b = (1 + 0.3 * torch.randn(200, generator=g)).cuda(), torch.randn(200, generator=g).cuda()
    y, mean, rstd = lp.laplex_layer_norm(x, w, b)
    dx, dw, db = lp.laplex_layer_norm_backward(x, dy, mean, rstd, w)
    f = lambda t, ww=w, bb=b: (lp.laplex_layer_norm(t, ww, bb)[0].double() * dy.double()).sum()  # noqa: E731
    one = float(f(x + 2.0 ** -6 * e) - f(x - 2.0 ** -6 * e)) * 2 ** 5
    two = float(f(x + 2.0 ** -5 * e) - f(x - 2.0 ** -5 * e)) * 2 ** 4
    noise = 8 * U * float((y.double() * dy.double()).square().sum().sqrt()) * 2 ** 6 * 4
    assert abs(one - float((dx.double() * e.double()).sum())) <= abs(two - one) + noise
    ew = torch.randn(200, generator=g).cuda()
    noise = 64 * U * float((y.double().abs() * dy.double().abs()).sum())
    assert abs(float(f(x, w + ew) - f(x, w - ew)) / 2 - float((dw.double() * ew.double()).sum())) <= noise
    assert abs(float(f(x, w, b + ew) - f(x, w, b - ew)) / 2 - float((db.double() * ew.double()).sum())) <= noise


def test_layer_norm_rows_do_not_mix():
    import torch
    import laplace_prefix_scans_amd as lp
    for dtype in dtypes():
        g = torch.Generator().manual_seed(2)
        x = torch.randn(50, 513, generator=g).to(dtype).cuda()
        want = lp.laplex_layer_norm(x)[0]
        x[7, 100], x[20, 0], x[33] = float("inf"), float("nan"), 0.25
        y, mean, rstd = lp.laplex_layer_norm(x)
        keep = [i for i in range(50) if i not in (7, 20, 33)]
        assert torch.equal(y[keep], want[keep])
        assert not torch.isfinite(y[7]).any() and not torch.isfinite(y[20]).any()
        assert not y[33].any() and abs(float(rstd[33]) - 1e-5 ** -0.5) < 1e-3  # a constant row: variance 0


def test_layer_norm_unaligned_and_empty():
    import torch
    import laplace_prefix_scans_amd as lp
    for dtype in dtypes():
        for width in (64, 1000, 4096):
            buf = torch.randn(9 * width + 1, device="cuda").to(dtype)
            wb = torch.randn(2 * width + 1, device="cuda").to(dtype)
            x, w, b = buf[1:].view(9, width), wb[1:width + 1], wb[width + 1:]
            y, mean, rstd = lp.laplex_layer_norm(x, w, b)
            y2, mean2, rstd2 = lp.laplex_layer_norm(x.clone(), w.clone(), b.clone())
            near("y", host(y.float()), host(y2.float()).astype(np.float64), np.abs(host(y2.float())) + 20, width, dtype == torch.bfloat16)
            near("mean", host(mean), host(mean2).astype(np.float64), 1.0, width)
        x = torch.empty(0, 77, device="cuda", dtype=dtype)
        y, mean, rstd = lp.laplex_layer_norm(x)
        dx, dw, db = lp.laplex_layer_norm_backward(x, x, mean, rstd)
        assert y.shape == (0, 77) and dx.shape == (0, 77) and not dw.any() and not db.any()


def test_layer_norm_repeats_give_the_same_bits():
    import torch
    import laplace_prefix_scans_amd as lp
    for dtype in dtypes():
        x, dy = (torch.randn(3000, 700, device="cuda").to(dtype) for _ in range(2))
        y, mean, rstd = lp.laplex_layer_norm(x)
        a = lp.laplex_layer_norm_backward(x, dy, mean, rstd)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b = lp.laplex_layer_norm_backward(x, dy, mean, rstd)
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, b))


# ------------------------------------------------------------------ embedding
def ids_of(kind, tokens, vocab, seed):
    r = np.random.default_rng(seed)
    if kind == "same":
        return np.full(tokens, vocab // 2)
    if kind == "uniform":
        return r.integers(0, vocab, tokens)
    if kind == "outside":
        return r.choice(np.array([-1, vocab, -2 ** 31, 2 ** 31 - 1, 0, vocab - 1]), tokens)
    return np.minimum((np.exp(r.uniform(0, np.log(vocab + 1.0), tokens)) - 1).astype(np.int64), vocab - 1)


@pytest.mark.parametrize("shape", [(1, 1, 1), (5, 3, 7), (64, 257, 64), (1000, 10, 65), (3000, 5000, 129), (2049, 300, 512), (40, 70000, 33),
                                   (20000, 100, 24), (7, 1, 2000)], ids=str)
@pytest.mark.parametrize("kind", ["zipf", "uniform", "same", "outside"])
@pytest.mark.parametrize("dt", ["f32", "bf16", "bf16_f32"])
@pytest.mark.parametrize("wide", [False, True], ids=["i32", "i64"])
def test_embedding(shape, kind, dt, wide):
    import torch
    import laplace_prefix_scans_amd as lp
    tokens, vocab, width = shape
    print("embed", shape, kind, dt, wide, flush=True)
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    ids = ids_of(kind, tokens, vocab, tokens)
    g = torch.Generator().manual_seed(tokens)
    table, dy = torch.randn(vocab, width, generator=g).to(dtype), torch.randn(tokens, width, generator=g).to(dtype)
    ids_d = torch.from_numpy(ids).to(torch.int64 if wide else torch.int32).cuda()
    scale = 1.75
    y = host(lp.laplex_embedding(ids_d, table.cuda(), scale=scale).float())
    live = (ids >= 0) & (ids < vocab)
    want = np.where(live[:, None], scale * table.float().numpy().astype(np.float64)[np.where(live, ids, 0)], 0.0)
    near("y", y, want, np.abs(want), 1, dtype == torch.bfloat16)
    out = torch.float32 if dt == "bf16_f32" else dtype
    grad = lp.laplex_embedding_backward(ids_d, dy.cuda(), vocab, scale=scale, dtype=out)
    assert grad.dtype == out
    want = ref.embedding_backward(ids, dy.float().numpy(), vocab, scale)
    env = ref.embedding_backward(ids, np.abs(dy.float().numpy()), vocab, scale)
    near("dtable", host(grad.float()), want, env, tokens, out == torch.bfloat16)


@pytest.mark.parametrize("shape", [(16385, 300, 33), (40000, 1, 8), (70001, 5000, 40), (131072, 250000, 5), (131073, 4000, 17),
                                   (20000, 300000, 9)], ids=str)
@pytest.mark.parametrize("kind", ["zipf", "uniform", "same", "outside"])
def test_embedding_gradient_of_many_tokens(shape, kind):
    """Tokens that are sorted in tiles, a whole and a broken last tile, and more or larger ids than tiles are for."""
    import torch
    import laplace_prefix_scans_amd as lp
    tokens, vocab, width = shape
    print("embed many", shape, kind, flush=True)
    ids = ids_of(kind, tokens, vocab, tokens)
    dy = torch.randn(tokens, width, generator=torch.Generator().manual_seed(tokens))
    grad = lp.laplex_embedding_backward(torch.from_numpy(ids).to(torch.int64).cuda(), dy.cuda(), vocab, scale=0.5)
    want = ref.embedding_backward(ids, dy.numpy(), vocab, 0.5)
    near("dtable", host(grad), want, ref.embedding_backward(ids, np.abs(dy.numpy()), vocab, 0.5), tokens)


@pytest.mark.parametrize("width", [641, 1283, 2600, 5003])
@pytest.mark.parametrize("dt", ["f32", "bf16", "bf16_f32"])
def test_embedding_of_long_odd_rows(width, dt):
    """Rows that are no whole number of aligned pieces, by width and by address."""
    import torch
    import laplace_prefix_scans_amd as lp
    tokens, vocab = 300, 40
    print("embed odd", width, dt, flush=True)
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(width)
    buf = torch.randn(1 + (tokens + vocab) * width, generator=g).to(dtype)
    ids = ids_of("zipf", tokens, vocab + 1, width)
    dev = buf.cuda()
    table, dy = (b[1:1 + vocab * width].view(vocab, width) for b in (buf, dev)), (b[1 + vocab * width:].view(tokens, width) for b in (buf, dev))
    (table, table_d), (dy, dy_d) = table, dy
    ids_d = torch.from_numpy(ids).cuda()
    live = ids < vocab
    want = np.where(live[:, None], 2.5 * table.float().numpy().astype(np.float64)[np.where(live, ids, 0)], 0.0)
    near("y", host(lp.laplex_embedding(ids_d, table_d, scale=2.5).float()), want, np.abs(want), 1, dtype == torch.bfloat16)
    out = torch.float32 if dt == "bf16_f32" else dtype
    grad = lp.laplex_embedding_backward(ids_d, dy_d, vocab, scale=2.5, dtype=out)
    want = ref.embedding_backward(ids, dy.float().numpy(), vocab, 2.5)
    near("dtable", host(grad.float()), want, ref.embedding_backward(ids, np.abs(dy.float().numpy()), vocab, 2.5), tokens, out == torch.bfloat16)


def test_embedding_gradient_against_differences():
    """<dy, y> is linear in the table: a difference with a step of 1 has rounding errors only."""
    import torch
    import laplace_prefix_scans_amd as lp
    g = torch.Generator().manual_seed(3)
    ids = torch.randint(0, 50, (600,), generator=g).cuda()
    table, e = torch.randn(50, 40, generator=g).cuda(), torch.randn(50, 40, generator=g).cuda()
    dy = torch.randn(600, 40, generator=g).cuda()
    f = lambda t: (lp.laplex_embedding(ids, t, scale=3.0).double() * dy.double()).sum()  # noqa: E731
    grad = lp.laplex_embedding_backward(ids, dy, 50, scale=3.0)
    size = 3.0 * float(((table.abs() + e.abs())[ids].double() * dy.double().abs()).sum())
    assert abs(float(f(table + e) - f(table - e)) / 2 - float((grad.double() * e.double()).sum())) <= 32 * U * size


def test_embedding_shapes_repeats_and_empty():
    import torch
    import laplace_prefix_scans_amd as lp
    for dtype in dtypes():
        ids = torch.randint(-1, 90, (4, 700), device="cuda")
        table = torch.randn(90, 48, device="cuda").to(dtype)
        y = lp.laplex_embedding(ids, table)
        assert y.shape == (4, 700, 48)
        assert torch.equal(y.view(-1, 48), lp.laplex_embedding(ids.view(-1), table))
        dy = torch.randn(4, 700, 48, device="cuda").to(dtype)
        a, b = lp.laplex_embedding_backward(ids, dy, 90), lp.laplex_embedding_backward(ids.to(torch.int32), dy, 90)
        assert torch.equal(a, b)
        # unaligned rows
        buf = torch.randn(2800 * 48 + 1, device="cuda").to(dtype)
        u = buf[1:].view(4, 700, 48)
        assert torch.equal(lp.laplex_embedding_backward(ids, u, 90), lp.laplex_embedding_backward(ids, u.clone(), 90))
        none = torch.empty(0, dtype=torch.int64, device="cuda")
        assert lp.laplex_embedding(none, table).shape == (0, 48)
        z = lp.laplex_embedding_backward(none, torch.empty(0, 48, device="cuda", dtype=dtype), 90)
        assert z.shape == (90, 48) and not z.any()
        # non-finite gradients stay in their row
        ids = torch.arange(90, device="cuda")
        dy = torch.ones(90, 48, device="cuda", dtype=dtype)
        dy[13] = float("nan")
        dy[14, 0] = float("inf")
        grad = lp.laplex_embedding_backward(ids, dy, 90)
        assert torch.isnan(grad[13]).all() and torch.isinf(grad[14, 0]) and torch.isfinite(grad[15:]).all() and torch.isfinite(grad[:13]).all()


# ------------------------------------------------------------------ under a graph
def test_layers_under_a_graph():
    """Capture of every entry point; replays with eager work in between give the eager result each time."""
    import torch
    import laplace_prefix_scans_amd as lp
    torch.manual_seed(4)
    q, k, v, go = (torch.randn(700, 2, 64, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    rate = torch.tensor([0.02, 0.3], device="cuda")
    off = torch.tensor([0, 300, 700], dtype=torch.int32, device="cuda")
    ids = torch.randint(0, 200, (700,), device="cuda")
    table = torch.randn(200, 128, device="cuda", dtype=torch.bfloat16)
    state = torch.zeros(700, 2, 64, 64, device="cuda")

    def work():
        x = lp.laplex_embedding(ids, table)
        y, mean, rstd = lp.laplex_layer_norm(x)
        o = lp.laplex_decay_attn(q, k, v, rate, offsets=off)
        s = lp.laplex_decay_attn_step(q, k, v, rate, state)
        g = lp.laplex_decay_attn_backward(q, k, v, rate, go, offsets=off)
        return (x, y, o, s) + g[:4] + lp.laplex_layer_norm_backward(x, y, mean, rstd) + (lp.laplex_embedding_backward(ids, x, 200),)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for i in range(4):
        ids.copy_(torch.randint(0, 200, (700,), device="cuda"))
        q.copy_(torch.randn(700, 2, 64, device="cuda").bfloat16())
        state.zero_()
        want = [t.clone() for t in work()]
        torch.cuda.synchronize()
        state.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i
