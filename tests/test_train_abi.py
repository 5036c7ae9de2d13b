"""The training-step operators' entry points reject bad arguments on the host (no GPU work is started: every call fails a
check, or has nothing to do, before a launch), the binding rejects tensors of the wrong kind, and workspaces grow with
the tokens."""
import ctypes
import os

import pytest

OK, NULL, SIZE, ALIGN, WS, OVERLAP, ARG = 0, 1, 2, 3, 4, 7, 9
vp = ctypes.c_void_p
MB = 1 << 20


def at(mb, off=0):
    return vp(mb * MB + off)  # never dereferenced


@pytest.fixture(scope="module")
def L():
    import laplace_prefix_scans_amd as lp
    from laplace_prefix_scans_amd import _training
    if not os.path.exists(lp.lib_path()):
        pytest.skip("liblaplex.so not built")
    return _training._lib()


def shape(**over):
    from laplace_prefix_scans_amd._training import _Scan
    s = _Scan(0, 0, 2, 64, 100, None, 64, 64)
    for k, v in over.items():
        setattr(s, k, v)
    return ctypes.byref(s)


def scan(L, s, g=at(10), x=at(20), si=None, so=None, h=at(30), c=None, ws=at(100), wb=64 * MB):
    return L.laplex_gated_scan(s, g, x, si, so, h, c, ws, wb, None)


def back(L, s, g=at(10), x=at(20), c=at(25), dh=at(30), si=None, dso=None, dg=at(40), dx=at(50), dsi=None, ws=at(100), wb=64 * MB):
    return L.laplex_gated_scan_backward(s, g, x, c, dh, si, dso, dg, dx, dsi, ws, wb, None)


@pytest.mark.parametrize("call", [scan, back])
def test_scan_shapes(L, call):
    assert call(L, None) == NULL
    assert call(L, shape(dtype=2)) == ARG and call(L, shape(gate=2)) == ARG and call(L, shape(channels=0)) == ARG
    assert call(L, shape(tokens=1 << 31)) == SIZE and call(L, shape(seqs=(1 << 20) + 1)) == SIZE and call(L, shape(channels=(1 << 24) + 1)) == SIZE
    assert call(L, shape(tokens=101)) == ARG  # equal lengths do not divide
    assert call(L, shape(seqs=0)) == ARG      # tokens of no sequence
    assert call(L, shape(gate_token=-1)) == ARG and call(L, shape(x_token=1 << 62)) == ARG
    assert call(L, shape(seqs=0, tokens=0)) == OK and call(L, shape(tokens=0)) == OK


def test_scan_pointers(L):
    assert scan(L, shape(), g=None) == NULL and scan(L, shape(), h=None) == NULL
    assert scan(L, shape(), x=at(20, 2)) == ALIGN and scan(L, shape(dtype=1), h=at(30, 1)) == ALIGN
    assert scan(L, shape(), si=at(60, 2)) == ALIGN and scan(L, shape(offsets=at(5, 1).value)) == ALIGN
    assert scan(L, shape(), h=at(10, 64)) == OVERLAP and scan(L, shape(), si=at(60), so=at(60)) == OVERLAP
    assert scan(L, shape(), c=at(30)) == OVERLAP and scan(L, shape(offsets=at(30).value)) == OVERLAP
    big = dict(tokens=100000, seqs=1)
    need = L.laplex_gated_scan_workspace_bytes(shape(**big))
    assert need > 0 and need % 256 == 0
    far = dict(g=at(1000), x=at(2000), h=at(3000), wb=need)
    assert scan(L, shape(**big), **{**far, "ws": None}) == NULL
    assert scan(L, shape(**big), **{**far, "ws": at(100, 128)}) == ALIGN
    assert scan(L, shape(**big), **{**far, "wb": need - 1}) == WS
    assert scan(L, shape(**big), **{**far, "ws": at(3000)}) == OVERLAP
    for name in ("c", "dh", "dg", "dx"):
        assert back(L, shape(), **{name: None}) == NULL
    assert back(L, shape(), dg=at(50)) == OVERLAP and back(L, shape(), dx=at(30)) == OVERLAP and back(L, shape(), dsi=at(25)) == OVERLAP
    assert back(L, shape(), dso=at(60), dsi=at(60, 16)) == OVERLAP and back(L, shape(), dh=at(30, 2)) == ALIGN


def test_scan_step(L):
    def step(s, g=at(10), x=at(20), slots=at(35), pool=8, state=at(40), h=at(50)):
        return L.laplex_gated_scan_step(s, g, x, slots, pool, state, h, None)
    one = dict(seqs=5, tokens=5)
    assert step(shape(seqs=5, tokens=6)) == ARG and step(shape(**one), slots=None, pool=4) == ARG
    assert step(shape(**one), g=None) == NULL and step(shape(**one), state=None) == NULL
    assert step(shape(**one), slots=at(35, 2)) == ALIGN and step(shape(**one), state=at(40, 2)) == ALIGN
    assert step(shape(**one), h=at(40, 64)) == OVERLAP and step(shape(**one), x=at(40)) == OVERLAP
    assert step(shape(seqs=1 << 20, tokens=1 << 20, channels=1 << 20)) == SIZE
    assert step(shape(seqs=0, tokens=0), g=None, state=None) == OK


def test_scan_workspaces_serve_fewer_tokens(L):
    for dtype in (0, 1):
        for channels in (1, 64, 65, 128, 1001, 4096, 300000):
            last = 0
            for tokens in list(range(0, 3000)) + list(range(3000, 300000, 517)) + [1 << 24, (1 << 31) - 1]:
                need = L.laplex_gated_scan_workspace_bytes(shape(dtype=dtype, channels=channels, tokens=tokens))
                assert need >= last, (channels, tokens)
                last = need
    assert L.laplex_gated_scan_workspace_bytes(shape(channels=0)) == 0


def test_cross_entropy(L):
    def loss(dt=0, y=at(5), nb=8, t=16, x=at(10), w=at(20), vocab=100, width=32, out=at(30), lse=at(31), ws=at(100), wb=64 * MB):
        return L.laplex_linear_cross_entropy(dt, y, nb, t, x, w, vocab, width, 1.0, out, lse, ws, wb, None)

    def grad(dt=0, y=at(5), nb=8, t=16, x=at(10), w=at(20), vocab=100, width=32, lse=at(31), d=at(32), de=None, dx=at(40), td=0, dw=at(50),
             ws=at(100), wb=256 * MB):
        return L.laplex_linear_cross_entropy_backward(dt, y, nb, t, x, w, vocab, width, 1.0, lse, d, de, dx, td, dw, ws, wb, None)
    for f in (loss, grad):
        assert f(dt=2) == ARG and f(nb=2) == ARG and f(width=0) == ARG and f(vocab=0) == ARG
        assert f(t=(1 << 28) + 1) == SIZE and f(vocab=(1 << 26) + 1) == SIZE and f(width=(1 << 24) + 1) == SIZE
        assert f(t=1 << 24, vocab=1 << 20) == SIZE
        assert f(y=None) == NULL and f(x=None) == NULL and f(w=None) == NULL and f(ws=None) == NULL
        assert f(y=at(5, 4)) == ALIGN and f(x=at(10, 2)) == ALIGN and f(w=at(20, 1)) == ALIGN and f(ws=at(100, 16)) == ALIGN
        assert f(wb=256) == WS
    assert loss(t=0, y=None) == OK and loss(out=None, lse=None) == NULL
    assert loss(out=at(31)) == OVERLAP and loss(lse=at(10)) == OVERLAP and loss(out=at(100)) == OVERLAP and loss(out=at(5)) == OVERLAP
    assert grad(dx=None, dw=None) == OK and grad(td=1) == ARG and grad(dt=1, td=2) == ARG
    assert grad(lse=None) == NULL and grad(d=None) == NULL and grad(d=at(32, 2)) == ALIGN and grad(dw=at(50, 2)) == ALIGN
    assert grad(dx=at(50)) == OVERLAP and grad(dw=at(20)) == OVERLAP and grad(dx=at(32)) == OVERLAP and grad(de=at(40)) == OVERLAP
    size = L.laplex_linear_cross_entropy_workspace_bytes
    assert size(2, 0, 10, 10, 10) == 0 and size(0, 0, 10, 10, 0) == 0 and size(1, 3, 10, 10, 10) == 0


@pytest.mark.parametrize("dims", [(257, 513), (65536, 2048), (50001, 72), (1, 1), (300, 4096), (131072, 64)], ids=str)
def test_cross_entropy_workspaces_serve_fewer_tokens(L, dims):
    for p in (0, 1):
        for dtype in (0, 1):
            last = 0
            for tokens in list(range(0, 1500)) + list(range(1500, 70000, 97)) + [1 << 20]:
                need = L.laplex_linear_cross_entropy_workspace_bytes(p, dtype, tokens, *dims)
                assert need >= last and need % 256 == 0, (p, dtype, tokens)
                last = need
    # the logits' gradient is formed in pieces: far less than it whole
    assert L.laplex_linear_cross_entropy_workspace_bytes(1, 1, 1 << 16, 131072, 64) < (1 << 16) * 131072 * 2 // 8


def tensors(*rows):
    import array
    return array.array("Q", [x for r in rows for x in r])


def test_adamw(L):
    from laplace_prefix_scans_amd._training import _AdamArgs

    def one(p=10, g=20, m=30, v=40, ms=0, vs=0, master=0, n=100, off=0):
        return [x * MB if x else 0 for x in (p, g, m, v, ms, vs, master)] + [n, 0]

    def step(rows, count=None, dt=0, gd=0, bits=32, st=1, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, **over):
        a = _AdamArgs(dt, gd, bits, 0, 0, st, lr, b1, b2, eps, None, None, None)
        for k, v in over.items():
            setattr(a, k, v)
        t = tensors(*rows)
        return L.laplex_adamw(ctypes.byref(a), t.buffer_info()[0] if rows else None, len(rows) if count is None else count, None)
    assert L.laplex_adamw(None, None, 0, None) == NULL
    assert step([]) == OK and step([one(n=0, p=0)]) == OK and step([], count=1) == NULL
    assert step([one()], dt=2) == ARG and step([one()], gd=-1) == ARG and step([one()], bits=16) == ARG and step([one()], st=0) == ARG
    assert step([one()], b1=1.0) == ARG and step([one()], b2=-0.1) == ARG and step([one()], eps=-1.0) == ARG
    assert step([one()], lr=float("nan")) == ARG and step([one()], b1=float("nan")) == ARG
    assert step([one()], lr_dev=6) == ALIGN and step([one()], step_dev=6) == ALIGN
    for name in ("p", "g", "m", "v"):
        assert step([one(**{name: 0})]) == NULL
    assert step([one()], bits=8) == NULL and step([one(ms=50)], bits=8) == NULL
    bad = one()
    bad[0] += 2
    assert step([bad]) == ALIGN
    bad = one(ms=50, vs=60)
    bad[5] += 2
    assert step([bad], bits=8) == ALIGN
    assert step([one(n=1 << 41)]) == SIZE
    # outputs on outputs, within a tensor and across them; on gradients; a shared gradient passes this check
    assert step([one(m=10)]) == OVERLAP and step([one(g=10)]) == OVERLAP and step([one(), one(g=70, m=80, v=90)]) == OVERLAP
    assert step([one(), one(p=110, m=130, v=20)]) == OVERLAP and step([one(master=10)]) == OVERLAP
    assert step([one(ms=50, vs=50)], bits=8) == OVERLAP
    assert step([one(n=1 << 20)] + [one(p=12, m=130, v=140, g=120)]) == OVERLAP  # inside the first one's four megabytes
    assert step([one()], lr_dev=10 * MB) == OVERLAP
    assert L.laplex_adamw_moments(None, 1, None) == NULL and L.laplex_adamw_moments(None, 0, None) == OK
    t = tensors(one(ms=50, vs=60, master=10))
    assert L.laplex_adamw_moments(t.buffer_info()[0], 1, None) == OVERLAP
    t = tensors(one(ms=50))
    assert L.laplex_adamw_moments(t.buffer_info()[0], 1, None) == NULL


def test_binding_refuses_cpu_tensors_and_wrong_types():
    import torch
    import laplace_prefix_scans_amd as lp
    x = torch.zeros(4, 8)
    y = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        lp.laplex_gated_scan(x, x)
    with pytest.raises(TypeError):
        lp.laplex_gated_scan(None, x)
    with pytest.raises(ValueError):
        lp.laplex_gated_scan_step(torch.zeros(2, 4, 8), x, x)
    with pytest.raises(ValueError):
        lp.laplex_linear_cross_entropy(x, torch.zeros(9, 8), y)
    with pytest.raises(ValueError):
        lp.laplex_adamw([x], [x], [x], [x], lr=1e-3, step=1)
    with pytest.raises(ValueError):
        lp.laplex_adamw([x], [x], [x], [], lr=1e-3, step=1)
    lp.laplex_adamw([], [], [], [], lr=1e-3, step=1)


@pytest.mark.gpu
def test_binding_refuses_wrong_shapes():
    import torch
    import laplace_prefix_scans_amd as lp
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    z = lambda *s, dt=torch.float32: torch.zeros(s, device="cuda", dtype=dt)  # noqa: E731
    g = z(10, 8)
    for over, err in ((dict(x=z(9, 8)), ValueError), (dict(x=z(10, 8, dt=torch.bfloat16)), TypeError), (dict(kind="tanh"), ValueError),
                      (dict(gate=z(10, 8, dt=torch.float16)), TypeError), (dict(gate=z(80), x=z(80)), ValueError),
                      (dict(gate=z(8, 10).t()), ValueError), (dict(offsets=z(3)), TypeError), (dict(offsets=torch.tensor([0, 10])), ValueError),
                      (dict(state_in=z(2, 8)), ValueError), (dict(state_out=z(1, 8, dt=torch.bfloat16)), TypeError), (dict(h=z(10, 9)), ValueError),
                      (dict(gate=z(2, 5, 8), x=z(2, 5, 8), offsets=z(3, dt=torch.int32)), ValueError),
                      (dict(gate=z(2, 9, 8)[:, :5], x=z(2, 5, 8)), ValueError), (dict(x=None), TypeError)):
        with pytest.raises(err):
            lp.laplex_gated_scan(**{"gate": g, "x": z(10, 8), **over})
    with pytest.raises(lp.LaplexError):
        lp.laplex_gated_scan(g, z(10, 8), h=g)
    h, c = lp.laplex_gated_scan(g, z(10, 8), keep=True)
    for over in (dict(carries=z(2, 8)), dict(dh=z(10, 7)), dict(dh=z(8, 10).t())):
        with pytest.raises(ValueError):
            lp.laplex_gated_scan_backward(**{"gate": g, "x": z(10, 8), "carries": c, "dh": h, **over})
    with pytest.raises(ValueError):
        lp.laplex_gated_scan_step(g, z(10, 8), z(9, 8))
    with pytest.raises(TypeError):
        lp.laplex_gated_scan_step(g, z(10, 8), z(10, 8), slots=torch.zeros(10, dtype=torch.int64, device="cuda"))
    x, w, y = z(6, 8), z(20, 8), torch.zeros(6, dtype=torch.int64, device="cuda")
    for over, err in ((dict(x=z(5, 8)), ValueError), (dict(x=z(6, 7)), ValueError), (dict(table=z(20, 8, dt=torch.bfloat16)), TypeError),
                      (dict(targets=z(6)), TypeError), (dict(table=z(8, 20).t()), ValueError), (dict(x=z(8, 6).t()), ValueError),
                      (dict(targets=y.cpu()), ValueError), (dict(table=z(0, 8)), ValueError), (dict(x=[1.0]), TypeError)):
        with pytest.raises(err):
            lp.laplex_linear_cross_entropy(**{"x": x, "table": w, "targets": y, **over})
    for over, err in ((dict(lse=z(5)), ValueError), (dict(dloss=z(6, dt=torch.bfloat16)), TypeError), (dict(dloss=None), TypeError),
                      (dict(dtype=torch.float16), TypeError), (dict(dlse=z(6, 1)), ValueError)):
        with pytest.raises(err):
            lp.laplex_linear_cross_entropy_backward(**{"x": x, "table": w, "targets": y, "lse": z(6), "dloss": z(6), **over})
    good = dict(params=[z(9)], grads=[z(9)], m=[z(9)], v=[z(9)], lr=1e-3, step=1)
    s8 = z(9, dt=torch.float8_e4m3fn)
    for over, err in ((dict(grads=[z(8)]), ValueError), (dict(params=[z(9), z(9)]), ValueError), (dict(m=[z(9, dt=torch.bfloat16)]), TypeError),
                      (dict(m=[s8], v=[s8.clone()]), ValueError), (dict(m_scale=[z(1)], v_scale=[z(1)]), ValueError), (dict(step=0), ValueError),
                      (dict(step=torch.tensor([1], device="cuda")), TypeError), (dict(lr=torch.tensor(0.1)), ValueError),
                      (dict(weight_decay=[0.1, 0.1]), ValueError), (dict(master=[z(9, dt=torch.bfloat16)]), TypeError),
                      (dict(m=[s8], v=[s8.clone()], m_scale=[z(1)], v_scale=[z(2)]), ValueError), (dict(grads=[None]), TypeError),
                      (dict(params=[z(9, dt=torch.float16)]), TypeError), (dict(params=[z(18)[::2]]), ValueError)):
        with pytest.raises(err):
            lp.laplex_adamw(**{**good, **over})
    with pytest.raises(lp.LaplexError):
        lp.laplex_adamw(**{**good, "betas": (1.0, 0.9)})
