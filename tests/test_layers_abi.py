"""The sequence layers' entry points reject bad arguments on the host (no GPU work
is started: every call fails a check, or has nothing to do, before a launch), and
the binding rejects tensors of the wrong kind."""
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
    from laplace_prefix_scans_amd import _layers
    if not os.path.exists(lp.lib_path()):
        pytest.skip("liblaplex.so not built")
    return _layers._lib()


def shape(**over):
    from laplace_prefix_scans_amd._layers import _Shape
    s = _Shape(0, 2, 4, 2, 32, 16, 100, None, 1 * MB, 1.0, 128, 32, 64, 32, 32, 16)
    for k, v in over.items():
        setattr(s, k, v)
    return ctypes.byref(s)


def forward(L, s, q=at(10), k=at(20), v=at(30), si=None, so=None, o=at(40), ws=at(100), wb=64 * MB):
    return L.laplex_decay_attn(s, q, k, v, si, so, o, ws, wb, None)


def backward(L, s, q=at(10), k=at(20), v=at(30), g=at(35), si=None, gso=None, dq=at(40), dk=at(45), dv=at(50), dr=at(55),
             dsi=None, ws=at(100), wb=64 * MB):
    return L.laplex_decay_attn_backward(s, q, k, v, g, si, gso, dq, dk, dv, dr, dsi, ws, wb, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_attention_shapes(L, call):
    assert call(L, None) == NULL
    assert call(L, shape(dtype=2)) == ARG
    assert call(L, shape(kv_heads=3)) == ARG
    assert call(L, shape(heads=0)) == ARG
    assert call(L, shape(dk=0)) == ARG
    assert call(L, shape(dk=257)) == SIZE
    assert call(L, shape(dv=300)) == SIZE
    assert call(L, shape(tokens=1 << 31)) == SIZE
    assert call(L, shape(seqs=1 << 20, heads=4096, kv_heads=1)) == SIZE
    assert call(L, shape(tokens=101)) == ARG       # equal lengths do not divide
    assert call(L, shape(seqs=0)) == ARG           # tokens of no sequence
    assert call(L, shape(rate=None)) == NULL
    assert call(L, shape(q_token=-1)) == ARG
    assert call(L, shape(k_head=1 << 62)) == ARG


def test_attention_pointers(L):
    assert forward(L, shape(), q=None) == NULL
    assert forward(L, shape(), o=None) == NULL
    assert forward(L, shape(), q=at(10, 2)) == ALIGN
    assert forward(L, shape(dtype=1), q=at(10, 1)) == ALIGN
    assert forward(L, shape(), ws=at(100, 128)) == ALIGN
    assert forward(L, shape(offsets=at(5, 2).value)) == ALIGN
    assert forward(L, shape(), o=at(10, 64)) == OVERLAP
    assert forward(L, shape(), si=at(60), so=at(60)) == OVERLAP
    assert forward(L, shape(offsets=at(40).value)) == OVERLAP
    assert backward(L, shape(), dk=at(40)) == OVERLAP
    assert backward(L, shape(), dr=at(1)) == OVERLAP   # the rates themselves
    assert backward(L, shape(), g=None) == NULL
    assert backward(L, shape(), ws=None) == NULL
    assert backward(L, shape(), wb=16) == WS
    assert backward(L, shape(), gso=at(60), dsi=at(60, 16)) == OVERLAP


def test_attention_nothing_to_do(L):
    assert forward(L, shape(seqs=0, tokens=0), q=None, k=None, v=None, o=None, ws=None, wb=0) == OK
    assert forward(L, shape(tokens=0), q=None, k=None, v=None, o=None, ws=None, wb=0) == OK
    assert backward(L, shape(seqs=0, tokens=0), q=None, k=None, v=None, g=None, dq=None, dk=None, dv=None, dr=None) == OK


def test_attention_workspace(L):
    size = lambda p, **o: L.laplex_decay_attn_workspace_bytes(p, shape(**o))  # noqa: E731
    assert size(2) == 0 and size(0, dk=300) == 0
    assert size(0) % 256 == 0 and size(1) % 256 == 0
    # short inputs need no segment states; long ones need more for the backward pass than for the forward pass
    assert size(0) == 0
    big = dict(tokens=1 << 16, seqs=1, heads=8, kv_heads=8, dk=128, dv=128)
    assert 0 < size(0, **big) < size(1, **big) < 1 << 30
    assert forward(L, shape(**big), q=at(1000), k=at(2000), v=at(3000), o=at(4000), ws=at(5000), wb=size(0, **big) - 256) == WS
    # shared heads keep per-head gradients
    assert size(1, **dict(big, kv_heads=2)) > size(1, **big)


def test_step(L):
    def step(s, q=at(10), k=at(20), v=at(30), slots=at(35), pool=8, state=at(40), o=at(50)):
        return L.laplex_decay_attn_step(s, q, k, v, slots, pool, state, o, None)
    one = dict(seqs=5, tokens=5)
    assert step(shape(seqs=5, tokens=6)) == ARG
    assert step(shape(**one), slots=None, pool=4) == ARG
    assert step(shape(**one), q=None) == NULL
    assert step(shape(**one), state=None) == NULL
    assert step(shape(**one), slots=at(35, 2)) == ALIGN
    assert step(shape(**one), o=at(40, 64)) == OVERLAP
    assert step(shape(**one), q=at(40)) == OVERLAP
    assert step(shape(seqs=0, tokens=0), q=None, state=None) == OK


def test_layer_norm(L):
    def norm(dt=0, rows=8, width=64, x=at(10), w=at(20), b=at(21), y=at(30), m=at(40), r=at(41)):
        return L.laplex_layer_norm(dt, rows, width, x, w, b, 1e-5, y, m, r, None)

    def back(dt=0, rows=8, width=64, x=at(10), dy=at(15), m=at(40), r=at(41), w=at(20), dx=at(30), dw=at(50), db=at(51),
             ws=at(100), wb=MB):
        return L.laplex_layer_norm_backward(dt, rows, width, x, dy, m, r, w, dx, dw, db, ws, wb, None)
    assert norm(dt=3) == ARG and norm(width=0) == ARG and norm(rows=1 << 32) == SIZE and norm(width=(1 << 24) + 1) == SIZE
    assert norm(rows=0) == OK
    assert norm(x=None) == NULL and norm(y=None) == NULL
    assert norm(x=at(10, 2)) == ALIGN and norm(dt=1, w=at(20, 1)) == ALIGN and norm(m=at(40, 2)) == ALIGN
    assert norm(y=at(10)) == OVERLAP and norm(m=at(40), r=at(40, 16)) == OVERLAP and norm(y=at(20)) == OVERLAP
    assert back(dt=-1) == ARG and back(width=0) == ARG
    assert back(m=None) == NULL and back(ws=None) == NULL
    assert back(ws=at(100, 4)) == ALIGN and back(dw=at(50, 1)) == ALIGN
    assert back(wb=64) == WS
    assert back(dx=at(15)) == OVERLAP and back(dw=at(50), db=at(50)) == OVERLAP and back(dw=at(100)) == OVERLAP
    assert L.laplex_layer_norm_workspace_bytes(8, 0) == 0
    sizes = [L.laplex_layer_norm_workspace_bytes(r, 512) for r in (0, 1, 100, 5000, 10 ** 6)]
    assert sizes == sorted(sizes)


def test_embedding(L):
    def look(dt=0, ids=at(5), nb=8, t=16, table=at(10), vocab=100, width=32, y=at(20)):
        return L.laplex_embedding(dt, ids, nb, t, table, vocab, width, 1.0, y, None)

    def back(dt=0, ids=at(5), nb=8, t=16, dy=at(10), vocab=100, width=32, td=0, out=at(20), ws=at(100), wb=64 * MB):
        return L.laplex_embedding_backward(dt, ids, nb, t, dy, vocab, width, 1.0, td, out, ws, wb, None)
    assert look(dt=2) == ARG and look(nb=2) == ARG and look(width=0) == ARG
    assert look(t=(1 << 28) + 1) == SIZE and look(vocab=(1 << 26) + 1) == SIZE
    assert look(t=0, ids=None, y=None) == OK
    assert look(ids=None) == NULL and look(table=None) == NULL and look(y=None) == NULL
    assert look(ids=at(5, 4)) == ALIGN and look(y=at(20, 2)) == ALIGN
    assert look(y=at(10, 128)) == OVERLAP and look(y=at(5)) == OVERLAP
    assert back(td=1) == ARG and back(dt=1, td=2) == ARG and back(nb=1) == ARG
    assert back(vocab=0) == OK
    assert back(out=None) == NULL and back(ws=None) == NULL and back(dy=None) == NULL
    assert back(ws=at(100, 8)) == ALIGN and back(ids=at(5, 4)) == ALIGN
    assert back(wb=256) == WS
    assert back(out=at(10)) == OVERLAP and back(out=at(100)) == OVERLAP
    assert L.laplex_embedding_workspace_bytes(10, 10, 0) == 0
    assert L.laplex_embedding_workspace_bytes(1 << 29, 10, 8) == 0
    sizes = [L.laplex_embedding_workspace_bytes(t, 5000, 64) for t in (0, 1, 100, 16384, 16385, 32769, 10 ** 6)]
    assert sizes == sorted(sizes)


def test_binding_refuses_cpu_tensors_and_wrong_types():
    import torch
    import laplace_prefix_scans_amd as lp
    q = torch.zeros(4, 2, 8)
    with pytest.raises(ValueError):
        lp.laplex_decay_attn(q, q, q, torch.zeros(2))
    with pytest.raises(TypeError):
        lp.laplex_decay_attn(None, q, q, torch.zeros(2))
    with pytest.raises(ValueError):
        lp.laplex_layer_norm(torch.zeros(3, 4))
    with pytest.raises(ValueError):
        lp.laplex_embedding(torch.zeros(3, dtype=torch.int64), torch.zeros(4, 4))
    with pytest.raises(TypeError):
        lp.laplex_layer_norm([1.0, 2.0])


@pytest.mark.gpu
def test_binding_refuses_wrong_shapes():
    import torch
    import laplace_prefix_scans_amd as lp
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    z = lambda *s, dt=torch.float32: torch.zeros(s, device="cuda", dtype=dt)  # noqa: E731
    q, k, v, r = z(10, 4, 8), z(10, 2, 8), z(10, 2, 6), z(4)
    good = dict(q=q, k=k, v=v, rate=r)
    bad = [(dict(q=z(10, 4, 8, dt=torch.float16)), TypeError), (dict(k=z(10, 2, 8, dt=torch.bfloat16)), TypeError),
           (dict(k=z(10, 3, 8), v=z(10, 3, 6)), ValueError), (dict(k=z(9, 2, 8)), ValueError), (dict(k=z(10, 2, 7)), ValueError),
           (dict(v=z(10, 1, 6)), ValueError), (dict(rate=z(3)), ValueError), (dict(rate=z(4, dt=torch.float64)), TypeError),
           (dict(rate=None), TypeError), (dict(q=z(10, 8, 4).transpose(1, 2)), ValueError), (dict(q=z(40, 8)), ValueError),
           (dict(offsets=torch.tensor([0, 10])), ValueError), (dict(offsets=z(3)), TypeError),
           (dict(state_in=z(1, 4, 8, 5)), ValueError), (dict(state_out=z(1, 4, 6, 8)), ValueError), (dict(o=z(10, 4, 8)), ValueError),
           (dict(ws=z(10)), ValueError)]
    for over, err in bad:
        with pytest.raises(err):
            lp.laplex_decay_attn(**{**good, **over})
    with pytest.raises(ValueError):  # a batch whose sequences do not follow each other
        lp.laplex_decay_attn(z(2, 8, 4, 8)[:, :5], z(2, 5, 2, 8), z(2, 5, 2, 6), r)
    with pytest.raises(ValueError):
        lp.laplex_decay_attn_backward(q, k, v, r, z(10, 4, 8))
    with pytest.raises(lp.LaplexError):
        lp.laplex_decay_attn(z(10, 4, 300), z(10, 2, 300), v, r)
    with pytest.raises(lp.LaplexError):  # the output lies on an input
        lp.laplex_decay_attn(q, k, z(10, 2, 8), r, o=q)
    with pytest.raises(ValueError):
        lp.laplex_decay_attn_step(q, k, v, r, z(9, 4, 8, 6))
    with pytest.raises(ValueError):
        lp.laplex_decay_attn_step(q, k, v, r, z(10, 4, 6, 8))
    with pytest.raises(TypeError):
        lp.laplex_decay_attn_step(q, k, v, r, z(10, 4, 8, 6), slots=torch.zeros(10, dtype=torch.int64, device="cuda"))
    x = z(5, 16)
    for over, err in ((dict(weight=z(15)), ValueError), (dict(bias=z(16, dt=torch.bfloat16)), TypeError), (dict(y=z(4, 16)), ValueError)):
        with pytest.raises(err):
            lp.laplex_layer_norm(x, **over)
    with pytest.raises(ValueError):
        lp.laplex_layer_norm(z(16, 5).t())
    with pytest.raises(lp.LaplexError):
        lp.laplex_layer_norm(x, y=x)
    with pytest.raises(ValueError):
        lp.laplex_layer_norm_backward(x, x, z(4), z(5))
    ids = torch.zeros(6, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        lp.laplex_embedding(z(6), z(4, 4))
    with pytest.raises(ValueError):
        lp.laplex_embedding(ids, z(4, 4).t()[1:])
    with pytest.raises(ValueError):
        lp.laplex_embedding_backward(ids, z(5, 4), 10)
    with pytest.raises(TypeError):
        lp.laplex_embedding_backward(ids, z(6, 4), 10, dtype=torch.float16)
