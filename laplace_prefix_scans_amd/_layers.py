"""Binding of the sequence layers of liblaplex.so: decayed linear attention,
layer norm and embedding (declarations in include/laplex.h)."""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from ._binding import LaplexError, _check, _ptr, _stream, lib

LAPLEX_F32, LAPLEX_BF16 = 0, 1
LAPLEX_ATTN_FORWARD, LAPLEX_ATTN_BACKWARD = 0, 1
_DTYPES = {torch.float32: LAPLEX_F32, torch.bfloat16: LAPLEX_BF16}


class _Shape(ctypes.Structure):
    """laplex_attn_shape"""
    _fields_ = [("dtype", ctypes.c_int32), ("seqs", ctypes.c_uint32), ("heads", ctypes.c_uint32), ("kv_heads", ctypes.c_uint32),
                ("dk", ctypes.c_uint32), ("dv", ctypes.c_uint32), ("tokens", ctypes.c_uint64), ("offsets", ctypes.c_void_p),
                ("rate", ctypes.c_void_p), ("scale", ctypes.c_float),
                ("q_token", ctypes.c_int64), ("q_head", ctypes.c_int64), ("k_token", ctypes.c_int64),
                ("k_head", ctypes.c_int64), ("v_token", ctypes.c_int64), ("v_head", ctypes.c_int64)]


_ready = None


def _lib():
    global _ready
    if _ready is None:
        L = lib()
        vp, u64, u32, sz, i32, f32 = (ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_size_t, ctypes.c_int,
                                      ctypes.c_float)
        shape = ctypes.POINTER(_Shape)
        L.laplex_decay_attn_workspace_bytes.argtypes = [i32, shape]
        L.laplex_decay_attn_workspace_bytes.restype = sz
        L.laplex_decay_attn.argtypes = [shape, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.laplex_decay_attn_backward.argtypes = [shape] + [vp] * 12 + [sz, vp]
        L.laplex_decay_attn_step.argtypes = [shape, vp, vp, vp, vp, u32, vp, vp, vp]
        L.laplex_layer_norm.argtypes = [i32, u64, u32, vp, vp, vp, f32, vp, vp, vp, vp]
        L.laplex_layer_norm_workspace_bytes.argtypes = [u64, u32]
        L.laplex_layer_norm_workspace_bytes.restype = sz
        L.laplex_layer_norm_backward.argtypes = [i32, u64, u32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.laplex_embedding.argtypes = [i32, vp, i32, u64, vp, u32, u32, f32, vp, vp]
        L.laplex_embedding_workspace_bytes.argtypes = [u64, u32, u32]
        L.laplex_embedding_workspace_bytes.restype = sz
        L.laplex_embedding_backward.argtypes = [i32, vp, i32, u64, vp, u32, u32, f32, i32, vp, vp, sz, vp]
        for f in (L.laplex_decay_attn, L.laplex_decay_attn_backward, L.laplex_decay_attn_step, L.laplex_layer_norm,
                  L.laplex_layer_norm_backward, L.laplex_embedding, L.laplex_embedding_backward):
            f.restype = i32
        _ready = L
    return _ready


# These calls are often a few microseconds of GPU work each (one token, one
# row), so the checks read every attribute of a tensor once and the stream
# comes as the raw handle.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(dev: torch.device) -> int:
    return _raw_stream(dev.index) if _raw_stream is not None else _stream(dev)


def _u32(where: str, sizes: int) -> None:
    """Sizes (or-ed together) go to the library in 32 bits: ctypes would wrap larger ones before its checks see them."""
    if sizes >> 32:
        raise LaplexError(2, where)  # LAPLEX_ERR_SIZE


def _dtype(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on a GPU device" % name)
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
    return code


def _like(t, name: str, shape, dtype, dev) -> Optional[torch.Tensor]:
    """t as a contiguous tensor of this shape, type and device (None passes)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.device != dev:
        raise ValueError("%s must be on %s" % (name, dev))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _out(t, name: str, shape, dtype, dev) -> torch.Tensor:
    return torch.empty(shape, dtype=dtype, device=dev) if t is None else _like(t, name, shape, dtype, dev)


def _bytes(ws: Optional[torch.Tensor], need: int, dev) -> Tuple[Optional[torch.Tensor], int]:
    """The workspace and its size; none where none is needed."""
    if ws is None:
        return (torch.empty(need, dtype=torch.uint8, device=dev), need) if need else (None, 0)
    if ws.device != dev or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on %s" % dev)
    return ws, ws.numel()


# ------------------------------------------------------------------ decayed attention
def _strides(t: torch.Tensor, shape, name: str, batched: bool) -> Tuple[int, int]:
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError("%s must have contiguous channels" % name)
    if not batched:
        return st[0], st[1]
    # (an axis of one token has no stride of its own: the batch's is the token's)
    if shape[0] > 1 and shape[1] > 1 and st[0] != shape[1] * st[1]:
        raise ValueError("%s: the tokens of a batch must lie one sequence after the other" % name)
    return (st[0] if shape[1] == 1 else st[1]), st[2]


def _shape(q, k, v, rate, offsets, scale) -> _Shape:
    code = _dtype(q, "q")
    dev, dtype, qs = q.device, q.dtype, q.shape
    dims = len(qs)
    if dims != 3 and dims != 4:
        raise ValueError("q must be (tokens, heads, channels) or (batch, tokens, heads, channels)")
    for t, name in ((k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch tensor" % name)
        if t.dtype != dtype or t.device != dev:
            raise TypeError("%s must have the type and device of q" % name)
    ks, vs = k.shape, v.shape
    batched = dims == 4
    lead = qs[:-2]
    if len(ks) != dims or len(vs) != dims or ks[:-2] != lead or vs[:-1] != ks[:-1] or ks[-1] != qs[-1]:
        raise ValueError("k must have the tokens and channels of q, v the tokens and heads of k: got q %s, k %s, v %s"
                         % (tuple(qs), tuple(ks), tuple(vs)))
    heads, kv_heads = qs[-2], ks[-2]
    if kv_heads == 0 or heads % kv_heads:
        raise ValueError("the %d heads of k and v must divide the %d of q" % (kv_heads, heads))
    _u32("decayed attention", qs[0] | heads | qs[-1] | vs[-1])
    if rate is None:
        raise TypeError("rate must be a torch tensor")
    _like(rate, "rate", (heads,), torch.float32, dev)
    seqs = qs[0] if batched else 1
    if offsets is not None:
        if batched:
            raise ValueError("offsets go with packed (tokens, heads, channels) tensors")
        if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 1:
            raise ValueError("offsets must be a 1-D tensor of sequence starts and the end of the last")
        _like(offsets, "offsets", offsets.shape, torch.int32, dev)
        seqs = offsets.numel() - 1
        _u32("decayed attention", seqs)
    tokens = qs[0] * qs[1] if batched else qs[0]
    (qt, qh), (kt, kh), (vt, vh) = (_strides(q, qs, "q", batched), _strides(k, ks, "k", batched),
                                    _strides(v, vs, "v", batched))
    return _Shape(code, seqs, heads, kv_heads, qs[-1], vs[-1], tokens, _ptr(offsets), rate.data_ptr(), scale,
                  qt, qh, kt, kh, vt, vh)


def laplex_decay_attn_workspace_bytes(backward: bool, q, k, v, rate, offsets=None) -> int:
    """Bytes of workspace of laplex_decay_attn (or its backward) for these tensors."""
    s = _shape(q, k, v, rate, offsets, 1.0)
    return int(_lib().laplex_decay_attn_workspace_bytes(LAPLEX_ATTN_BACKWARD if backward else LAPLEX_ATTN_FORWARD,
                                                        ctypes.byref(s)))


def laplex_decay_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rate: torch.Tensor,
                      offsets: Optional[torch.Tensor] = None, scale: float = 1.0, state_in: Optional[torch.Tensor] = None,
                      state_out: Optional[torch.Tensor] = None, o: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """o_i = scale sum_{j <= i} exp(-rate_h (i - j)) (q_i . k_j) v_j over each sequence.

    q: (tokens, heads, dk), k: (tokens, kv_heads, dk), v: (tokens, kv_heads, dv), float32 or bfloat16,
    channels contiguous, other strides free; with a leading batch axis, sequences of equal length.
    rate: (heads,) float32, >= 0.  offsets: int32 (seqs + 1,), the packed sequences' starts and the last
    one's end; without it and without a batch axis, one sequence.  state_in: (seqs, heads, dk, dv)
    float32 carried in, or None; state_out: the same shape, filled with the states after the last
    tokens.  Returns o, (tokens, heads, dv) in the type of q."""
    s = _shape(q, k, v, rate, offsets, scale)
    dev = q.device
    st = (s.seqs, s.heads, s.dk, s.dv)
    _like(state_in, "state_in", st, torch.float32, dev)
    _like(state_out, "state_out", st, torch.float32, dev)
    o = _out(o, "o", (*q.shape[:-1], s.dv), q.dtype, dev)
    L = _lib()
    ws, ws_bytes = _bytes(ws, L.laplex_decay_attn_workspace_bytes(LAPLEX_ATTN_FORWARD, ctypes.byref(s)), dev)
    _check(L.laplex_decay_attn(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(state_in), _ptr(state_out), _ptr(o), _ptr(ws),
                               ws_bytes, _stream_of(dev)), "laplex_decay_attn")
    return o


def laplex_decay_attn_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rate: torch.Tensor, go: torch.Tensor,
                               offsets: Optional[torch.Tensor] = None, scale: float = 1.0,
                               state_in: Optional[torch.Tensor] = None, dstate_out: Optional[torch.Tensor] = None,
                               rate_grad: bool = True, ws: Optional[torch.Tensor] = None):
    """Backward of laplex_decay_attn for go = dL/do and dstate_out = dL/dstate_out (None: zero).

    Returns (dq, dk, dv, drate, dstate_in): the gradients of q, k, v in their shapes and type, drate (heads,)
    float32 (None with rate_grad=False), dstate_in like state_in (None where state_in is None)."""
    s = _shape(q, k, v, rate, offsets, scale)
    dev = q.device
    st = (s.seqs, s.heads, s.dk, s.dv)
    if go is None:
        raise TypeError("go must be a torch tensor")
    _like(go, "go", (*q.shape[:-1], s.dv), q.dtype, dev)
    _like(state_in, "state_in", st, torch.float32, dev)
    _like(dstate_out, "dstate_out", st, torch.float32, dev)
    dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=dev) for t in (q, k, v))
    drate = torch.empty(s.heads, dtype=torch.float32, device=dev) if rate_grad else None
    dstate_in = torch.empty(st, dtype=torch.float32, device=dev) if state_in is not None else None
    L = _lib()
    ws, ws_bytes = _bytes(ws, L.laplex_decay_attn_workspace_bytes(LAPLEX_ATTN_BACKWARD, ctypes.byref(s)), dev)
    _check(L.laplex_decay_attn_backward(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(go), _ptr(state_in), _ptr(dstate_out),
                                        _ptr(dq), _ptr(dk), _ptr(dv), _ptr(drate), _ptr(dstate_in), _ptr(ws), ws_bytes,
                                        _stream_of(dev)), "laplex_decay_attn_backward")
    return dq, dk, dv, drate, dstate_in


def laplex_decay_attn_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rate: torch.Tensor, state: torch.Tensor,
                           slots: Optional[torch.Tensor] = None, scale: float = 1.0,
                           o: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token for each row: state = exp(-rate_h) state + k v^T in place, o = scale q state.

    q: (rows, heads, dk), k: (rows, kv_heads, dk), v: (rows, kv_heads, dv); state: (pool, heads, dk, dv)
    float32; slots: int32 (rows,), the state of each row (None: row r has state r).  A row whose slot is
    outside the pool has no sequence: its output is zero and no state changes.  Two rows must not share
    a slot."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be (rows, heads, dk)")
    s = _shape(q, k, v, rate, None, scale)
    dev, s.seqs = q.device, q.shape[0]
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be (pool, heads, dk, dv)")
    _like(state, "state", (state.shape[0], s.heads, s.dk, s.dv), torch.float32, dev)
    _like(slots, "slots", (s.seqs,), torch.int32, dev)
    _u32("laplex_decay_attn_step", state.shape[0])
    if slots is None and s.seqs > state.shape[0]:
        raise ValueError("state must have a row for each of the %d tokens" % s.seqs)
    o = _out(o, "o", (s.seqs, s.heads, s.dv), q.dtype, dev)
    _check(_lib().laplex_decay_attn_step(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(slots), state.shape[0], _ptr(state),
                                         _ptr(o), _stream_of(dev)), "laplex_decay_attn_step")
    return o


# ------------------------------------------------------------------ layer norm
def _rows(x: torch.Tensor, name: str) -> Tuple[int, int, int]:
    code = _dtype(x, name)
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError("%s must have rows of at least one element" % name)
    if not x.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    width = x.shape[-1]
    _u32("layer norm", width)
    return code, x.numel() // width, width


def laplex_layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                      eps: float = 1e-5, y: Optional[torch.Tensor] = None):
    """y = (x - mean) rstd weight + bias over the last axis.  x: (..., width) float32 or bfloat16; weight,
    bias: (width,) of the same type, or None.  Returns (y, mean, rstd), the last two float32 (...,)."""
    code, rows, width = _rows(x, "x")
    dev = x.device
    _like(weight, "weight", (width,), x.dtype, dev)
    _like(bias, "bias", (width,), x.dtype, dev)
    y = _out(y, "y", x.shape, x.dtype, dev)
    mean, rstd = torch.empty((2, *x.shape[:-1]), dtype=torch.float32, device=dev).unbind(0)
    _check(_lib().laplex_layer_norm(code, rows, width, _ptr(x), _ptr(weight), _ptr(bias), eps, _ptr(y), _ptr(mean), _ptr(rstd),
                                    _stream_of(dev)), "laplex_layer_norm")
    return y, mean, rstd


def laplex_layer_norm_backward(x: torch.Tensor, dy: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                               weight: Optional[torch.Tensor] = None, param_grads: bool = True,
                               ws: Optional[torch.Tensor] = None):
    """(dx, dweight, dbias) for the upstream gradient dy of laplex_layer_norm; dweight and dbias are float32
    (width,), or None with param_grads=False."""
    code, rows, width = _rows(x, "x")
    dev = x.device
    if dy is None or mean is None or rstd is None:
        raise TypeError("dy, mean and rstd must be torch tensors")
    _like(dy, "dy", x.shape, x.dtype, dev)
    _like(mean, "mean", x.shape[:-1], torch.float32, dev)
    _like(rstd, "rstd", x.shape[:-1], torch.float32, dev)
    _like(weight, "weight", (width,), x.dtype, dev)
    dx = torch.empty_like(x)
    dw, db = torch.empty((2, width), dtype=torch.float32, device=dev).unbind(0) if param_grads else (None, None)
    L = _lib()
    ws, ws_bytes = _bytes(ws, L.laplex_layer_norm_workspace_bytes(rows, width), dev)
    _check(L.laplex_layer_norm_backward(code, rows, width, _ptr(x), _ptr(dy), _ptr(mean), _ptr(rstd), _ptr(weight), _ptr(dx),
                                        _ptr(dw), _ptr(db), _ptr(ws), ws_bytes, _stream_of(dev)), "laplex_layer_norm_backward")
    return dx, dw, db


# ------------------------------------------------------------------ embedding
def _ids(ids: torch.Tensor, dev) -> int:
    if not isinstance(ids, torch.Tensor) or ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be an int32 or int64 tensor")
    if ids.device != dev or not ids.is_contiguous():
        raise ValueError("ids must be contiguous and on %s" % dev)
    return 8 if ids.dtype == torch.int64 else 4


def laplex_embedding(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0,
                     y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = scale table[ids], (*ids.shape, width); a zero row where an id is outside the table (padding)."""
    code = _dtype(table, "table")
    dev = table.device
    nb = _ids(ids, dev)
    if table.dim() != 2 or table.shape[1] == 0 or not table.is_contiguous():
        raise ValueError("table must be a contiguous (vocab, width) tensor")
    vocab, width = table.shape
    _u32("laplex_embedding", vocab | width)
    y = _out(y, "y", (*ids.shape, width), table.dtype, dev)
    _check(_lib().laplex_embedding(code, _ptr(ids), nb, ids.numel(), _ptr(table), vocab, width, scale, _ptr(y), _stream_of(dev)),
           "laplex_embedding")
    return y


def laplex_embedding_backward(ids: torch.Tensor, dy: torch.Tensor, vocab: int, scale: float = 1.0,
                              dtype: Optional[torch.dtype] = None, dtable: Optional[torch.Tensor] = None,
                              ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient (vocab, width) of the table for the upstream gradient dy (*ids.shape, width): the rows of dy
    added by id, in an order that the ids alone fix.  dtype: float32 or the type of dy (the default)."""
    code = _dtype(dy, "dy")
    dev = dy.device
    nb = _ids(ids, dev)
    if dy.dim() != ids.dim() + 1 or dy.shape[:-1] != ids.shape or dy.shape[-1] == 0 or not dy.is_contiguous():
        raise ValueError("dy must be a contiguous (%s, width) tensor" % ", ".join(map(str, ids.shape)))
    if vocab < 0:
        raise ValueError("vocab must not be negative")
    width = dy.shape[-1]
    _u32("laplex_embedding_backward", vocab | width)
    dtype = (dy.dtype if dtable is None else dtable.dtype) if dtype is None else dtype
    if dtype not in (torch.float32, dy.dtype):
        raise TypeError("the table's gradient is float32 or of the type of dy")
    dtable = _out(dtable, "dtable", (vocab, width), dtype, dev)
    L = _lib()
    ws, ws_bytes = _bytes(ws, L.laplex_embedding_workspace_bytes(ids.numel(), vocab, width), dev)
    _check(L.laplex_embedding_backward(code, _ptr(ids), nb, ids.numel(), _ptr(dy), vocab, width, scale, _DTYPES[dtype],
                                       _ptr(dtable), _ptr(ws), ws_bytes, _stream_of(dev)), "laplex_embedding_backward")
    return dtable
