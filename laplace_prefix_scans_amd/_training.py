"""Binding of the training-step operators of liblaplex.so: gated linear recurrence, linear softmax cross entropy and
AdamW (declarations in include/laplex.h)."""
from __future__ import annotations

import array
import ctypes
from itertools import chain
from typing import Optional, Sequence, Tuple, Union

import torch

from ._binding import _check, _ptr
from ._layers import LAPLEX_BF16, LAPLEX_F32, _DTYPES, _bytes, _dtype, _ids, _like, _out, _stream_of, _u32
from ._layers import _lib as _layers_lib

LAPLEX_SCAN_CHUNK = 16
_KINDS = {"rate": 0, "sigmoid": 1}


class _Scan(ctypes.Structure):
    """laplex_scan_shape"""
    _fields_ = [("dtype", ctypes.c_int32), ("gate", ctypes.c_int32), ("seqs", ctypes.c_uint32), ("channels", ctypes.c_uint32),
                ("tokens", ctypes.c_uint64), ("offsets", ctypes.c_void_p), ("gate_token", ctypes.c_int64),
                ("x_token", ctypes.c_int64)]


class _AdamArgs(ctypes.Structure):
    """laplex_adamw_args"""
    _fields_ = [("dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("state_bits", ctypes.c_int32),
                ("stochastic", ctypes.c_int32), ("seed", ctypes.c_uint32), ("step", ctypes.c_uint64), ("lr", ctypes.c_double),
                ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double), ("step_dev", ctypes.c_void_p),
                ("lr_dev", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p)]


_ready = None


def _lib():
    global _ready
    if _ready is None:
        L = _layers_lib()
        vp, u64, u32, sz, i32, f32 = (ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_size_t, ctypes.c_int,
                                      ctypes.c_float)
        scan = ctypes.POINTER(_Scan)
        L.laplex_gated_scan_workspace_bytes.argtypes = [scan]
        L.laplex_gated_scan.argtypes = [scan] + [vp] * 7 + [sz, vp]
        L.laplex_gated_scan_backward.argtypes = [scan] + [vp] * 10 + [sz, vp]
        L.laplex_gated_scan_step.argtypes = [scan, vp, vp, vp, u32, vp, vp, vp]
        L.laplex_linear_cross_entropy_workspace_bytes.argtypes = [i32, i32, u64, u32, u32]
        L.laplex_linear_cross_entropy_workspace_bytes_aligned.argtypes = [i32, i32, u64, u32, u32]
        L.laplex_linear_cross_entropy.argtypes = [i32, vp, i32, u64, vp, vp, u32, u32, f32, vp, vp, vp, sz, vp]
        L.laplex_linear_cross_entropy_backward.argtypes = [i32, vp, i32, u64, vp, vp, u32, u32, f32, vp, vp, vp, vp, i32, vp, vp, sz, vp]
        L.laplex_adamw.argtypes = [ctypes.POINTER(_AdamArgs), vp, u32, vp]
        L.laplex_adamw_moments.argtypes = [vp, u32, vp]
        for f in (L.laplex_gated_scan_workspace_bytes, L.laplex_linear_cross_entropy_workspace_bytes,
                  L.laplex_linear_cross_entropy_workspace_bytes_aligned):
            f.restype = sz
        for f in (L.laplex_gated_scan, L.laplex_gated_scan_backward, L.laplex_gated_scan_step, L.laplex_linear_cross_entropy,
                  L.laplex_linear_cross_entropy_backward, L.laplex_adamw, L.laplex_adamw_moments):
            f.restype = i32
        _ready = L
    return _ready


def _run(where: str, dev: torch.device, f, *args) -> None:
    """f(*args, stream) on the device of its tensors, which need not be the current one."""
    if dev.index == torch.cuda.current_device():
        _check(f(*args, _stream_of(dev)), where)
    else:
        with torch.cuda.device(dev):
            _check(f(*args, _stream_of(dev)), where)


# ------------------------------------------------------------------ gated linear recurrence
def _token_stride(t: torch.Tensor, shape, name: str) -> int:
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError("%s must have contiguous channels" % name)
    if len(shape) == 2:
        return st[0]
    # (an axis of one token has no stride of its own: the batch's is the token's)
    if shape[0] > 1 and shape[1] > 1 and st[0] != shape[1] * st[1]:
        raise ValueError("%s: the tokens of a batch must lie one sequence after the other" % name)
    return st[0] if shape[1] == 1 else st[1]


def _scan(gate, x, kind: str, offsets) -> _Scan:
    code = _dtype(gate, "gate")
    if kind not in _KINDS:
        raise ValueError("kind must be 'rate' or 'sigmoid', got %r" % (kind,))
    dev, shape = gate.device, gate.shape
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch tensor")
    if x.dtype != gate.dtype or x.device != dev:
        raise TypeError("x must have the type and device of gate")
    if len(shape) not in (2, 3) or x.shape != shape or shape[-1] == 0:
        raise ValueError("gate and x must both be (tokens, channels) or (batch, tokens, channels): got %s and %s"
                         % (tuple(shape), tuple(x.shape)))
    batched = len(shape) == 3
    seqs, tokens = (shape[0], shape[0] * shape[1]) if batched else (1, shape[0])
    if offsets is not None:
        if batched:
            raise ValueError("offsets go with packed (tokens, channels) tensors")
        if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 1:
            raise ValueError("offsets must be a 1-D tensor of sequence starts and the end of the last")
        _like(offsets, "offsets", offsets.shape, torch.int32, dev)
        seqs = offsets.numel() - 1
    _u32("gated scan", seqs | shape[-1])
    return _Scan(code, _KINDS[kind], seqs, shape[-1], tokens, _ptr(offsets), _token_stride(gate, shape, "gate"),
                 _token_stride(x, shape, "x"))


def laplex_gated_scan_workspace_bytes(gate, x, kind: str = "rate", offsets=None) -> int:
    """Bytes of workspace of laplex_gated_scan and of its backward for these tensors."""
    return int(_lib().laplex_gated_scan_workspace_bytes(ctypes.byref(_scan(gate, x, kind, offsets))))


def laplex_gated_scan(gate: torch.Tensor, x: torch.Tensor, kind: str = "rate", offsets: Optional[torch.Tensor] = None,
                      state_in: Optional[torch.Tensor] = None, state_out: Optional[torch.Tensor] = None, keep: bool = False,
                      h: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """h_t = a_t h_{t-1} + w_t x_t over each sequence, per channel.

    kind "rate": a = exp(-gate), w = 1 (gate >= 0); "sigmoid": a = sigmoid(gate), w = 1 - a.  gate, x: (tokens,
    channels) float32 or bfloat16, channels contiguous; with a leading batch axis, sequences of equal length.  offsets:
    int32 (seqs + 1,), the packed sequences' starts and the last one's end.  state_in, state_out: (seqs, channels)
    float32, the states before the first tokens (None: zero) and, filled, after the last.  Returns h like x,
    contiguous; with keep=True also the carries (float32, a state for every LAPLEX_SCAN_CHUNK tokens) that
    laplex_gated_scan_backward reads."""
    s = _scan(gate, x, kind, offsets)
    dev = gate.device
    _like(state_in, "state_in", (s.seqs, s.channels), torch.float32, dev)
    _like(state_out, "state_out", (s.seqs, s.channels), torch.float32, dev)
    h = _out(h, "h", gate.shape, gate.dtype, dev)
    carries = torch.empty((_carries(s), s.channels), dtype=torch.float32, device=dev) if keep else None
    L = _lib()
    ws, ws_bytes = _bytes(ws, L.laplex_gated_scan_workspace_bytes(ctypes.byref(s)), dev)
    _run("laplex_gated_scan", dev, L.laplex_gated_scan, ctypes.byref(s), _ptr(gate), _ptr(x), _ptr(state_in), _ptr(state_out), _ptr(h),
         _ptr(carries), _ptr(ws), ws_bytes)
    return (h, carries) if keep else h


def _carries(s: _Scan) -> int:
    return -(-s.tokens // LAPLEX_SCAN_CHUNK)


def laplex_gated_scan_backward(gate: torch.Tensor, x: torch.Tensor, carries: torch.Tensor, dh: torch.Tensor, kind: str = "rate",
                               offsets: Optional[torch.Tensor] = None, state_in: Optional[torch.Tensor] = None,
                               dstate_out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """Backward of laplex_gated_scan for dh = dL/dh and dstate_out = dL/dstate_out (None: zero), from the carries of the
    forward call.  Returns (dgate, dx, dstate_in), the last (seqs, channels) float32, or None where state_in is None."""
    s = _scan(gate, x, kind, offsets)
    dev = gate.device
    if carries is None or dh is None:
        raise TypeError("carries and dh must be torch tensors")
    _like(carries, "carries", (_carries(s), s.channels), torch.float32, dev)
    _like(dh, "dh", gate.shape, gate.dtype, dev)
    _like(state_in, "state_in", (s.seqs, s.channels), torch.float32, dev)
    _like(dstate_out, "dstate_out", (s.seqs, s.channels), torch.float32, dev)
    dgate, dx = (torch.empty(gate.shape, dtype=gate.dtype, device=dev) for _ in range(2))
    dstate_in = torch.empty((s.seqs, s.channels), dtype=torch.float32, device=dev) if state_in is not None else None
    L = _lib()
    ws, ws_bytes = _bytes(ws, L.laplex_gated_scan_workspace_bytes(ctypes.byref(s)), dev)
    _run("laplex_gated_scan_backward", dev, L.laplex_gated_scan_backward, ctypes.byref(s), _ptr(gate), _ptr(x), _ptr(carries), _ptr(dh),
         _ptr(state_in), _ptr(dstate_out), _ptr(dgate), _ptr(dx), _ptr(dstate_in), _ptr(ws), ws_bytes)
    return dgate, dx, dstate_in


def laplex_gated_scan_step(gate: torch.Tensor, x: torch.Tensor, state: torch.Tensor, kind: str = "rate",
                           slots: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token for each row: its state becomes a state + w x in place, and is the row's output.

    gate, x: (rows, channels); state: (pool, channels) float32; slots: int32 (rows,), the state of each row (None: row r
    has state r).  A row whose slot is outside the pool has no sequence: its output is zero and no state changes.  Two
    rows must not share a slot."""
    if not isinstance(gate, torch.Tensor) or gate.dim() != 2:
        raise ValueError("gate must be (rows, channels)")
    s = _scan(gate, x, kind, None)
    dev, s.seqs = gate.device, gate.shape[0]
    _u32("laplex_gated_scan_step", gate.shape[0])
    if not isinstance(state, torch.Tensor) or state.dim() != 2:
        raise ValueError("state must be (pool, channels)")
    _like(state, "state", (state.shape[0], s.channels), torch.float32, dev)
    _like(slots, "slots", (s.seqs,), torch.int32, dev)
    _u32("laplex_gated_scan_step", state.shape[0])
    if slots is None and s.seqs > state.shape[0]:
        raise ValueError("state must have a row for each of the %d tokens" % s.seqs)
    h = _out(h, "h", gate.shape, gate.dtype, dev)
    _run("laplex_gated_scan_step", dev, _lib().laplex_gated_scan_step, ctypes.byref(s), _ptr(gate), _ptr(x), _ptr(slots), state.shape[0],
         _ptr(state), _ptr(h))
    return h


# ------------------------------------------------------------------ linear softmax cross entropy
def _xent(x, table, targets) -> Tuple[int, int, int, int, int]:
    code = _dtype(x, "x")
    dev = x.device
    if not isinstance(table, torch.Tensor):
        raise TypeError("table must be a torch tensor")
    if table.dtype != x.dtype or table.device != dev:
        raise TypeError("table must have the type and device of x")
    nb = _ids(targets, dev)
    if table.dim() != 2 or 0 in table.shape or not table.is_contiguous():
        raise ValueError("table must be a contiguous (vocab, width) tensor")
    vocab, width = table.shape
    if x.dim() != targets.dim() + 1 or x.shape[:-1] != targets.shape or x.shape[-1] != width or not x.is_contiguous():
        raise ValueError("x must be a contiguous (%s) tensor" % ", ".join(map(str, (*targets.shape, width))))
    _u32("linear cross entropy", vocab | width)
    return code, nb, targets.numel(), vocab, width


def _xent_bytes(backward: bool, x, table, code: int, tokens: int, vocab: int, width: int) -> int:
    L = _lib()
    f = L.laplex_linear_cross_entropy_workspace_bytes
    if (x.data_ptr() | table.data_ptr()) % 16 == 0:
        f = L.laplex_linear_cross_entropy_workspace_bytes_aligned
    return int(f(1 if backward else 0, code, tokens, vocab, width))


def laplex_linear_cross_entropy_workspace_bytes(backward: bool, x: torch.Tensor, table: torch.Tensor, targets: torch.Tensor) -> int:
    """Bytes of workspace of laplex_linear_cross_entropy (or its backward) for these tensors: also for fewer tokens, and
    for other tensors of these sizes, but that where x and table begin at multiples of 16 bytes, they have to as well."""
    code, _, tokens, vocab, width = _xent(x, table, targets)
    return _xent_bytes(backward, x, table, code, tokens, vocab, width)


def laplex_linear_cross_entropy(x: torch.Tensor, table: torch.Tensor, targets: torch.Tensor, scale: float = 1.0,
                                ws: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(loss, lse), float32 in the shape of targets: with logits l = scale x table^T, lse = log sum exp l and loss = lse -
    l_target.  The logits are not kept.  x: (*targets.shape, width); table: (vocab, width) of the same type; targets:
    int32 or int64.  A target outside the vocabulary leaves its token out: its loss and lse are zero."""
    code, nb, tokens, vocab, width = _xent(x, table, targets)
    dev = x.device
    loss, lse = torch.empty((2, *targets.shape), dtype=torch.float32, device=dev).unbind(0)
    L = _lib()
    ws, ws_bytes = _bytes(ws, _xent_bytes(False, x, table, code, tokens, vocab, width), dev)
    _run("laplex_linear_cross_entropy", dev, L.laplex_linear_cross_entropy, code, _ptr(targets), nb, tokens, _ptr(x), _ptr(table), vocab,
         width, scale, _ptr(loss), _ptr(lse), _ptr(ws), ws_bytes)
    return loss, lse


def laplex_linear_cross_entropy_backward(x: torch.Tensor, table: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                                         dloss: torch.Tensor, dlse: Optional[torch.Tensor] = None, scale: float = 1.0,
                                         x_grad: bool = True, table_grad: bool = True, dtype: Optional[torch.dtype] = None,
                                         ws: Optional[torch.Tensor] = None):
    """(dx, dtable) of laplex_linear_cross_entropy for dloss = dL/dloss and dlse = dL/dlse (None: zero), from the lse of
    the forward call.  dtype: of dtable, float32 or the type of the table (the default).  None in the place of a
    gradient that is not asked for."""
    code, nb, tokens, vocab, width = _xent(x, table, targets)
    dev = x.device
    if lse is None or dloss is None:
        raise TypeError("lse and dloss must be torch tensors")
    for t, name in ((lse, "lse"), (dloss, "dloss"), (dlse, "dlse")):
        _like(t, name, targets.shape, torch.float32, dev)
    dtype = x.dtype if dtype is None else dtype
    if dtype not in (torch.float32, x.dtype):
        raise TypeError("the table's gradient is float32 or of the table's type")
    dx = torch.empty_like(x) if x_grad else None
    dtable = torch.empty((vocab, width), dtype=dtype, device=dev) if table_grad else None
    L = _lib()
    ws, ws_bytes = _bytes(ws, _xent_bytes(True, x, table, code, tokens, vocab, width), dev)
    _run("laplex_linear_cross_entropy_backward", dev, L.laplex_linear_cross_entropy_backward, code, _ptr(targets), nb, tokens, _ptr(x),
         _ptr(table), vocab, width, scale, _ptr(lse), _ptr(dloss), _ptr(dlse), _ptr(dx), _DTYPES[dtype], _ptr(dtable), _ptr(ws), ws_bytes)
    return dx, dtable


# ------------------------------------------------------------------ AdamW
def _list(name: str, ts, count: int, dtype, dev, sizes):
    """The pointers of `count` contiguous tensors of a type and of these numbers of elements."""
    if len(ts) != count:
        raise ValueError("%s must have a tensor for each of the %d parameters, got %d" % (name, count, len(ts)))
    at, got = dev.index, []
    try:
        for t, n in zip(ts, sizes):
            if t.dtype is not dtype:
                raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
            if t.numel() != n or t.get_device() != at or not t.is_contiguous():
                raise ValueError("%s must be contiguous, on %s and of its parameter's size" % (name, dev))
            got.append(t.data_ptr())
    except AttributeError:
        raise TypeError("%s must hold torch tensors" % name) from None
    return got


def _bits(m) -> int:
    kind = m[0].dtype
    if kind is torch.float32:
        return 32
    if kind in (torch.float8_e4m3fn, torch.uint8):
        return 8
    raise TypeError("moments must be float32, or e4m3 codes (float8_e4m3fn or uint8), got %s" % kind)


def laplex_adamw(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], m: Sequence[torch.Tensor], v: Sequence[torch.Tensor], *,
                 lr: Union[float, torch.Tensor], step: Union[int, torch.Tensor], betas: Tuple[float, float] = (0.9, 0.999),
                 eps: float = 1e-8, weight_decay: Union[float, Sequence[float]] = 0.0,
                 m_scale: Optional[Sequence[torch.Tensor]] = None, v_scale: Optional[Sequence[torch.Tensor]] = None,
                 master: Optional[Sequence[torch.Tensor]] = None, grad_scale: Optional[torch.Tensor] = None,
                 seed: Optional[int] = None) -> None:
    """One AdamW step over a list of parameters, in place.

    params and grads: float32 or bfloat16, one type each.  m, v: the moments, zero before the first step: float32, or
    e4m3 codes (float8_e4m3fn or uint8) of m and of sqrt(v) with m_scale and v_scale, float32 tensors of ceil(n / 256)
    scales.  master: float32 copies of the parameters, which are then what is updated.  step: 1 for the first; step and lr
    may be device tensors of one int32 and one float32 (for captured graphs).  weight_decay: a number, or one for each
    parameter.  grad_scale: a device float32 that every gradient is multiplied by; where it is not finite, nothing is
    changed.  seed: of the random bits that 8-bit moments are rounded with (None: to nearest)."""
    count = len(params)
    if not (len(grads) == len(m) == len(v) == count):
        raise ValueError("params, grads, m and v must be as many")
    if count == 0:
        return
    _dtype(params[0], "params")
    dev = params[0].device
    bits = _bits(m)
    if (m_scale is not None and v_scale is not None) != (bits == 8) or (m_scale is None) != (v_scale is None):
        raise ValueError("m_scale and v_scale go with 8-bit moments")
    sizes = [p.numel() for p in params]
    blocks = [-(-n // 256) for n in sizes] if bits == 8 else sizes
    code = _dtype(params[0], "params")
    zero = [0] * count
    decay = [float(weight_decay)] * count if isinstance(weight_decay, (int, float)) else [float(w) for w in weight_decay]
    if len(decay) != count:
        raise ValueError("weight_decay must be a number, or one for each parameter")
    if not isinstance(grads[0], torch.Tensor) or grads[0].dtype not in _DTYPES:
        raise TypeError("grads must be float32 or bfloat16 tensors")
    columns = (_list("params", params, count, params[0].dtype, dev, sizes), _list("grads", grads, count, grads[0].dtype, dev, sizes),
               _list("m", m, count, m[0].dtype, dev, sizes), _list("v", v, count, m[0].dtype, dev, sizes),
               _list("m_scale", m_scale, count, torch.float32, dev, blocks) if bits == 8 else zero,
               _list("v_scale", v_scale, count, torch.float32, dev, blocks) if bits == 8 else zero,
               _list("master", master, count, torch.float32, dev, sizes) if master is not None else zero,
               sizes, array.array("I", array.array("f", decay).tobytes()))
    table = array.array("Q", chain.from_iterable(zip(*columns)))  # laplex_adamw_tensor, field by field
    step_dev, lr_dev = isinstance(step, torch.Tensor), isinstance(lr, torch.Tensor)
    if step_dev:
        _scalar(step, "step", torch.int32, dev)
    elif step < 1:
        raise ValueError("step must be at least 1")
    if lr_dev:
        _scalar(lr, "lr", torch.float32, dev)
    if grad_scale is not None:
        _scalar(grad_scale, "grad_scale", torch.float32, dev)
    args = _AdamArgs(code, _DTYPES[grads[0].dtype], bits, 0 if seed is None else 1, (seed or 0) & 0xFFFFFFFF, 1 if step_dev else step,
                     0.0 if lr_dev else lr, betas[0], betas[1], eps, _ptr(step) if step_dev else None, _ptr(lr) if lr_dev else None,
                     _ptr(grad_scale))
    _run("laplex_adamw", dev, _lib().laplex_adamw, ctypes.byref(args), table.buffer_info()[0], count)


def _scalar(t, name: str, dtype, dev) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.numel() != 1:
        raise TypeError("%s on the device must be one %s" % (name, dtype))
    if t.device != dev:
        raise ValueError("%s must be on %s" % (name, dev))


def laplex_adamw_moments(m: Sequence[torch.Tensor], v: Sequence[torch.Tensor], m_scale: Sequence[torch.Tensor],
                         v_scale: Sequence[torch.Tensor], m_out: Optional[Sequence[torch.Tensor]] = None,
                         v_out: Optional[Sequence[torch.Tensor]] = None):
    """(m_out, v_out): the float32 values that the 8-bit moments of laplex_adamw stand for, in lists of tensors."""
    count = len(m)
    if count == 0:
        return [], []
    if _bits(m) != 8:
        raise TypeError("moments must be e4m3 codes")
    if not m[0].is_cuda:
        raise ValueError("moments must be on a GPU device")
    dev, sizes = m[0].device, [t.numel() for t in m]
    blocks = [-(-n // 256) for n in sizes]
    m_out = [torch.empty(t.shape, dtype=torch.float32, device=dev) for t in m] if m_out is None else m_out
    v_out = [torch.empty(t.shape, dtype=torch.float32, device=dev) for t in v] if v_out is None else v_out
    zero = [0] * count
    columns = (_list("m_out", m_out, count, torch.float32, dev, sizes), zero, _list("m", m, count, m[0].dtype, dev, sizes),
               _list("v", v, count, m[0].dtype, dev, sizes), _list("m_scale", m_scale, count, torch.float32, dev, blocks),
               _list("v_scale", v_scale, count, torch.float32, dev, blocks),
               _list("v_out", v_out, count, torch.float32, dev, sizes), sizes, zero)
    table = array.array("Q", chain.from_iterable(zip(*columns)))
    _run("laplex_adamw_moments", dev, _lib().laplex_adamw_moments, table.buffer_info()[0], count)
    return m_out, v_out
