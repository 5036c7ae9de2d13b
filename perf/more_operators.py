"""Cases of three more operators of a sequence model's training step: the gated linear recurrence, the softmax cross entropy
of a linear output table, and the AdamW update of many tensors.

Each case is one pass through one operator as a training step, a prompt or a decoding step calls it.  ``own`` false computes
it in plain torch operations in 32 bits; ``own`` true calls laplace_prefix_scans_amd.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BLOCK = 256  # values that share a scale in an 8-bit state
LR, BETA1, BETA2, EPS, DECAY, STEP, SEED = 3e-4, 0.9, 0.95, 1e-8, 0.1, 1000, 12345


# ------------------------------------------------------------------ cases
# scan: `seqs` sequences of `tokens` tokens in all (ragged: packed, of different lengths, some empty or one token long; else
# equal lengths), `channels` channels.  gate: "rate" (decay exp(-r)) or "sigmoid" (decay and input weight from one logit).
# train: forward and backward; states: an initial state comes in and the final one goes out.
# step: one token for each of `seqs` sequences whose states lie in a pool, updated in place.
# ce: `tokens` rows of `width` against a `vocab` x `width` table; train: with the gradients of both.
# adamw: the tensors of a model of `layers` blocks of `width` and a `vocab` x `width` table; parameters of type `dtype`, gradients
# of the same, states of `bits` bits; master: a float32 copy of bfloat16 parameters is what is updated.
def listed():
    return [
        # one user's next token: a call whose latency is all that counts
        {"name": "scan_step_one_f32", "op": "step", "dtype": "f32", "gate": "rate", "seqs": 1, "channels": 513},
        # a full decoding batch of a wide layer with some of its places free
        {"name": "scan_step_batch_bf16", "op": "step", "dtype": "bf16", "gate": "sigmoid", "seqs": 256, "channels": 8192},
        # one very long document of a narrow layer: few rows to spread over the chip, so the time axis is what is split
        {"name": "scan_long_f32", "op": "scan", "dtype": "f32", "gate": "rate", "seqs": 1, "tokens": 65536, "channels": 256,
         "ragged": False, "train": False, "states": False},
        # packed documents of an odd width, gradients through their states
        {"name": "scan_packed_f32", "op": "scan", "dtype": "f32", "gate": "sigmoid", "seqs": 23, "tokens": 16411, "channels": 1001,
         "ragged": True, "train": True, "states": True},
        # an ordinary pre-training micro-batch
        {"name": "scan_train_bf16", "op": "scan", "dtype": "bf16", "gate": "sigmoid", "seqs": 8, "tokens": 16384, "channels": 4096,
         "ragged": False, "train": True, "states": False},
        # the likelihood of one token against a whole vocabulary: reading the table is all there is to it
        {"name": "ce_one_bf16", "op": "ce", "dtype": "bf16", "tokens": 1, "vocab": 65536, "width": 2048, "train": False},
        # scoring a document
        {"name": "ce_score_bf16", "op": "ce", "dtype": "bf16", "tokens": 2043, "vocab": 65536, "width": 2048, "train": False},
        # a small model in single precision with a vocabulary of bytes and an odd width
        {"name": "ce_train_f32", "op": "ce", "dtype": "f32", "tokens": 4096, "vocab": 257, "width": 513, "train": True},
        # an ordinary pre-training micro-batch
        {"name": "ce_train_bf16", "op": "ce", "dtype": "bf16", "tokens": 16384, "vocab": 65536, "width": 2048, "train": True},
        # a small model's step: many small tensors, so launches and the host count
        {"name": "adamw_small_f32", "op": "adamw", "dtype": "f32", "layers": 2, "width": 256, "vocab": 64, "bits": 32, "master": False},
        # a large model's step, parameters in bfloat16 beside their float32 copies
        {"name": "adamw_large_bf16", "op": "adamw", "dtype": "bf16", "layers": 8, "width": 2048, "vocab": 65536, "bits": 32,
         "master": True},
        # states in 8 bits, and tensors that end inside a block of them
        {"name": "adamw_8bit_bf16", "op": "adamw", "dtype": "bf16", "layers": 6, "width": 1001, "vocab": 32771, "bits": 8,
         "master": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_once(rng):
    op = rng.choice(["scan", "scan", "step", "ce", "ce", "adamw"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "ce":
        return {"op": op, "dtype": dtype, "tokens": _log_int(rng, 1, 32768), "vocab": _log_int(rng, 64, 131072),
                "width": _log_int(rng, 32, 4096), "train": rng.random() < 0.6}
    if op == "adamw":
        return {"op": op, "dtype": dtype, "layers": rng.randint(1, 12), "width": _log_int(rng, 24, 2500),
                "vocab": _log_int(rng, 64, 70000), "bits": rng.choice([8, 32]), "master": dtype == "bf16" and rng.random() < 0.5}
    gate, channels = rng.choice(["rate", "sigmoid"]), _log_int(rng, 16, 8192)
    if op == "step":
        return {"op": op, "dtype": dtype, "gate": gate, "seqs": _log_int(rng, 1, 512), "channels": channels}
    seqs = _log_int(rng, 1, 32)
    ragged = rng.random() < 0.6
    tokens = max(seqs, _log_int(rng, 1, 65536))
    if not ragged:
        tokens -= tokens % seqs
    return {"op": op, "dtype": dtype, "gate": gate, "seqs": seqs, "tokens": tokens, "channels": channels, "ragged": ragged,
            "train": rng.random() < 0.6, "states": rng.random() < 0.5}


def draw(rng):
    top = {}
    for c in listed():  # the most of any listed case of the operator
        w, kind = work(c), "scan" if c["op"] == "step" else c["op"]
        top[kind] = {m: max(w[m], top.get(kind, w)[m]) for m in ("bytes", "flops")}
    while True:
        c = _draw_once(rng)
        w, most = work(c), top["scan" if c["op"] == "step" else c["op"]]
        # float products take many times as long as bfloat16's
        cost = w["flops"] * (8 if c["op"] == "ce" and c["dtype"] == "f32" else 1)
        if w["bytes"] <= most["bytes"] and cost <= most["flops"]:
            return c


def _sizes(case):
    """Shapes of the model's tensors, and which of them decay."""
    w, got = case["width"], [((case["vocab"], case["width"]), True)]
    for _ in range(case["layers"]):
        got += [((w,), False)] * 4 + [((w, 3 * w), True), ((w, w), True), ((w, 4 * w), True), ((2 * w, w), True)]
    return got + [((w,), False)] * 2


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "adamw":
        n = sum(math.prod(s) for s, _ in _sizes(case))
        # 8 bits: codes and scales of both states read and written, and the values they stand for written
        state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK + 8
        return {"bytes": n * (3 * e - (e if case["master"] else 0) + state + (8 if case["master"] else 0)), "flops": 16 * n}
    if case["op"] == "ce":
        t, v, d = case["tokens"], case["vocab"], case["width"]
        mats, rows = e * (t * d + v * d), 16 * t
        return {"bytes": mats * (3 if case["train"] else 1) + rows, "flops": (8 if case["train"] else 2) * t * v * d}
    c, n = case["channels"], case["seqs"]
    t = n if case["op"] == "step" else case["tokens"]
    if case["op"] == "step":
        return {"bytes": 3 * e * t * c + 8 * n * c, "flops": 10 * t * c}
    states = 8 * n * c if case["states"] else 0
    if not case["train"]:
        return {"bytes": 3 * e * t * c + states, "flops": 10 * t * c}
    return {"bytes": 8 * e * t * c + 2 * states, "flops": 30 * t * c}


# ------------------------------------------------------------------ inputs
def _lengths(case, seed):
    """Lengths of packed sequences: spread over about a factor of ten, one empty and one of one token where there are enough."""
    n, t = case["seqs"], case["tokens"]
    if not case["ragged"]:
        return np.full(n, t // n, dtype=np.int64)
    r = np.random.default_rng([seed, 13])
    fixed = [0, 1] if n >= 4 else []
    share = np.exp(r.uniform(0, math.log(10.0), n - len(fixed)))
    cut = np.floor(np.concatenate([[0.0], np.cumsum(share)]) / share.sum() * (t - sum(fixed)) + 0.5).astype(np.int64)
    return r.permutation(np.concatenate([np.diff(cut), np.array(fixed, dtype=np.int64)]))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return torch.randn(shape, generator=g, device=dev).mul_(std).add_(mean).to(dtype)

    s = {"case": case}
    if case["op"] == "adamw":
        return _prepare_adamw(case, s, normal)
    if case["op"] == "ce":
        t, v, d = case["tokens"], case["vocab"], case["width"]
        s["table"] = normal(v, d, std=2.0 * d ** -0.5)  # logits spread by about 2
        # word frequencies fall off like 1 / rank; some places are padding (-1)
        u = torch.rand(t, generator=g, device=dev, dtype=torch.float64)
        rank = torch.clamp((torch.exp(u * math.log(v + 1.0)) - 1.0).long(), max=v - 1)
        ids = torch.randperm(v, generator=g, device=dev)[rank]
        # rows that lean towards their targets, from not at all to certainty; a few rows alone do not, so that their losses are
        # not all differences of nearly equal numbers
        lean = torch.rand(t, 1, generator=g, device=dev) * (5.0 if t >= 64 else 0.0)
        s["x"] = (normal(t, d, dtype=torch.float32) + lean * s["table"][ids].float()).to(dt)
        if t > 1:
            ids[torch.rand(t, generator=g, device=dev) < 0.02] = -1
        s["ids"] = ids
        s["dloss"] = (torch.rand(t, generator=g, device=dev) + 0.5) / t  # a mean with weights
        return s
    c, n = case["channels"], case["seqs"]

    def gates(rows):
        # memories from a few tokens to thousands, spread over the channels, moved by the data
        memory = torch.exp(torch.linspace(math.log(2.0), math.log(4000.0), c, device=dev))
        if case["gate"] == "rate":
            return (torch.exp(0.7 * torch.randn(rows, c, generator=g, device=dev)) / memory).to(dt)
        return (torch.log(memory) + 1.5 * torch.randn(rows, c, generator=g, device=dev)).to(dt)

    if case["op"] == "step":
        pool = n + n // 8 + 1
        s["slots"] = torch.randperm(pool - 1, generator=g, device=dev)[:n].to(torch.int32)
        if n >= 8:  # places of the batch with no request
            s["slots"][:: 8] = -1
        s.update(gate=gates(n), x=normal(n, c), state=normal(pool, c, dtype=torch.float32))
        return s
    t = case["tokens"]
    lengths = _lengths(case, seed)
    s["offsets"] = None
    if case["ragged"]:
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)).to(dev)
    s.update(gate=gates(t), x=normal(t, c), dh=normal(t, c))
    s["state_in"] = normal(n, c, dtype=torch.float32) if case["states"] else None
    s["dstate_out"] = normal(n, c, dtype=torch.float32) if case["states"] else None
    if not case["ragged"]:  # equal lengths: a batch axis
        for name in ("gate", "x", "dh"):
            s[name] = s[name].view(n, t // n, c)
    return s


def _prepare_adamw(case, s, normal):
    """Tensors that are slices of one buffer of each kind, each from a multiple of BLOCK on, and zeros between them."""
    dev, dt = torch.device("cuda"), DTYPES[case["dtype"]]
    shapes = _sizes(case)
    blocks = np.array([-(-math.prod(x) // BLOCK) for x, _ in shapes])
    first = np.concatenate([[0], np.cumsum(blocks)])
    total = int(first[-1])
    s["tensor_of"] = torch.from_numpy(np.repeat(np.arange(len(shapes)), blocks)).to(dev)  # of each block
    s["block_of"] = torch.arange(total, device=dev) - torch.from_numpy(first[:-1]).to(dev)[s["tensor_of"]]
    s["decays"] = [DECAY if x else 0.0 for _, x in shapes]
    sizes = torch.tensor([math.prod(x) for x, _ in shapes], device=dev)
    s["inside"] = (s["block_of"][:, None] * BLOCK + torch.arange(BLOCK, device=dev) < sizes[s["tensor_of"]][:, None]).view(-1)

    def whole(std, kind=torch.float32):
        return torch.where(s["inside"], normal(total * BLOCK, std=std, dtype=torch.float32), 0.0).to(kind)

    def slices(flat, by=BLOCK):
        if by == 1:
            return [flat[a:a + b] for a, b in zip(first, blocks)]
        return [flat[a * by:a * by + math.prod(x)].view(x) for a, (x, _) in zip(first, shapes)]

    f = {"p": whole(0.02), "g": whole(1e-3, dt)}
    if case["master"]:
        f["master"] = f["p"]
    f["p"] = f["p"].to(dt)
    m, v = whole(3e-4), whole(1e-3).square_().add_(1e-8).mul_(s["inside"])
    if case["bits"] == 32:
        f["m"], f["v"] = m, v
    else:
        for name, x in (("m", m), ("v", v.sqrt())):
            x = x.view(total, BLOCK)
            f[name + "_scale"] = x.abs().amax(1) / 448.0
            f[name] = (x / f[name + "_scale"].clamp(min=1e-30)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(-1)
        f["m_out"], f["v_out"] = torch.zeros(2, total * BLOCK, device=dev).unbind(0)  # the values that the codes stand for
    s["flat"] = f
    s["lists"] = {k: slices(x, 1 if k.endswith("_scale") else BLOCK) for k, x in f.items()}
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return {"scan": _scan, "step": _step, "ce": _ce, "adamw": _adamw}[state["case"]["op"]](state)


def _decay(gate, kind):
    """(decay of the state, weight of the input)"""
    if kind == "rate":
        return torch.exp(-gate), torch.ones_like(gate)
    return torch.sigmoid(gate), torch.sigmoid(-gate)


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t from zero, over the first axis: stretches of 1, 2, 4, ... tokens joined."""
    s = 1
    while s < a.shape[0]:
        b = torch.cat([b[:s], b[s:] + a[s:] * b[:-s]])
        a = torch.cat([a[:s], a[s:] * a[:-s]])
        s *= 2
    return b


def _scan(s):
    c = s["case"]
    if own:
        import laplace_prefix_scans_amd as lp
        state_out = torch.empty_like(s["state_in"]) if c["states"] else None
        if not c["train"]:
            out = {"h": lp.laplex_gated_scan(s["gate"], s["x"], c["gate"], offsets=s["offsets"], state_in=s["state_in"],
                                             state_out=state_out)}
        else:
            h, carries = lp.laplex_gated_scan(s["gate"], s["x"], c["gate"], offsets=s["offsets"], state_in=s["state_in"],
                                              state_out=state_out, keep=True)
            dgate, dx, dstate_in = lp.laplex_gated_scan_backward(s["gate"], s["x"], carries, s["dh"], c["gate"],
                                                                 offsets=s["offsets"], state_in=s["state_in"],
                                                                 dstate_out=s["dstate_out"])
            out = {"h": h, "dgate": dgate, "dx": dx}
            if c["states"]:
                out["dstate_in"] = dstate_in
        if c["states"]:
            out["state_out"] = state_out
        return out
    shape, dt, n, ch = s["x"].shape, s["x"].dtype, c["seqs"], c["channels"]
    gate, x = s["gate"].reshape(-1, ch).float(), s["x"].reshape(-1, ch).float()
    t, dev = x.shape[0], x.device
    bounds = torch.arange(n + 1, device=dev) * (t // n) if s["offsets"] is None else s["offsets"].long()
    lengths = bounds.diff()
    token = torch.arange(t, device=dev)
    seq = torch.searchsorted(bounds[1:].contiguous(), token, right=True)
    starts, ends = (token == bounds[seq])[:, None], (token == bounds[seq + 1] - 1)[:, None]
    a, w = _decay(gate, c["gate"])
    # each sequence's first token takes the initial state in the place of the token before
    initial = s["state_in"][seq] if c["states"] else torch.zeros_like(x)
    h = _doubling(torch.where(starts, 0.0, a), w * x + torch.where(starts, a * initial, 0.0))
    out = {"h": h.to(dt).view(shape)}
    first, last = bounds[:-1].clamp(max=t - 1), (bounds[1:] - 1).clamp(min=0)
    empty = (lengths == 0)[:, None]
    if c["states"]:
        out["state_out"] = torch.where(empty, s["state_in"], h[last])
    if c["train"]:
        dh = s["dh"].reshape(-1, ch).float()
        if c["states"]:
            dh = dh + torch.where(ends, s["dstate_out"][seq], 0.0)
        after = torch.cat([a[1:], torch.zeros_like(a[:1])])
        lam = _doubling(torch.where(ends, 0.0, after).flip(0), dh.flip(0)).flip(0)
        before = torch.where(starts, initial, torch.cat([torch.zeros_like(h[:1]), h[:-1]]))
        dgate = -a * before * lam if c["gate"] == "rate" else a * w * (before - x) * lam
        out.update(dgate=dgate.to(dt).view(shape), dx=(w * lam).to(dt).view(shape))
        if c["states"]:
            out["dstate_in"] = torch.where(empty, s["dstate_out"], (a * lam)[first])
    return out


def _step(s):
    c = s["case"]
    if own:
        import laplace_prefix_scans_amd as lp
        h = lp.laplex_gated_scan_step(s["gate"], s["x"], s["state"], c["gate"], slots=s["slots"])
        return {"h": h, "state": s["state"]}
    slot = s["slots"].long()
    live = (slot >= 0)[:, None]
    a, w = _decay(s["gate"].float(), c["gate"])
    new = a * s["state"][slot.clamp(min=0)] + w * s["x"].float()
    # the pool's last row is nobody's: a place without a request puts there what is there already
    s["state"].index_copy_(0, torch.where(live.view(-1), slot, s["state"].shape[0] - 1), torch.where(live, new, s["state"][-1]))
    return {"h": torch.where(live, new, 0.0).to(s["x"].dtype), "state": s["state"]}


def _ce(s):
    c = s["case"]
    if own:
        import laplace_prefix_scans_amd as lp
        loss, lse = lp.laplex_linear_cross_entropy(s["x"], s["table"], s["ids"])
        out = {"loss": loss, "lse": lse}
        if c["train"]:
            out["dx"], out["dtable"] = lp.laplex_linear_cross_entropy_backward(s["x"], s["table"], s["ids"], lse, s["dloss"])
        return out
    live = s["ids"] >= 0
    at = s["ids"].clamp(min=0)[:, None]
    x, table = torch.where(live[:, None], s["x"].float(), 0.0), s["table"].float()
    logits = x @ table.t()
    most = logits.amax(1, keepdim=True)
    lse = most + torch.log(torch.exp(logits - most).sum(1, keepdim=True))
    out = {"loss": torch.where(live, (lse - logits.gather(1, at))[:, 0], 0.0), "lse": torch.where(live, lse[:, 0], 0.0)}
    if c["train"]:
        weight = torch.where(live, s["dloss"], 0.0)[:, None]
        grad = torch.exp(logits - lse) * weight
        grad.scatter_add_(1, at, -weight)
        out.update(dx=(grad @ table).to(s["x"].dtype), dtable=(grad.t().contiguous() @ x).to(s["x"].dtype))
    return out


def _mix(x):
    """MurmurHash3's 32-bit finalizer (public domain), on int64 values below 2^32."""
    x = ((x ^ (x >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    x = ((x ^ (x >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _codes(x, bits):
    """(codes, scales) of blocks of x: e4m3 magnitudes rounded up with the probability that 16 random bits give them."""
    most = x.abs().amax(1)
    scale = most / torch.full_like(most, 448.0)
    y = (x.abs() * torch.where(most > 0, torch.full_like(most, 448.0) / most, 0.0)[:, None]).clamp(max=448.0)
    small = y < 2.0 ** -6  # multiples of 2^-9: those from 2^-6 on, 2^-6 higher
    t = torch.where(small, y + 2.0 ** -6, y)
    code = ((t.view(torch.int32).long() + (bits << 4)) >> 20) - 960 - 8 * small.long()
    return code, scale


def _adamw(s):
    c, f, q = s["case"], s["flat"], s["lists"]
    eight = c["bits"] == 8
    if own:
        import laplace_prefix_scans_amd as lp
        lp.laplex_adamw(q["p"], q["g"], q["m"], q["v"], lr=LR, step=STEP, betas=(BETA1, BETA2), eps=EPS,
                        weight_decay=s["decays"], m_scale=q.get("m_scale"), v_scale=q.get("v_scale"), master=q.get("master"),
                        seed=SEED if eight else None)
        if eight:
            lp.laplex_adamw_moments(q["m"], q["v"], q["m_scale"], q["v_scale"], m_out=q["m_out"], v_out=q["v_out"])
            return {"p": f["p"], "m": f["m_out"], "v": f["v_out"]}
        return {k: f[k] for k in ("p", "m", "v", "master") if k in f}
    f32 = lambda x: torch.full((), x, device="cuda")  # noqa: E731  (constants rounded to float32 first)
    g = f["g"].float()
    if eight:
        m = f["m"].float().view(-1, BLOCK) * f["m_scale"][:, None]
        root = f["v"].float().view(-1, BLOCK) * f["v_scale"][:, None]
        m, v = m.view(-1), (root * root).view(-1)
    else:
        m, v = f["m"], f["v"]
    m = f32(BETA1) * m + f32(1 - BETA1) * g
    v = f32(BETA2) * v + f32(1 - BETA2) * (g * g)
    decay = torch.tensor([1 - LR * x for x in s["decays"]], device="cuda")[s["tensor_of"]].repeat_interleave(BLOCK)
    p = f["master"] if c["master"] else f["p"].float()
    rate, root_c2 = f32(LR / (1 - BETA1 ** STEP)), f32(math.sqrt(1 - BETA2 ** STEP))
    p = p * decay - rate * m / (torch.sqrt(v) / root_c2 + f32(EPS))
    f["p"].copy_(p)
    if c["master"]:
        f["master"].copy_(p)
    if not eight:
        m, v = f["m"].copy_(m), f["v"].copy_(v)
        return {k: f[k] for k in ("p", "m", "v", "master") if k in f}
    key = _mix((_mix((s["tensor_of"] * 0x9E3779B9 + STEP) & 0xFFFFFFFF)) ^ SEED)
    index = s["block_of"][:, None] * BLOCK + torch.arange(BLOCK, device="cuda")
    bits = _mix(index ^ key[:, None])
    m, root = m.view(-1, BLOCK), torch.sqrt(v).view(-1, BLOCK)
    cm, f["m_scale"][:] = _codes(m, bits & 0xFFFF)
    cv, f["v_scale"][:] = _codes(root, bits >> 16)
    cv = torch.where((root > 0) & (cv == 0), 1, cv)  # a second moment that is not zero stays so
    f["m"].view(torch.uint8).copy_((cm + 128 * (m < 0)).view(-1))
    f["v"].view(torch.uint8).copy_(cv.view(-1))
    inside = s["inside"].view(-1, BLOCK)
    f["m_out"].copy_(torch.where(inside, f["m"].float().view(-1, BLOCK) * f["m_scale"][:, None], 0.0).view(-1))
    root = f["v"].float().view(-1, BLOCK) * f["v_scale"][:, None]
    f["v_out"].copy_(torch.where(inside, root * root, 0.0).view(-1))
    return {"p": f["p"], "m": f["m_out"], "v": f["v_out"]}


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    return {"scan": _exact_scan, "step": _exact_step, "ce": _exact_ce, "adamw": _exact_adamw}[case["op"]](s)


def _exact_decay(s):
    z = s["gate"].reshape(-1, s["case"]["channels"]).double()
    if s["case"]["gate"] == "rate":
        return 1.0 / torch.exp(z), torch.ones_like(z), None
    up = torch.exp(z)
    return up / (1.0 + up), 1.0 / (1.0 + up), up / (1.0 + up) ** 2  # decay, weight, slope of the decay


def _exact_scan(s):
    """One token after the other."""
    c = s["case"]
    n, ch, t = c["seqs"], c["channels"], c["tokens"]
    a, w, slope = _exact_decay(s)
    x, dh = (s[y].reshape(-1, ch).double() for y in ("x", "dh"))
    wx = w * x
    bounds = [i * (t // n) for i in range(n + 1)] if s["offsets"] is None else s["offsets"].tolist()
    zero = torch.zeros(n, ch, dtype=torch.float64, device="cuda")
    initial = s["state_in"].double() if c["states"] else zero
    h, before, lam = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    finals, firsts = initial.clone(), (s["dstate_out"].double() if c["states"] else zero.clone())
    for q in range(n):
        state = initial[q]
        for i in range(bounds[q], bounds[q + 1]):
            before[i] = state
            state = torch.addcmul(wx[i], a[i], state, out=h[i])
        finals[q] = state
        if c["train"]:
            mu = firsts[q]
            for i in reversed(range(bounds[q], bounds[q + 1])):
                mu = a[i] * torch.add(dh[i], mu, out=lam[i])
            firsts[q] = mu
    out = {"h": h.view(s["x"].shape)}
    if c["states"]:
        out["state_out"] = finals
    if c["train"]:
        dgate = before * lam * -a if slope is None else (before * lam - x * lam) * slope
        out.update(dgate=dgate.view(s["x"].shape), dx=(w * lam).view(s["x"].shape))
        if c["states"]:
            out["dstate_in"] = firsts
    return out


def _exact_step(s):
    a, w, _ = _exact_decay(s)
    state, h = s["state"].double(), torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    for row, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            state[slot] = h[row] = state[slot] * a[row] + s["x"][row].double() * w[row]
    return {"h": h, "state": state}


def _exact_ce(s):
    """Rows of live tokens in pieces, each against the whole table."""
    c = s["case"]
    t, v, d = c["tokens"], c["vocab"], c["width"]
    table = s["table"].double()
    f64 = {"dtype": torch.float64, "device": "cuda"}
    loss, lse = torch.zeros(t, **f64), torch.zeros(t, **f64)
    dx, dtable = torch.zeros(t, d, **f64), torch.zeros(v, d, **f64)
    rows = torch.nonzero(s["ids"] >= 0)[:, 0]
    for at in rows.split(max(1, (1 << 27) // v)):
        x, y = s["x"][at].double(), s["ids"][at]
        logits = torch.matmul(x, table.t())
        lse[at] = torch.logsumexp(logits, 1)
        hit = torch.arange(at.numel(), device="cuda"), y
        loss[at] = lse[at] - logits[hit]
        if c["train"]:
            grad = torch.softmax(logits, 1)
            grad[hit] -= 1.0
            grad *= s["dloss"][at].double()[:, None]
            dx[at] = torch.matmul(grad, table)
            dtable += torch.matmul(grad.t().contiguous(), x)
    out = {"loss": loss, "lse": lse}
    if c["train"]:
        out.update(dx=dx, dtable=dtable)
    return out


def _exact_adamw(s):
    c, f = s["case"], s["flat"]
    eight = c["bits"] == 8
    m, v = f["m"].double(), f["v"].double()
    if eight:
        m = m * f["m_scale"].double().repeat_interleave(BLOCK)
        v = (v * f["v_scale"].double().repeat_interleave(BLOCK)) ** 2
    g = f["g"].double()
    m = m + (g - m) * (1 - BETA1)
    v = v + (g ** 2 - v) * (1 - BETA2)
    p = f["master" if c["master"] else "p"].double()
    wd = torch.tensor(s["decays"], dtype=torch.float64, device="cuda")[s["tensor_of"]].repeat_interleave(BLOCK)
    p = p - LR * (wd * p + m / (1 - BETA1 ** STEP) / ((v / (1 - BETA2 ** STEP)) ** 0.5 + EPS))
    out = {"p": p, "m": None if eight else m, "v": None if eight else v}  # (rounding to codes draws random bits)
    if c["master"]:
        out["master"] = p
    return out
