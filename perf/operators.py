"""Cases of the sequence-layer operators: decayed linear attention, layer norm and embedding.

Each case is one pass through one operator as a training step, a prompt or a
decoding step calls it.  ``own`` false computes it in plain torch operations
in 32 bits; ``own`` true calls laplace_prefix_scans_amd.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CHUNK = 64  # tokens per chunk of the plain attention


# ------------------------------------------------------------------ cases
# attn: `seqs` sequences of `tokens` tokens in all (ragged: packed, of different lengths, some empty
# or one token long; else equal lengths), `heads` query heads over `kv` key/value heads of dk and dv
# channels.  train: forward and backward, with the decay rates' gradient; states: an initial
# state comes in and the final one goes out (and their gradients in training).
# step: one token for each of `seqs` sequences whose states lie in a pool, updated in place.
# norm: `rows` x `width`.  embed: `tokens` ids into a `vocab` x `width` table.
def listed():
    return [
        # the tail of a short request: little more than one chunk, widths that fill no tile
        {"name": "prompt_short_f32", "op": "attn", "dtype": "f32", "seqs": 1, "tokens": 131, "heads": 4, "kv": 4, "dk": 80,
         "dv": 96, "ragged": False, "train": False, "states": True},
        # a server's batch of prompts of different lengths, key/value heads shared by four query heads
        {"name": "prompt_packed_bf16", "op": "attn", "dtype": "bf16", "seqs": 24, "tokens": 16411, "heads": 16, "kv": 4,
         "dk": 128, "dv": 128, "ragged": True, "train": False, "states": True},
        # one very long document: few rows to spread over the chip, so the time axis is what is split
        {"name": "prompt_long_bf16", "op": "attn", "dtype": "bf16", "seqs": 1, "tokens": 65536, "heads": 8, "kv": 8, "dk": 128,
         "dv": 128, "ragged": False, "train": False, "states": False},
        # an ordinary pre-training micro-batch
        {"name": "attn_train_bf16", "op": "attn", "dtype": "bf16", "seqs": 8, "tokens": 16384, "heads": 16, "kv": 16, "dk": 128,
         "dv": 128, "ragged": False, "train": True, "states": False},
        # a small model in single precision on packed documents, gradients through its states
        {"name": "attn_train_f32", "op": "attn", "dtype": "f32", "seqs": 9, "tokens": 4099, "heads": 8, "kv": 4, "dk": 64,
         "dv": 64, "ragged": True, "train": True, "states": True},
        # one user's next token: a call whose latency is all that counts
        {"name": "step_one_f32", "op": "step", "dtype": "f32", "seqs": 1, "heads": 8, "kv": 8, "dk": 64, "dv": 64},
        # a full decoding batch with some of its places free
        {"name": "step_batch_bf16", "op": "step", "dtype": "bf16", "seqs": 256, "heads": 16, "kv": 16, "dk": 128, "dv": 128},
        # the norm in front of a decoding step
        {"name": "norm_few_bf16", "op": "norm", "dtype": "bf16", "rows": 8, "width": 2048, "train": False},
        # a training micro-batch's norm with the weight's gradient
        {"name": "norm_train_bf16", "op": "norm", "dtype": "bf16", "rows": 16384, "width": 4096, "train": True},
        # an odd width in single precision
        {"name": "norm_train_f32", "op": "norm", "dtype": "f32", "rows": 4099, "width": 1001, "train": True},
        # a training micro-batch's lookup and the gradient of the whole table
        {"name": "embed_train_bf16", "op": "embed", "dtype": "bf16", "tokens": 16384, "vocab": 65536, "width": 2048},
        # a small vocabulary whose rows are each used many times
        {"name": "embed_train_f32", "op": "embed", "dtype": "f32", "tokens": 4096, "vocab": 257, "width": 513},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_once(rng):
    op = rng.choice(["attn", "attn", "attn", "step", "norm", "embed"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "norm":
        return {"op": op, "dtype": dtype, "rows": _log_int(rng, 1, 32768), "width": _log_int(rng, 32, 8192),
                "train": rng.random() < 0.7}
    if op == "embed":
        return {"op": op, "dtype": dtype, "tokens": _log_int(rng, 16, 65536), "vocab": _log_int(rng, 64, 131072),
                "width": _log_int(rng, 32, 4096)}
    kv = rng.choice([1, 2, 4, 8, 16])
    heads = kv * rng.choice([1, 1, 2, 4])
    dk, dv = rng.choice([(64, 64), (128, 128), (64, 128), (128, 64), (256, 256), (rng.randint(16, 160), rng.randint(16, 160))])
    if op == "step":
        return {"op": op, "dtype": dtype, "seqs": _log_int(rng, 1, 512), "heads": heads, "kv": kv, "dk": dk, "dv": dv}
    seqs = _log_int(rng, 1, 32)
    ragged = rng.random() < 0.6
    tokens = max(seqs, _log_int(rng, 64, 65536))
    if not ragged:
        tokens -= tokens % seqs
    return {"op": op, "dtype": dtype, "seqs": seqs, "tokens": tokens, "heads": heads, "kv": kv, "dk": dk, "dv": dv,
            "ragged": ragged, "train": rng.random() < 0.5, "states": rng.random() < 0.5}


def draw(rng):
    top = [work(c) for c in listed()]
    most = {m: max(w[m] for w in top) for m in ("bytes", "flops")}
    while True:
        c = _draw_once(rng)
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        if not case["train"]:
            return {"bytes": 2 * e * n + 8 * case["rows"] + 2 * e * case["width"], "flops": 8 * n}
        return {"bytes": 5 * e * n + 8 * case["rows"] + (2 * e + 8) * case["width"], "flops": 20 * n}
    if case["op"] == "embed":
        t, v, d = case["tokens"], case["vocab"], case["width"]
        used = v * (1.0 - (1.0 - 1.0 / v) ** t)  # rows read, at most: distinct ids of a uniform draw
        return {"bytes": e * d * (used + t) + e * d * (t + v) + 8 * t, "flops": 2 * t * d}
    h, kv, dk, dv, n = case["heads"], case["kv"], case["dk"], case["dv"], case["seqs"]
    t = n if case["op"] == "step" else case["tokens"]
    token = e * t * (h * dk + kv * dk + kv * dv)
    out = e * t * h * dv
    state = 4 * n * h * dk * dv
    pair = t * h * dk * dv
    if case["op"] == "step":
        return {"bytes": token + out + 2 * state, "flops": 4 * pair}
    if not case["train"]:
        return {"bytes": token + out + (2 * state if case["states"] else 0), "flops": 4 * pair}
    return {"bytes": 3 * token + 2 * out + (4 * state if case["states"] else 0), "flops": 14 * pair}


# ------------------------------------------------------------------ inputs
def _lengths(case, seed):
    """Lengths of packed sequences: spread over about a factor of ten, one empty and one of one token where there are enough."""
    n, t = case["seqs"], case["tokens"]
    if not case["ragged"]:
        return np.full(n, t // n, dtype=np.int64)
    r = np.random.default_rng([seed, 11])
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
        return (torch.randn(shape, generator=g, device=dev) * std + mean).to(dtype)

    s = {"case": case}
    if case["op"] == "norm":
        r, d = case["rows"], case["width"]
        s.update(x=normal(r, d, std=1.5, mean=0.25), w=normal(d, std=0.2, mean=1.0), b=normal(d, std=0.1), dy=normal(r, d))
        return s
    if case["op"] == "embed":
        t, v, d = case["tokens"], case["vocab"], case["width"]
        # word frequencies fall off like 1 / rank; the ranks are dealt to the ids at random; some places are padding (-1)
        u = torch.rand(t, generator=g, device=dev, dtype=torch.float64)
        rank = torch.clamp((torch.exp(u * math.log(v + 1.0)) - 1.0).long(), max=v - 1)
        ids = torch.randperm(v, generator=g, device=dev)[rank]
        ids[torch.rand(t, generator=g, device=dev) < 0.02] = -1
        s.update(ids=ids, table=normal(v, d, std=0.02), dy=normal(t, d), scale=math.sqrt(d))
        return s
    h, kv, dk, dv, n = case["heads"], case["kv"], case["dk"], case["dv"], case["seqs"]
    # decays from a few tokens' memory to thousands, spread over the heads
    s["rate"] = torch.exp(torch.linspace(math.log(0.3), math.log(2e-4), h, device=dev)).float()
    s["scale"] = dk ** -0.5
    if case["op"] == "step":
        pool = n + n // 8 + 1
        s["slots"] = torch.randperm(pool - 1, generator=g, device=dev)[:n].to(torch.int32)
        if n >= 8:  # places of the batch with no request
            s["slots"][:: 8] = -1
        s.update(q=normal(n, h, dk), k=normal(n, kv, dk), v=normal(n, kv, dv),
                 state=normal(pool, h, dk, dv, std=2.0, dtype=torch.float32))
        return s
    t = case["tokens"]
    lengths = _lengths(case, seed)
    s["longest"] = int(lengths.max())
    s["offsets"] = None
    if case["ragged"]:
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)).to(dev)
    s.update(q=normal(t, h, dk), k=normal(t, kv, dk), v=normal(t, kv, dv), do=normal(t, h, dv))
    s["state_in"] = normal(n, h, dk, dv, std=2.0, dtype=torch.float32) if case["states"] else None
    s["dstate_out"] = normal(n, h, dk, dv, std=0.2, dtype=torch.float32) if case["states"] else None
    if not case["ragged"]:  # equal lengths: a batch axis
        for name in ("q", "k", "v", "do"):
            s[name] = s[name].view(n, t // n, *s[name].shape[1:])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return {"attn": _attn, "step": _step, "norm": _norm, "embed": _embed}[state["case"]["op"]](state)


def _attn(s):
    c = s["case"]
    if own:
        import laplace_prefix_scans_amd as lp
        state_out = torch.empty_like(s["state_in"]) if c["states"] else None
        o = lp.laplex_decay_attn(s["q"], s["k"], s["v"], s["rate"], offsets=s["offsets"], scale=s["scale"],
                                 state_in=s["state_in"], state_out=state_out)
        out = {"o": o}
        if c["states"]:
            out["state_out"] = state_out
        if c["train"]:
            g = lp.laplex_decay_attn_backward(s["q"], s["k"], s["v"], s["rate"], s["do"], offsets=s["offsets"], scale=s["scale"],
                                              state_in=s["state_in"], dstate_out=s["dstate_out"])
            out.update(dq=g[0], dk=g[1], dv=g[2], drate=g[3])
            if c["states"]:
                out["dstate_in"] = g[4]
        return out
    leaves = [x if x is None else x.float().requires_grad_(c["train"])
              for x in (s["q"].detach(), s["k"].detach(), s["v"].detach(), s["rate"].detach().clone(),
                        None if s["state_in"] is None else s["state_in"].detach().clone())]
    o, state_out = _plain_attn(*leaves, s["offsets"], s["longest"], s["scale"], c["states"])
    out = {"o": o.detach().to(s["q"].dtype)}
    if c["states"]:
        out["state_out"] = state_out.detach()
    if c["train"]:
        ins = [x for x in leaves if x is not None]
        g = torch.autograd.grad([o] + ([state_out] if c["states"] else []), ins,
                                [s["do"].float()] + ([s["dstate_out"]] if c["states"] else []))
        out.update(dq=g[0].to(s["q"].dtype), dk=g[1].to(s["q"].dtype), dv=g[2].to(s["q"].dtype), drate=g[3])
        if c["states"]:
            out["dstate_in"] = g[4]
    return out


def _plain_attn(q, k, v, rate, state_in, offsets, longest, scale, states):
    """Chunks of CHUNK tokens: a masked product inside each, and the states that chunks hand on as one product over chunks."""
    shape_o = (*q.shape[:-1], v.shape[-1])
    h, dk, dv = q.shape[-2], q.shape[-1], v.shape[-1]
    nc = -(-longest // CHUNK)
    if offsets is None:
        n = q.shape[0]
        length = torch.full((n,), longest, device=q.device)
        place = (torch.arange(n, device=q.device)[:, None] * (nc * CHUNK) + torch.arange(longest, device=q.device)).reshape(-1)
    else:
        n = offsets.numel() - 1
        length = offsets.diff()
        t = torch.arange(q.shape[0], device=q.device)
        seq = torch.searchsorted(offsets[1:].long(), t, right=True)
        place = seq * (nc * CHUNK) + t - offsets.long()[seq]

    def padded(x):  # (tokens, heads, d) -> (n, h, chunks, CHUNK, d)
        x = x.reshape(-1, *x.shape[-2:]).repeat_interleave(h // x.shape[-2], dim=1)
        y = torch.zeros(n * nc * CHUNK, *x.shape[1:], device=x.device).index_copy(0, place, x)
        return y.view(n, nc, CHUNK, h, -1).permute(0, 3, 1, 2, 4).contiguous()

    q, k, v = padded(q), padded(k), padded(v)
    r = rate.view(h, 1, 1)
    i = torch.arange(CHUNK, device=q.device, dtype=torch.float32)
    lag = i[:, None] - i
    w = torch.where(lag >= 0, torch.exp(-r * lag.clamp(min=0)), 0.0).view(h, 1, CHUNK, CHUNK)
    o = ((q @ k.transpose(-1, -2).contiguous()) * w) @ v
    tail = torch.exp(-r * (CHUNK - 1 - i)).view(h, 1, CHUNK, 1)
    kv = ((k * tail).transpose(-1, -2).contiguous() @ v).view(n, h, nc, dk * dv)
    c = torch.arange(nc, device=q.device, dtype=torch.float32)
    back = c[:, None] - 1 - c
    m = torch.where(back >= 0, torch.exp(-r * CHUNK * back.clamp(min=0)), 0.0)
    start = m @ kv
    if state_in is not None:
        start = start + torch.exp(-r * CHUNK * c[:, None]) * state_in.view(n, h, 1, dk * dv)
    o = o + torch.exp(-r * (i[:, None] + 1)).view(h, 1, CHUNK, 1) * (q @ start.view(n, h, nc, dk, dv))
    o = scale * o.permute(0, 2, 3, 1, 4).reshape(n * nc * CHUNK, h, dv)[place].view(shape_o)
    if not states:
        return o, None
    left = length.view(n, 1, 1) - 1 - torch.arange(nc * CHUNK, device=q.device, dtype=torch.float32)
    wl = torch.where(left >= 0, torch.exp(-rate.view(1, h, 1) * left.clamp(min=0)), 0.0)
    k2 = (k.view(n, h, nc * CHUNK, dk) * wl[..., None]).transpose(-1, -2).contiguous()
    state = k2 @ v.view(n, h, nc * CHUNK, dv)
    return o, state + torch.exp(-rate.view(1, h, 1, 1) * length.view(n, 1, 1, 1)) * state_in


def _step(s):
    if own:
        import laplace_prefix_scans_amd as lp
        o = lp.laplex_decay_attn_step(s["q"], s["k"], s["v"], s["rate"], s["state"], slots=s["slots"], scale=s["scale"])
        return {"o": o, "state": s["state"]}
    h, slot = s["q"].shape[1], s["slots"].long()
    live = slot >= 0
    group = h // s["k"].shape[1]
    k, v = s["k"].float().repeat_interleave(group, dim=1), s["v"].float().repeat_interleave(group, dim=1)
    new = torch.exp(-s["rate"]).view(h, 1, 1) * s["state"][slot.clamp(min=0)] + k[..., None] * v[..., None, :]
    o = s["scale"] * (s["q"].float()[..., None] * new).sum(-2)
    # the pool's last row is nobody's: a place without a request puts there what is there already
    live = live.view(-1, 1, 1)
    s["state"].index_copy_(0, torch.where(live.view(-1), slot, s["state"].shape[0] - 1),
                           torch.where(live[..., None], new, s["state"][-1]))
    return {"o": torch.where(live, o, 0.0).to(s["q"].dtype), "state": s["state"]}


def _norm(s):
    c, eps = s["case"], 1e-5
    if own:
        import laplace_prefix_scans_amd as lp
        y, mean, rstd = lp.laplex_layer_norm(s["x"], s["w"], s["b"], eps=eps)
        out = {"y": y, "mean": mean, "rstd": rstd}
        if c["train"]:
            out["dx"], out["dw"], out["db"] = lp.laplex_layer_norm_backward(s["x"], s["dy"], mean, rstd, s["w"])
        return out
    x, w = s["x"].float(), s["w"].float()
    mean = x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((x - mean).square().mean(-1, keepdim=True) + eps)
    xh = (x - mean) * rstd
    out = {"y": (xh * w + s["b"].float()).to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if c["train"]:
        g = s["dy"].float()
        gw = g * w
        dx = rstd * (gw - gw.mean(-1, keepdim=True) - xh * (gw * xh).mean(-1, keepdim=True))
        out.update(dx=dx.to(s["x"].dtype), dw=(g * xh).sum(0), db=g.sum(0))
    return out


def _embed(s):
    if own:
        import laplace_prefix_scans_amd as lp
        y = lp.laplex_embedding(s["ids"], s["table"], scale=s["scale"])
        return {"y": y, "dtable": lp.laplex_embedding_backward(s["ids"], s["dy"], s["table"].shape[0], scale=s["scale"])}
    live = (s["ids"] >= 0).view(-1, 1)
    at = s["ids"].clamp(min=0)
    y = torch.where(live, s["scale"] * s["table"][at].float(), 0.0)
    g = torch.where(live, s["scale"] * s["dy"].float(), 0.0)
    dtable = torch.zeros(s["table"].shape, device=g.device).index_add_(0, at, g)
    return {"y": y.to(s["table"].dtype), "dtable": dtable.to(s["table"].dtype)}


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "step": _exact_step, "norm": _exact_norm, "embed": _exact_embed}[case["op"]](s)


def _exact_attn(s):
    """Every pair (i, j) of every sequence, in blocks of rows i."""
    c = s["case"]
    h, kvh, dk, dv, n = c["heads"], c["kv"], c["dk"], c["dv"], c["seqs"]
    f64 = torch.float64
    flat = {x: s[x].reshape(-1, *s[x].shape[-2:]).to(f64).transpose(0, 1).contiguous() for x in ("q", "k", "v", "do")}
    rate, scale = s["rate"].to(f64).view(h, 1, 1), s["scale"]
    if s["offsets"] is None:
        bounds = [x * (c["tokens"] // n) for x in range(n + 1)]
    else:
        bounds = s["offsets"].tolist()
    t = c["tokens"]
    o = torch.zeros(h, t, dv, dtype=f64, device="cuda")
    dq, dk_, dv_ = torch.zeros(h, t, dk, dtype=f64, device="cuda"), torch.zeros(h, t, dk, dtype=f64, device="cuda"), \
        torch.zeros(h, t, dv, dtype=f64, device="cuda")
    drate = torch.zeros(h, dtype=f64, device="cuda")
    finals, dins = [], []
    for a, b in zip(bounds[:-1], bounds[1:]):
        x = len(finals)
        ln = b - a
        q, g = flat["q"][:, a:b], flat["do"][:, a:b]
        k, v = (flat[y][:, a:b].repeat_interleave(h // kvh, dim=0) for y in ("k", "v"))
        s0 = s["state_in"][x].to(f64) if c["states"] else torch.zeros(h, dk, dv, dtype=f64, device="cuda")
        gf = s["dstate_out"][x].to(f64) if c["states"] else torch.zeros(h, dk, dv, dtype=f64, device="cuda")
        j = torch.arange(ln, dtype=f64, device="cuda")
        rows = max(1, min(ln, (1 << 26) // max(1, h * ln)))
        for i0 in range(0, ln, rows):
            i1 = min(ln, i0 + rows)
            lag = (j[i0:i1, None] - j[None, :i1]).unsqueeze(0)
            w = torch.where(lag >= 0, torch.exp(-rate * lag.clamp(min=0)), 0.0) * scale
            p = torch.matmul(q[:, i0:i1], k[:, :i1].transpose(1, 2).contiguous())
            o[:, a + i0:a + i1] = torch.matmul(w * p, v[:, :i1].contiguous())
            if c["train"]:
                d = torch.matmul(g[:, i0:i1], v[:, :i1].transpose(1, 2).contiguous())
                dq[:, a + i0:a + i1] = torch.matmul(w * d, k[:, :i1].contiguous())
                dk_[:, a:a + i1] += torch.matmul((w * d).transpose(1, 2).contiguous(), q[:, i0:i1].contiguous())
                dv_[:, a:a + i1] += torch.matmul((w * p).transpose(1, 2).contiguous(), g[:, i0:i1].contiguous())
                drate -= (lag * w * p * d).sum((1, 2))
        up = torch.exp(-rate * (j.view(1, -1, 1) + 1)) * scale
        down = torch.exp(-rate * (ln - 1 - j.view(1, -1, 1)))
        whole = torch.exp(-rate * ln)
        qs = torch.matmul(q, s0)
        o[:, a:b] += up * qs
        finals.append(whole * s0 + torch.matmul((down * k).transpose(1, 2).contiguous(), v.contiguous()))
        if c["train"]:
            kg, vg = torch.matmul(k, gf), torch.matmul(v, gf.transpose(1, 2).contiguous())
            dq[:, a:b] += up * torch.matmul(g, s0.transpose(1, 2).contiguous())
            dk_[:, a:b] += down * vg
            dv_[:, a:b] += down * kg
            dins.append(whole * gf + torch.matmul((up * q).transpose(1, 2).contiguous(), g.contiguous()))
            drate -= ((j.view(1, -1) + 1) * (up * qs * g).sum(-1)).sum(-1)
            drate -= ((ln - 1 - j.view(1, -1)) * (down * kg * v).sum(-1)).sum(-1)
            drate -= ln * (whole * s0 * gf).sum((1, 2))

    def back(y, like, heads):
        y = y.view(heads, -1, t, y.shape[-1]).sum(1)
        return y.transpose(0, 1).reshape(s[like].shape)

    out = {"o": o.transpose(0, 1).reshape(s["do"].shape)}
    if c["states"]:
        out["state_out"] = torch.stack(finals)
    if c["train"]:
        out.update(dq=back(dq, "q", h), dk=back(dk_, "k", kvh), dv=back(dv_, "v", kvh), drate=drate)
        if c["states"]:
            out["dstate_in"] = torch.stack(dins)
    return out


def _exact_step(s):
    state = s["state"].double()
    o = torch.zeros(s["q"].shape[0], s["q"].shape[1], s["v"].shape[2], dtype=torch.float64, device="cuda")
    group = s["q"].shape[1] // s["k"].shape[1]
    for x, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        k, v = (s[y][x].double().repeat_interleave(group, dim=0) for y in ("k", "v"))
        state[slot] = state[slot] * torch.exp(-s["rate"].double()).view(-1, 1, 1) + k.unsqueeze(2) * v.unsqueeze(1)
        o[x] = s["scale"] * torch.matmul(s["q"][x].double().unsqueeze(1), state[slot]).squeeze(1)
    return {"o": o, "state": state}


def _exact_norm(s):
    x, w, b, g = (s[y].double() for y in ("x", "w", "b", "dy"))
    d = x.shape[1]
    mean = x.sum(1) / d
    var = ((x - mean.unsqueeze(1)) ** 2).sum(1) / d
    rstd = (var + 1e-5) ** -0.5
    z = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1)
    out = {"y": z * w + b, "mean": mean, "rstd": rstd}
    if s["case"]["train"]:
        # the Jacobian of z: (I - 1 1^T / d - z z^T / d) rstd
        u = g * w
        out["dx"] = (u - u.sum(1, keepdim=True) / d - z * ((u * z).sum(1, keepdim=True) / d)) * rstd.unsqueeze(1)
        out["dw"], out["db"] = (g * z).sum(0), g.sum(0)
    return out


def _exact_embed(s):
    t, (v, d) = s["ids"].shape[0], s["table"].shape
    y = torch.zeros(t, d, dtype=torch.float64, device="cuda")
    at = torch.nonzero(s["ids"] >= 0)[:, 0]
    y[at] = s["scale"] * s["table"].double()[s["ids"][at]]
    # the gradient by sorted tokens: differences of running sums would lose bits, so rows are added group by group
    dtable = torch.zeros(v, d, dtype=torch.float64, device="cuda")
    dtable.index_put_((s["ids"][at],), s["scale"] * s["dy"].double()[at], accumulate=True)
    return {"y": y, "dtable": dtable}
