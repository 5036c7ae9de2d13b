"""A small language model on the library's sequence layers, trained and run.

    python examples/decay_lm.py [--steps 200] [--dtype bf16] [--mixer gated] [--fused] [--moments 8]

embedding -> blocks of [layer norm, decayed linear attention, layer norm, gated
feed-forward] -> layer norm -> tied output table.  The decay rates are learned
with the weights (started so that the heads remember from a few tokens to
hundreds).  With --mixer gated the attention's place is taken by a gated linear
recurrence, whose decays each token sets for itself.  With --fused the loss is
formed from the last layer's rows and the table, without the logits in memory,
and one launch updates all parameters (with --moments 8, moments of one byte).
Training packs documents of different lengths into one row of
tokens; generation reads a prompt in one pass, which leaves each layer's state,
and continues token by token from it.  The task is synthetic: a document's first
token names one of a few fixed permutations of the vocabulary, and each later
token is that permutation of the one before -- so the first token has to be
remembered to the end.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import laplace_prefix_scans_amd as lp  # noqa: E402


class Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale):
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.scale = table.shape[0], scale
        return lp.laplex_embedding(ids, table, scale=scale)

    @staticmethod
    @once_differentiable  # the library has first derivatives
    def backward(ctx, g):
        (ids,) = ctx.saved_tensors
        return None, lp.laplex_embedding_backward(ids, g.contiguous(), ctx.vocab, scale=ctx.scale), None


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        x = x.contiguous()
        y, mean, rstd = lp.laplex_layer_norm(x, weight, bias)
        ctx.save_for_backward(x, mean, rstd, weight)
        return y

    @staticmethod
    @once_differentiable  # the library has first derivatives
    def backward(ctx, g):
        x, mean, rstd, weight = ctx.saved_tensors
        if not any(ctx.needs_input_grad[1:]):
            return lp.laplex_layer_norm_backward(x, g.contiguous(), mean, rstd, weight, param_grads=False)
        dx, dw, db = lp.laplex_layer_norm_backward(x, g.contiguous(), mean, rstd, weight)
        return dx, dw.to(weight.dtype), db.to(weight.dtype)


class DecayAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, rate, offsets, scale):
        ctx.save_for_backward(q, k, v, rate, offsets)
        ctx.scale = scale
        return lp.laplex_decay_attn(q, k, v, rate, offsets=offsets, scale=scale)

    @staticmethod
    @once_differentiable  # the library has first derivatives
    def backward(ctx, g):
        q, k, v, rate, offsets = ctx.saved_tensors
        dq, dk, dv, drate, _ = lp.laplex_decay_attn_backward(q, k, v, rate, g.contiguous(), offsets=offsets, scale=ctx.scale,
                                                             rate_grad=ctx.needs_input_grad[3])
        return dq, dk, dv, drate, None, None


class GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, x, offsets):
        h, carries = lp.laplex_gated_scan(gate, x, "sigmoid", offsets=offsets, keep=True)
        ctx.save_for_backward(gate, x, offsets, carries)
        return h

    @staticmethod
    @once_differentiable  # the library has first derivatives
    def backward(ctx, g):
        gate, x, offsets, carries = ctx.saved_tensors
        dgate, dx, _ = lp.laplex_gated_scan_backward(gate, x, carries, g.contiguous(), "sigmoid", offsets=offsets)
        return dgate, dx, None


class LinearCrossEntropy(torch.autograd.Function):
    """The loss of each token (zero where its target is outside the vocabulary), in float32."""

    @staticmethod
    def forward(ctx, x, table, targets):
        x = x.contiguous()
        loss, lse = lp.laplex_linear_cross_entropy(x, table, targets)
        ctx.save_for_backward(x, table, targets, lse)
        return loss

    @staticmethod
    @once_differentiable  # the library has first derivatives
    def backward(ctx, g):
        x, table, targets, lse = ctx.saved_tensors
        return (*lp.laplex_linear_cross_entropy_backward(x, table, targets, lse, g.contiguous(), x_grad=ctx.needs_input_grad[0],
                                                         table_grad=ctx.needs_input_grad[1]), None)


class AdamW:
    """All parameters in one call for each type of theirs; bfloat16 ones have float32 copies, which are what is updated."""

    def __init__(self, params, lr, weight_decay=0.01, bits=32):
        self.lr, self.weight_decay, self.bits, self.count = lr, weight_decay, bits, 0
        self.groups = []
        params = list(params)
        for dtype in (torch.float32, torch.bfloat16):
            ps = [p for p in params if p.dtype is dtype]
            if ps:
                kind = torch.float32 if bits == 32 else torch.uint8
                state = {k: [torch.zeros(p.shape, dtype=kind, device=p.device) for p in ps] for k in ("m", "v")}
                if bits == 8:
                    for k in ("m_scale", "v_scale"):
                        state[k] = [torch.zeros(-(-p.numel() // 256), device=p.device) for p in ps]
                if dtype is torch.bfloat16:
                    state["master"] = [p.detach().float() for p in ps]
                self.groups.append((ps, state))

    @torch.no_grad()
    def step(self):
        self.count += 1
        for ps, state in self.groups:
            lp.laplex_adamw([p.detach() for p in ps], [p.grad for p in ps], lr=self.lr, step=self.count, weight_decay=self.weight_decay,
                            seed=self.count if self.bits == 8 else None, **state)

    def zero_grad(self):
        for ps, _ in self.groups:
            for p in ps:
                p.grad = None


class DecayLM:
    """Parameters in a dict; forward() for packed documents, prefill() and step() for generation."""

    def __init__(self, vocab=64, width=256, heads=4, layers=2, dtype=torch.float32, device="cuda", seed=0, mixer="attention"):
        assert mixer in ("attention", "gated"), mixer
        g = torch.Generator().manual_seed(seed)
        self.vocab, self.width, self.heads, self.layers, self.dtype = vocab, width, heads, layers, dtype
        self.head, self.mixer = width // heads, mixer
        self.scale = self.head ** -0.5

        def normal(*shape, std):
            return (torch.randn(shape, generator=g) * std).to(device, dtype).requires_grad_()

        def const(n, value):
            return torch.full((n,), value, device=device, dtype=dtype).requires_grad_()

        p = {"table": normal(vocab, width, std=width ** -0.5), "norm.w": const(width, 1.0), "norm.b": const(width, 0.0)}
        for i in range(layers):
            p.update({"%d.n1.w" % i: const(width, 1.0), "%d.n1.b" % i: const(width, 0.0), "%d.n2.w" % i: const(width, 1.0),
                      "%d.n2.b" % i: const(width, 0.0)})
            if mixer == "attention":
                p["%d.qkv" % i] = normal(width, 3 * width, std=width ** -0.5)
            else:
                p["%d.gx" % i] = normal(width, 2 * width, std=width ** -0.5)
                # decays 1 - 1 / m where the projection gives 0: memories m of 4 to 400 tokens
                p["%d.gate.b" % i] = torch.log(torch.logspace(math.log10(4), math.log10(400), width) - 1).to(device, dtype).requires_grad_()
            p.update({
                      "%d.out" % i: normal(width, width, std=0.5 * width ** -0.5),
                      "%d.up" % i: normal(width, 4 * width, std=width ** -0.5),
                      "%d.down" % i: normal(2 * width, width, std=0.5 * width ** -0.5)})
            if mixer == "attention":
                # the rates' logarithms: memories of about 4 to 400 tokens
                p["%d.rate" % i] = torch.log(torch.logspace(math.log10(0.25), math.log10(0.0025), heads)).to(device).requires_grad_()
        self.p = p

    def _qkv(self, x, i):
        t = x.shape[0]
        y = LayerNorm.apply(x, self.p["%d.n1.w" % i], self.p["%d.n1.b" % i]) @ self.p["%d.qkv" % i]
        # slices of one projection: the attention takes them as they lie
        return y.view(t, 3, self.heads, self.head).unbind(1)

    def _gate_x(self, x, i):
        y = LayerNorm.apply(x, self.p["%d.n1.w" % i], self.p["%d.n1.b" % i]) @ self.p["%d.gx" % i]
        gate, v = y.chunk(2, -1)  # the recurrence takes the second slice as it lies
        return gate + self.p["%d.gate.b" % i], v

    def _rest(self, x, o, i):
        x = x + o.reshape(x.shape) @ self.p["%d.out" % i]
        a, b = (LayerNorm.apply(x, self.p["%d.n2.w" % i], self.p["%d.n2.b" % i]) @ self.p["%d.up" % i]).chunk(2, -1)
        return x + (torch.nn.functional.silu(a) * b) @ self.p["%d.down" % i]

    def _last(self, x):
        return LayerNorm.apply(x, self.p["norm.w"], self.p["norm.b"])

    def _logits(self, x):
        return (self._last(x) @ self.p["table"].t()).float()

    def _rate(self, i):
        return torch.exp(self.p["%d.rate" % i])

    def _blocks(self, ids, offsets):
        x = Embedding.apply(ids, self.p["table"], math.sqrt(self.width))
        for i in range(self.layers):
            if self.mixer == "gated":
                x = self._rest(x, GatedScan.apply(*self._gate_x(x, i), offsets), i)
                continue
            q, k, v = self._qkv(x, i)
            x = self._rest(x, DecayAttention.apply(q, k, v, self._rate(i), offsets, self.scale), i)
        return x

    def forward(self, ids, offsets):
        return self._logits(self._blocks(ids, offsets))

    def losses(self, ids, offsets, targets):
        """The cross entropy of each token's target (a target of -1: zero), without the logits in memory."""
        return LinearCrossEntropy.apply(self._last(self._blocks(ids, offsets)), self.p["table"], targets)

    @torch.no_grad()
    def prefill(self, ids, offsets):
        """Logits of every prompt token, and each layer's states after the prompts."""
        x = lp.laplex_embedding(ids, self.p["table"], scale=math.sqrt(self.width))
        states = []
        for i in range(self.layers):
            if self.mixer == "gated":
                state = torch.empty(offsets.numel() - 1, self.width, device=x.device)
                o = lp.laplex_gated_scan(*self._gate_x(x, i), "sigmoid", offsets=offsets, state_out=state)
                states.append(state)
                x = self._rest(x, o, i)
                continue
            q, k, v = self._qkv(x, i)
            state = torch.empty(offsets.numel() - 1, self.heads, self.head, self.head, device=x.device)
            o = lp.laplex_decay_attn(q, k, v, self._rate(i), offsets=offsets, scale=self.scale, state_out=state)
            states.append(state)
            x = self._rest(x, o, i)
        return self._logits(x), states

    @torch.no_grad()
    def step(self, ids, states, slots=None):
        """One token for each row; the states move on in place."""
        x = lp.laplex_embedding(ids, self.p["table"], scale=math.sqrt(self.width))
        for i in range(self.layers):
            if self.mixer == "gated":
                x = self._rest(x, lp.laplex_gated_scan_step(*self._gate_x(x, i), states[i], "sigmoid", slots=slots), i)
                continue
            q, k, v = self._qkv(x, i)
            o = lp.laplex_decay_attn_step(q, k, v, self._rate(i), states[i], slots=slots, scale=self.scale)
            x = self._rest(x, o, i)
        return self._logits(x)


KEYS = 4  # permutations; their names are the ids 0 .. KEYS - 1


def follower(vocab):
    """(KEYS, vocab): the token after each one, under each permutation of the ids from KEYS on."""
    g = torch.Generator().manual_seed(1234)
    return torch.stack([torch.cat([torch.arange(KEYS), KEYS + torch.randperm(vocab - KEYS, generator=g)]) for _ in range(KEYS)])


def documents(count, vocab, gen, device="cuda"):
    """Packed documents of 24 to 160 tokens and their offsets."""
    table = follower(vocab)
    parts, ends = [], [0]
    for _ in range(count):
        key = int(torch.randint(0, KEYS, (1,), generator=gen))
        doc = [key, int(torch.randint(KEYS, vocab, (1,), generator=gen))]
        for _ in range(int(torch.randint(22, 159, (1,), generator=gen))):
            doc.append(int(table[key, doc[-1]]))
        parts.append(torch.tensor(doc))
        ends.append(ends[-1] + len(doc))
    return torch.cat(parts).to(device), torch.tensor(ends, dtype=torch.int32, device=device)


def train(model, steps, docs=32, lr=2e-3, seed=1, log=None, fused=False, moments=32):
    gen = torch.Generator().manual_seed(seed)
    opt = AdamW(model.p.values(), lr, bits=moments) if fused else torch.optim.AdamW(model.p.values(), lr=lr)
    losses = []
    for s in range(steps):
        ids, offsets = documents(docs, model.vocab, gen)
        target = torch.roll(ids, -1)
        last = offsets[1:].long() - 1
        mask = torch.ones_like(ids, dtype=torch.bool)
        mask[last] = False  # a document's last token has nothing after it
        mask[offsets[:-1].long()] = False  # and what follows the key is free
        if fused:
            loss = model.losses(ids, offsets, target.masked_fill(~mask, -1)).sum() / mask.sum()
        else:
            loss = torch.nn.functional.cross_entropy(model.forward(ids, offsets)[mask], target[mask])
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
        if log and (s % log == 0 or s == steps - 1):
            print("step %4d  loss %.3f" % (s, losses[-1]), flush=True)
    return losses


@torch.no_grad()
def generate(model, prompts, offsets, tokens):
    logits, states = model.prefill(prompts, offsets)
    ids = logits[offsets[1:].long() - 1].argmax(-1)
    out = [ids]
    for _ in range(tokens - 1):
        ids = model.step(ids, states).argmax(-1)
        out.append(ids)
    return torch.stack(out, 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    ap.add_argument("--mixer", choices=("attention", "gated"), default="attention")
    ap.add_argument("--fused", action="store_true")
    ap.add_argument("--moments", type=int, choices=(32, 8), default=32)
    a = ap.parse_args()
    if a.moments == 8 and not a.fused:
        ap.error("--moments 8 goes with --fused")
    model = DecayLM(dtype=torch.float32 if a.dtype == "f32" else torch.bfloat16, mixer=a.mixer)
    train(model, a.steps, log=20, fused=a.fused, moments=a.moments)
    ids, offsets = documents(4, model.vocab, torch.Generator().manual_seed(99))
    got = generate(model, ids, offsets, 12).tolist()
    table = follower(model.vocab)
    for d in range(4):
        lo, hi = int(offsets[d]), int(offsets[d + 1])
        key, want = int(ids[lo]), [int(ids[hi - 1])]
        for _ in range(12):
            want.append(int(table[key, want[-1]]))
        print("key %d ... %s -> %s, %d of 12 right" % (key, ids[hi - 5:hi].tolist(), got[d], sum(x == y for x, y in zip(got[d], want[1:]))))


if __name__ == "__main__":
    main()
