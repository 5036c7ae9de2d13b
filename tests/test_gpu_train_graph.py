"""A training step of the operators in one run: gated recurrence, cross entropy against a table, both backward, AdamW.
Eager against float64, each operator for what the one before gave it, and the whole one's loss against differences; then
captured into HIP graphs and replayed with other inputs and eager work between, which has to give the eager run's bits."""
import numpy as np
import pytest

import train_ref as ref
from gpu_util import have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


class Step:
    """Parameters gate, x (tokens, width) and table (vocab, width), trained on targets; all tensors but the results of the
    calls stay where they are."""

    def __init__(self, lengths, width, vocab, dtype, kind, bits, seed=0, workspaces=None):
        import torch
        import laplace_prefix_scans_amd as lp
        g = torch.Generator().manual_seed(seed)
        n = sum(lengths)
        self.kind, self.bits, self.dtype, self.vocab, self.tokens = kind, bits, dtype, vocab, n
        z = torch.rand(n, width, generator=g) * 2 if kind == "rate" else torch.randn(n, width, generator=g) * 2
        x = torch.randn(n, width, generator=g)
        table = torch.randn(vocab, width, generator=g) * width ** -0.5
        self.params = [t.to(dtype).cuda() for t in (z, x, table)]
        self.offsets = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()
        self.targets = torch.zeros(n, dtype=torch.int64, device="cuda")
        self.dloss = torch.zeros(n, device="cuda")
        self.state_in = torch.zeros(len(lengths), width, device="cuda")
        self.step = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.lr = torch.tensor([1e-2], device="cuda")
        code = torch.float32 if bits == 32 else torch.uint8
        self.state = {k: [torch.zeros(p.shape, dtype=code, device="cuda") for p in self.params] for k in ("m", "v")}
        if bits == 8:
            for k in ("m_scale", "v_scale"):
                self.state[k] = [torch.zeros(-(-p.numel() // 256), device="cuda") for p in self.params]
        if dtype is torch.bfloat16:
            self.state["master"] = [p.float() for p in self.params]
        if workspaces is None:
            sizes = [lp.laplex_gated_scan_workspace_bytes(self.params[0], self.params[1], kind, self.offsets)]
            sizes += [lp.laplex_linear_cross_entropy_workspace_bytes(b, self.params[1], self.params[2], self.targets) for b in (False, True)]
            workspaces = [torch.empty(max(s, 1), dtype=torch.uint8, device="cuda") for s in sizes]
        self.ws = workspaces

    def fill(self, r):
        """Inputs of run r."""
        import torch
        g = torch.Generator().manual_seed(100 + r)
        y = torch.randint(0, self.vocab, (self.tokens,), generator=g)
        y[::7] = -1
        self.targets.copy_(y)
        self.dloss.copy_(torch.rand(self.tokens, generator=g) / self.tokens)
        self.state_in.copy_(torch.randn(self.state_in.shape, generator=g))
        self.lr.fill_(1e-2 / (1 + r))

    def run(self):
        import laplace_prefix_scans_amd as lp
        z, x, table = self.params
        state_out = self.state_in.new_empty(self.state_in.shape)
        h, carries = lp.laplex_gated_scan(z, x, self.kind, offsets=self.offsets, state_in=self.state_in, state_out=state_out, keep=True,
                                          ws=self.ws[0])
        loss, lse = lp.laplex_linear_cross_entropy(h, table, self.targets, ws=self.ws[1])
        dh, dtable = lp.laplex_linear_cross_entropy_backward(h, table, self.targets, lse, self.dloss, ws=self.ws[2])
        dz, dx, dstate = lp.laplex_gated_scan_backward(z, x, carries, dh, self.kind, offsets=self.offsets, state_in=self.state_in,
                                                       ws=self.ws[0])
        self.step += 1
        lp.laplex_adamw(self.params, [dz, dx, dtable], lr=self.lr, step=self.step, weight_decay=[0.0, 0.0, 0.1],
                        seed=9 if self.bits == 8 else None, **self.state)
        return {"h": h, "state_out": state_out, "loss": loss, "lse": lse, "dh": dh, "dtable": dtable, "dz": dz, "dx": dx, "dstate": dstate}

    def everything(self):
        return [*self.params, self.step, *(t for k in sorted(self.state) for t in self.state[k])]


LENGTHS = [1, 0, 130, 700, 17]


@pytest.mark.parametrize("kind", ["rate", "sigmoid"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_a_step_of_all_of_them(kind, dt):
    import torch
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    s = Step(LENGTHS, 96, 333, dtype, kind, 32)
    bounds = np.concatenate([[0], np.cumsum(LENGTHS)])
    half = 2.0 ** -8 if dt == "bf16" else 2.0 ** -24
    f = lambda t: host(t.float())  # noqa: E731

    def check(name, got, want, bound, half):
        got = f(got)
        tol = bound + np.abs(want) * half + 1e-37
        assert (np.abs(got - want) <= tol).all(), (name, (np.abs(got - want) / tol).max())
    for r in range(3):
        s.fill(r)
        before = [f(p) for p in (s.state["master"] if dt == "bf16" else s.params)]
        moments = [[f(t) for t in s.state[k]] for k in ("m", "v")]
        z, x, table = (f(p) for p in s.params)
        out = s.run()
        y, w, si = s.targets.cpu().numpy(), f(s.dloss), f(s.state_in)
        a = ref.scan(z, x, kind, bounds, si, f(out["dh"]))
        check("h", out["h"], a["h"], a["~h"], half)
        check("state_out", out["state_out"], a["state_out"], a["~state_out"], 2.0 ** -24)
        check("dz", out["dz"], a["dgate"], a["~dgate"], half)
        check("dx", out["dx"], a["dx"], a["~dx"], half)
        check("dstate", out["dstate"], a["dstate_in"], a["~dstate_in"], 2.0 ** -24)
        c = ref.cross_entropy(f(out["h"]), table, y, 1.0, w, None, dt == "bf16")
        check("loss", out["loss"], c["loss"], c["~loss"], 2.0 ** -24)
        check("dh", out["dh"], c["dx"], c["~dx"], half)
        check("dtable", out["dtable"], c["dtable"], c["~dtable"], half)
        for i, (g, wd) in enumerate(zip(("dz", "dx", "dtable"), (0.0, 0.0, 0.1))):
            p, m, v, err = ref.adamw(before[i], f(out[g]), moments[0][i], moments[1][i], float(s.lr), 0.9, 0.999, 1e-8, wd, r + 1)
            check("master %d" % i, s.state["master"][i] if dt == "bf16" else s.params[i], p, err, 2.0 ** -24)
            check("param %d" % i, s.params[i], p, err, half)


def test_the_steps_gradient_against_differences():
    """The weighted loss along one direction of all parameters: truncation from the difference at twice the step, rounding
    from the bound of the loss's own error over the step."""
    import torch
    import laplace_prefix_scans_amd as lp
    s = Step(LENGTHS, 64, 100, torch.float32, "sigmoid", 32)
    s.fill(0)
    z, x, table = [p.clone() for p in s.params]
    out = s.run()
    g = torch.Generator().manual_seed(3)
    d = [torch.randn(p.shape, generator=g).cuda() for p in (z, x, table)]
    want = sum(float((a.double() * b.double()).sum()) for a, b in zip(d, (out["dz"], out["dx"], out["dtable"])))

    def at(e):
        p, q, t = (a + e * b for a, b in zip((z, x, table), d))
        h = lp.laplex_gated_scan(p, q, "sigmoid", offsets=s.offsets, state_in=s.state_in)
        return float((lp.laplex_linear_cross_entropy(h, t, s.targets)[0].double() * s.dloss.double()).sum())
    e = 2.0 ** -9
    one, two = (at(e) - at(-e)) / (2 * e), (at(2 * e) - at(-2 * e)) / (4 * e)
    # each side's loss is off by its tokens' bounds, weighted (train_ref.cross_entropy for the states as they are, and what
    # the states' own errors, train_ref.scan's, give it through the logits' gradient, which is at most 2 |table| a token)
    f = lambda t: host(t.float())  # noqa: E731
    c = ref.cross_entropy(f(out["h"]), f(table), s.targets.cpu().numpy(), 1.0)
    a = ref.scan(f(z), f(x), "sigmoid", np.concatenate([[0], np.cumsum(LENGTHS)]), f(s.state_in))
    off = float((f(s.dloss) * (c["~loss"] + 2 * (a["~h"] + 2.0 ** -24 * np.abs(a["h"])).sum(1) * np.abs(f(table)).max())).sum())
    assert abs(one - want) <= abs(two - one) + 2 * off / e, (one, two, want, off / e)


def snapshot(s):
    return [t.clone() for t in s.everything()]


@pytest.mark.parametrize("dt,kind,bits,lengths", [("f32", "rate", 32, LENGTHS), ("bf16", "sigmoid", 32, [900, 300]), ("bf16", "rate", 8, LENGTHS),
                                                  ("f32", "sigmoid", 8, [3, 2])], ids=str)
def test_captured_steps_give_the_eager_bits(dt, kind, bits, lengths):
    """Two graphs of different sequences, of one pair of workspaces, replayed in turn."""
    import torch
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    make = lambda i, ws: Step(lengths if i == 0 else lengths[::-1] + [40], 96, 333, dtype, kind, bits, seed=i, workspaces=ws)  # noqa: E731
    big = make(1, None)  # (the second has more tokens: its workspaces serve both)
    ws = big.ws
    eager = [make(i, None) for i in range(2)]
    held = [make(i, ws) for i in range(2)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for s in held:
        s.fill(0)
        kept = snapshot(s)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.run()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(s.run())
        for t, k in zip(s.everything(), kept):
            t.copy_(k)
        graphs.append(graph)
    for r in range(4):
        for i in range(2):
            eager[i].fill(r)
            want = eager[i].run()
            held[i].fill(r)
            for w in ws:
                w.fill_(r * 85)
            graphs[i].replay()
            torch.cuda.synchronize()
            for k in want:
                assert torch.equal(outs[i][k], want[k]), (r, i, k)
            for n, (p, q) in enumerate(zip(held[i].everything(), eager[i].everything())):
                assert torch.equal(p, q), (r, i, n)


@pytest.mark.parametrize("width", [1100, 4100])  # (of a few tokens' rows, the latter take more LDS than a kernel has unasked)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_captured_decoding(dt, width):
    """Single tokens: the recurrence's step in a pool of states, and the score of a few tokens."""
    import torch
    import laplace_prefix_scans_amd as lp
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    rows, vocab, pool = 4, 777, 9
    g = torch.Generator().manual_seed(1)
    table = torch.randn(vocab, width, generator=g).to(dtype).cuda()
    z, x = torch.zeros(rows, width, dtype=dtype, device="cuda"), torch.zeros(rows, width, dtype=dtype, device="cuda")
    slots, y = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda")
    state = torch.randn(pool, width, generator=g).cuda()

    def run(state):
        h = lp.laplex_gated_scan_step(z, x, state, "sigmoid", slots=slots)
        return (h, *lp.laplex_linear_cross_entropy(h, table, y, scale=0.1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(state.clone())
    torch.cuda.current_stream().wait_stream(side)
    other = state.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(state)
    assert torch.equal(state, other)
    for r in range(4):
        z.copy_(torch.randn(rows, width, generator=g))
        x.copy_(torch.randn(rows, width, generator=g))
        slots.copy_(torch.randperm(pool, generator=g)[:rows])
        slots[r] = -1
        y.copy_(torch.randint(-1, vocab, (rows,), generator=g))
        want = run(other)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(state, other) and all(torch.equal(p, q) for p, q in zip(got, want)), r
