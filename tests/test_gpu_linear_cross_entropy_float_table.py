"""The float32 gradient of a bfloat16 table, for more tokens than two parts of the logits' gradient are held otherwise."""
import pytest

import train_ref as ref
from gpu_util import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


# vocabularies of less than a tile, of one, of several pieces of the workspace, and of more tokens than fit a piece of 128 entries
@pytest.mark.parametrize("dims", [(2049, 50, 72), (2500, 64, 64), (3000, 300, 130), (2100, 129, 256), (6000, 50001, 72), (4100, 70001, 40), (70000, 257, 64)],
                         ids=str)
def test_a_float_gradient_of_the_table_is_off_by_two_parts_rounding(dims):
    """Against float64 on the GPU.  G is held in two bfloat16 parts, whose second is off by half a step (2^-8) of what the first left
    out (2^-8 of G at most): 2^-16 of it, where one part is off by 2^-8."""
    import torch
    import laplace_prefix_scans_amd as lp
    tokens, vocab, width = dims
    g = torch.Generator().manual_seed(tokens)
    table = (2 * width ** -0.5 * torch.randn(vocab, width, generator=g)).bfloat16()
    y = torch.randint(0, vocab, (tokens,), generator=g)
    x = (torch.randn(tokens, width, generator=g) + torch.rand(tokens, 1, generator=g) * 5 * table[y].float()).bfloat16()
    y[::50] = -1
    x, table, y, w = x.cuda(), table.cuda(), y.cuda(), torch.randn(tokens, generator=g).cuda()
    _, lse = lp.laplex_linear_cross_entropy(x, table, y)
    dx, dtable = lp.laplex_linear_cross_entropy_backward(x, table, y, lse, w, dtype=torch.float32)
    assert dx.dtype == torch.bfloat16 and dtable.dtype == torch.float32
    dx2, coarse = lp.laplex_linear_cross_entropy_backward(x, table, y, lse, w)
    none, alone = lp.laplex_linear_cross_entropy_backward(x, table, y, lse, w, dtype=torch.float32, x_grad=False)
    assert none is None and torch.equal(alone, dtable)
    inside = y >= 0
    want, off = torch.zeros(vocab, width, dtype=torch.float64, device="cuda"), torch.zeros(vocab, width, dtype=torch.float64, device="cuda")
    t64 = table.double()
    for at in torch.arange(tokens, device="cuda").split(max(1, (1 << 27) // vocab)):
        x64, l = x[at].double(), x[at].double() @ t64.t()
        d = torch.where(inside[at], w[at], 0.0).double()[:, None]
        exact = torch.logsumexp(l, 1)
        assert ((lse[at].double() - exact)[inside[at]].abs() < 4e-5).all()
        p = torch.softmax(l, 1) * d
        # errors of a logit, of the lse (4e-5, above) and of the exponential, as in train_ref.cross_entropy
        e = p.abs() * ((width ** 0.5 * 8 + 4) * ref.U * (x64.abs() @ t64.abs().t()) + 4e-5 + 8 * ref.U + 3 * ref.U * (l - exact[:, None]).abs())
        p[torch.arange(at.numel(), device="cuda"), y[at].clamp(0, vocab - 1)] -= d[:, 0]
        # two parts, and the sum over the tokens
        e += (2.0 ** -16 + 2 * ref.U + 8 * tokens ** 0.5 * ref.U) * p.abs()
        want += p.t().contiguous() @ x64
        off += e.t().contiguous() @ x64.abs()
    assert ((dtable.double() - want).abs() <= off + 2.0 ** -24 * want.abs() + 1e-30).all()
    size = float(want.norm())
    two, one = float((dtable.double() - want).norm()) / size, float((coarse.double() - want).norm()) / size
    print("%s: off by %.2e of its size, in bfloat16 %.2e" % (dims, two, one))
    # the same result to bfloat16 (its rounding and the one part's), and the rows' gradient to two roundings
    assert float((dx.double() - dx2.double()).norm()) <= 2 * 2.0 ** -8 * float(dx2.double().norm())


def test_workspaces_are_as_large_as_for_bfloat16():
    """The same workspace serves both types of the table's gradient, and what lies behind it is left alone."""
    import torch
    import laplace_prefix_scans_amd as lp
    g = torch.Generator().manual_seed(1)
    for tokens, vocab, width in ((2049, 64, 64), (2049, 65, 64), (3000, 129, 72), (5000, 1000, 64), (2200, 40000, 64)):
        x, table = torch.randn(tokens, width, generator=g).bfloat16().cuda(), torch.randn(vocab, width, generator=g).bfloat16().cuda()
        y, w = torch.randint(0, vocab, (tokens,), generator=g).cuda(), torch.randn(tokens, generator=g).cuda()
        _, lse = lp.laplex_linear_cross_entropy(x, table, y)
        need = lp.laplex_linear_cross_entropy_workspace_bytes(True, x, table, y)
        buf = torch.full((need + (1 << 20),), 85, dtype=torch.uint8, device="cuda")
        want = lp.laplex_linear_cross_entropy_backward(x, table, y, lse, w, dtype=torch.float32)
        got = lp.laplex_linear_cross_entropy_backward(x, table, y, lse, w, dtype=torch.float32, ws=buf[:need])
        assert (buf[need:] == 85).all() and all(torch.equal(p, q) for p, q in zip(got, want))
