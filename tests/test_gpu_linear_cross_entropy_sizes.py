"""Linear softmax cross entropy at the largest sizes that it serves."""
import numpy as np
import pytest

import train_ref as ref
from gpu_util import have_gpu, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


def test_as_many_tokens_as_it_serves():
    """2^28 tokens, which repeat after 1024: the first 1024 against float64, the others the same bits."""
    import torch
    import laplace_prefix_scans_amd as lp
    torch.cuda.empty_cache()
    g = torch.Generator().manual_seed(1)
    table = torch.randn(3, 1, generator=g).bfloat16()
    x, y = torch.randn(1024, 1, generator=g).bfloat16(), torch.randint(-1, 4, (1024,), generator=g, dtype=torch.int32)
    turns = 1 << 18
    got = lp.laplex_linear_cross_entropy(x.cuda().repeat(turns, 1), table.cuda(), y.cuda().repeat(turns))
    want = ref.cross_entropy(x.float().numpy(), table.float().numpy(), y.numpy(), 1.0)
    for name, t in zip(("loss", "lse"), got):
        t = t.view(turns, 1024)
        assert (t == t[0]).all(), name
        first = host(t[0])
        assert (np.abs(first - want[name]) <= want["~" + name] + 2.0 ** -24 * np.abs(want[name])).all(), name


def moved(t):
    """t at an address that is a multiple of its element alone."""
    import torch
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:]
    return flat.copy_(t.reshape(-1)).view(t.shape)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 2, 3, 70, 300])
def test_a_workspace_of_just_the_size(dt, tokens):
    """For tensors that begin at multiples of 16 bytes, and for those that do not: the same bits, in just as much room as is
    asked for, with what lies behind it left alone; a smaller one is refused."""
    import torch
    import laplace_prefix_scans_amd as lp
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(tokens)
    x, table = torch.randn(tokens, 128, generator=g).to(dtype).cuda(), torch.randn(501, 128, generator=g).to(dtype).cuda()
    y, w = torch.randint(0, 501, (tokens,), generator=g).cuda(), torch.randn(tokens, generator=g).cuda()
    sizes, first = [], None
    for a, b in ((x, table), (moved(x), table), (x, moved(table)), (moved(x), moved(table))):
        need = [lp.laplex_linear_cross_entropy_workspace_bytes(back, a, b, y) for back in (False, True)]
        sizes.append(need)
        buf = [torch.full((n + 4096,), 85, dtype=torch.uint8, device="cuda") for n in need]
        ws = [t[:n] for t, n in zip(buf, need)]
        loss, lse = lp.laplex_linear_cross_entropy(a, b, y, ws=ws[0])
        got = (loss, lse, *lp.laplex_linear_cross_entropy_backward(a, b, y, lse, w, ws=ws[1]))
        assert all((t[n:] == 85).all() for t, n in zip(buf, need))
        first = got if first is None else first
        assert all(torch.equal(p, q) for p, q in zip(got, first))
        for i, call in enumerate((lambda s: lp.laplex_linear_cross_entropy(a, b, y, ws=s),
                                  lambda s: lp.laplex_linear_cross_entropy_backward(a, b, y, lse, w, ws=s))):
            with pytest.raises(lp.LaplexError):
                call(ws[i][:-1])
    assert sizes[1] == sizes[2] == sizes[3]
    copy = 501 * 128 * x.element_size()
    assert sizes[1][1] - sizes[0][1] >= copy and (sizes[1][0] - sizes[0][0] >= copy or tokens <= 2)


def test_the_memory_of_a_call():
    """One token and a training batch against 65536 x 2048 in bfloat16 (268 MB): nothing of the table's size beside the results
    and, in the backward, pieces of the logits' gradient of 512 MiB."""
    import torch
    import laplace_prefix_scans_amd as lp
    table = torch.zeros(65536, 2048, dtype=torch.bfloat16, device="cuda")
    x, y = torch.zeros(4096, 2048, dtype=torch.bfloat16, device="cuda"), torch.zeros(4096, dtype=torch.int64, device="cuda")
    lse = torch.zeros(4096, device="cuda")

    def most(f):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        f()
        torch.cuda.synchronize()
        return torch.cuda.max_memory_allocated() - before
    assert most(lambda: lp.laplex_linear_cross_entropy(x[:1], table, y[:1])) < 1 << 20
    # statistics of each token and 64 entries, parts of split logits
    assert most(lambda: lp.laplex_linear_cross_entropy(x, table, y)) < (4096 * 1024 * 8) + (32 << 20) + (1 << 20)
    # a copy of x, dx in float, parts, dx
    assert most(lambda: lp.laplex_linear_cross_entropy_backward(x, table, y, lse, lse, table_grad=False)) < (512 << 20) + 4096 * 2048 * 8 + (32 << 20) + (1 << 20)


@pytest.mark.parametrize("tokens", [1, 20])
def test_a_table_of_2_36_elements(tokens):
    """4194304 x 16384 in bfloat16, 137 GB, read as it lies: rows of zeros, but for some on both sides of 2^32 elements and at
    the end."""
    import torch
    import laplace_prefix_scans_amd as lp
    vocab, width = 1 << 22, 1 << 14
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < vocab * width * 2 + (8 << 30):
        pytest.skip("needs 146 GB of GPU memory")
    table = torch.zeros(vocab, width, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1000, (1 << 32) // width - 1, (1 << 32) // width, vocab - 2, vocab - 1]
    g = torch.Generator().manual_seed(3)
    some, x = (torch.randn(len(rows), width, generator=g) * 0.1).bfloat16(), torch.randn(tokens, width, generator=g).bfloat16()
    for r, row in zip(rows, some.cuda()):
        table[r].copy_(row)
    y = torch.tensor([rows[(i + 5) % len(rows)] if i % 4 < 3 else 77 for i in range(tokens)])
    loss, lse = lp.laplex_linear_cross_entropy(x.cuda(), table, y.cuda())
    del table
    torch.cuda.empty_cache()
    x64, s64 = x.double().numpy(), some.double().numpy()
    logits = x64 @ s64.T
    m = np.maximum(logits.max(1), 0.0)
    want = m + np.log(np.exp(logits - m[:, None]).sum(1) + (vocab - len(rows)) * np.exp(-m))
    hit = np.array([logits[i, rows.index(int(y[i]))] if int(y[i]) in rows else 0.0 for i in range(tokens)])
    # a sum of D products of random signs: 8 sqrt(D) roundings of its terms' magnitudes; 2^22 exponentials of zeros added up in
    # float32, in sums of sums: 8 sqrt(2^22) roundings at most; the logarithm, the maximum and the difference
    el = (np.abs(x64) @ np.abs(s64).T).max(1) * (8 * np.sqrt(width) + 4) * ref.U
    bound = 2 * el + (8 * np.sqrt(vocab) + 8) * ref.U + 8 * ref.U * (np.abs(want) + np.abs(m))
    assert (np.abs(host(lse) - want) <= bound).all()
    assert (np.abs(host(loss) - (want - hit)) <= bound + el).all()
