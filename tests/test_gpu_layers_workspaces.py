"""Calls with a workspace that was sized for more tokens, on both sides of the sizes where what a call keeps there
changes: the same bits as with one of its own, also where the workspace holds rubbish."""
import pytest

from gpu_util import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


def rubbish(n):
    import torch
    return torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("case", [(4185, 8, 4, 40, 128), (2108, 8, 8, 33, 200), (129, 257, 257, 16, 100), (129, 130, 130, 16, 24), (700, 3, 1, 64, 64)], ids=str)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_attention(case, dt):
    import torch
    import laplace_prefix_scans_amd as lp
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    tokens, heads, kv, dk, dv = case
    g = torch.Generator(device="cuda").manual_seed(tokens)
    q, k, v, go = (torch.randn(tokens + 100, h, d, generator=g, device="cuda").to(dtype) for h, d in ((heads, dk), (kv, dk), (kv, dv), (heads, dv)))
    rate = torch.linspace(0, 0.5, heads, device="cuda")
    big = [max(lp.laplex_decay_attn_workspace_bytes(b, q[:t], k[:t], v[:t], rate) for t in (tokens, tokens + 1, tokens + 63, tokens + 100))
           for b in (False, True)]
    for t in (tokens - 1, tokens, tokens + 1, tokens // 2):
        print("attention workspace", case, dt, t, flush=True)
        x = (q[:t], k[:t], v[:t], rate)
        assert torch.equal(lp.laplex_decay_attn(*x), lp.laplex_decay_attn(*x, ws=rubbish(big[0])))
        for a, b in zip(lp.laplex_decay_attn_backward(*x, go[:t])[:4], lp.laplex_decay_attn_backward(*x, go[:t], ws=rubbish(big[1]))[:4]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("case", [(32769, 3000, 256), (131073, 5000, 8), (32769, 300000, 40), (16385, 64, 33)], ids=str)
def test_embedding(case):
    import torch
    import laplace_prefix_scans_amd as lp
    from laplace_prefix_scans_amd._layers import _lib
    tokens, vocab, width = case
    g = torch.Generator(device="cuda").manual_seed(tokens)
    ids = torch.randint(-1, vocab, (tokens,), device="cuda", generator=g)
    dy = torch.randn(tokens, width, generator=g, device="cuda")
    need = _lib().laplex_embedding_workspace_bytes(tokens, vocab, width)
    for t in (tokens, tokens - 1, tokens - 300, tokens // 3):
        print("embedding workspace", case, t, flush=True)
        assert torch.equal(lp.laplex_embedding_backward(ids[:t], dy[:t], vocab), lp.laplex_embedding_backward(ids[:t], dy[:t], vocab, ws=rubbish(need)))
