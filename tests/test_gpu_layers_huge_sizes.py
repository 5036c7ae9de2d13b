"""Sizes past 32 bits are refused (with the library's own status), not wrapped to small ones.  Nothing is launched:
the tensors are views of few elements, or memory that is reserved and never touched."""
import pytest

from gpu_util import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

WRAP = 1 << 32


def refused(call, *args, **kw):
    import laplace_prefix_scans_amd as lp
    with pytest.raises(lp.LaplexError) as e:
        call(*args, **kw)
    assert e.value.code == 2


def test_attention():
    import torch
    import laplace_prefix_scans_amd as lp
    x = torch.zeros(1, 1, 8, device="cuda")
    many = x.expand(1, WRAP + 1, 8)  # heads
    refused(lp.laplex_decay_attn, many, x, x, torch.zeros(1, device="cuda"))
    refused(lp.laplex_decay_attn_backward, many, x, x, torch.zeros(1, device="cuda"), x)
    long = x.expand(WRAP + 1, 1, 8)  # rows of a step
    refused(lp.laplex_decay_attn_step, long, long, long, torch.zeros(1, device="cuda"), torch.zeros(1, 1, 8, 8, device="cuda"))
    wide = torch.empty(1, 1, WRAP + 8, device="cuda", dtype=torch.bfloat16)  # channels
    one = torch.zeros(1, 1, 8, device="cuda", dtype=torch.bfloat16)
    refused(lp.laplex_decay_attn, wide, wide, one, torch.zeros(1, device="cuda"))
    del wide
    pool = torch.empty(WRAP + 1, 1, 1, 1, device="cuda")
    y = torch.zeros(1, 1, 1, device="cuda")
    refused(lp.laplex_decay_attn_step, y, y, y, torch.zeros(1, device="cuda"), pool)


def test_norm_and_embedding():
    import torch
    import laplace_prefix_scans_amd as lp
    row = torch.empty(1, WRAP + 8, device="cuda", dtype=torch.bfloat16)
    refused(lp.laplex_layer_norm, row)
    stat = torch.zeros(1, device="cuda")
    refused(lp.laplex_layer_norm_backward, row, row, stat, stat)
    ids = torch.zeros(1, dtype=torch.int64, device="cuda")
    refused(lp.laplex_embedding, ids, row)
    refused(lp.laplex_embedding, ids, row.view(-1, 1))
    refused(lp.laplex_embedding_backward, ids, row, 4)
    refused(lp.laplex_embedding_backward, ids, torch.zeros(1, 4, device="cuda"), WRAP + 3)
