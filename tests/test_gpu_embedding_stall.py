"""The table's gradient where the sort of its tokens gives up (forced from the host as in test_gpu_failure_paths):
every row is NaN, nothing is read through the undefined order, and the next call is right again."""
import numpy as np
import pytest

import layers_ref as ref
from gpu_util import have_gpu, host
from test_gpu_norm_embed import near

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


@pytest.mark.parametrize("shape", [(140000, 5000, 24), (150001, 70000, 7), (20000, 300000, 8)], ids=str)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_forced_stall_gives_nan(shape, dt, monkeypatch):
    import torch
    import laplace_prefix_scans_amd as lp
    from laplace_prefix_scans_amd._layers import _lib
    tokens, vocab, width = shape
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    r = np.random.default_rng(tokens)
    ids = r.integers(-1, vocab, tokens)
    dy = torch.randn(tokens, width, generator=torch.Generator().manual_seed(tokens)).to(dtype)
    ids_d, dy_d = torch.from_numpy(ids).cuda(), dy.cuda()
    ws = torch.empty(_lib().laplex_embedding_workspace_bytes(tokens, vocab, width), dtype=torch.uint8, device="cuda")
    print("forced stall: embedding", shape, dt, flush=True)
    monkeypatch.setenv("LAPLEX_DEBUG_STALL", "4")
    grad = lp.laplex_embedding_backward(ids_d, dy_d, vocab, ws=ws)
    assert torch.isnan(grad).all()
    monkeypatch.delenv("LAPLEX_DEBUG_STALL")
    grad = lp.laplex_embedding_backward(ids_d, dy_d, vocab, ws=ws)
    want = ref.embedding_backward(ids, dy.float().numpy(), vocab, 1.0)
    env = ref.embedding_backward(ids, np.abs(dy.float().numpy()), vocab, 1.0)
    near("dtable", host(grad.float()), want, env, tokens, dt == "bf16")
