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
