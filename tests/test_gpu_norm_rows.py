"""Layer norm of more rows than a launch has places for, at every shape a row can take in registers and beyond:
blocks that take several rows in turn.  References and tolerances as in test_gpu_norm_embed."""
import pytest

import test_gpu_norm_embed as base
from gpu_util import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

# rows, width in bfloat16, width in float32
ROWS = [(17003, 301, 151), (17000, 512, 256), (12001, 1003, 503), (9001, 2001, 1001), (9000, 2048, 1024), (4207, 4095, 2047), (4200, 4096, 2048),
        (4203, 5001, 2501), (1101, 9001, 4501), (1100, 16384, 8192), (1103, 20001, 10001), (601, 33001, 16501)]


@pytest.mark.parametrize("shape", ROWS, ids=str)
@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_many_rows(shape, dt):
    rows, bf16, f32 = shape
    base.test_layer_norm((rows, bf16 if dt else f32), True, dt)


@pytest.mark.parametrize("shape", [(9001, 2000, 1000), (4203, 4096, 2048), (4203, 5000, 2500), (1101, 9000, 4500), (1101, 20000, 10000), (77, 33000, 16500)],
                         ids=str)
@pytest.mark.parametrize("dt", [0, 1], ids=["f32", "bf16"])
def test_results_do_not_depend_on_alignment(shape, dt):
    import torch
    import laplace_prefix_scans_amd as lp
    dtype = base.dtypes()[dt]
    rows, width = shape[0], shape[1] if dt else shape[2]
    g = torch.Generator(device="cuda").manual_seed(rows + width)

    def pair(*size):
        """The same values at 16-byte aligned and at odd addresses."""
        n = 1
        for s in size:
            n *= s
        buf = torch.randn(n + 1, device="cuda", generator=g).to(dtype)
        return buf[1:].view(size).clone(), buf[1:].view(size)

    x, dy, w, b = pair(rows, width), pair(rows, width), pair(width), pair(width)
    out = []
    for i in (0, 1):
        y, mean, rstd = lp.laplex_layer_norm(x[i], w[i], b[i])
        out.append((y, mean, rstd) + lp.laplex_layer_norm_backward(x[i], dy[i], mean, rstd, w[i]))
    for p, q in zip(*out):
        assert torch.equal(p, q)
