"""8-bit moments of the AdamW step at values that are easy to get wrong: first moments that are NaN beside second ones that
are not."""
import pytest

from gpu_util import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


def state(n, scale=1.0 / 448):
    """A parameter, its gradient and zero moments of 8 bits."""
    import torch
    g = torch.Generator().manual_seed(n)
    x = {"p": torch.randn(n, generator=g).cuda(), "g": (1e-2 * torch.randn(n, generator=g)).cuda()}
    for k in ("m", "v"):
        x[k] = torch.zeros(n, dtype=torch.uint8, device="cuda")
        x[k + "_scale"] = torch.full((-(-n // 256),), scale, device="cuda")
    return x


def step(x, **over):
    import laplace_prefix_scans_amd as lp
    lp.laplex_adamw([x["p"]], [x["g"]], [x["m"]], [x["v"]], m_scale=[x["m_scale"]], v_scale=[x["v_scale"]],
                    **{**dict(lr=1e-3, step=2, betas=(0.9, 0.95)), **over})


@pytest.mark.parametrize("seed", [None, 3])
def test_a_first_moment_that_is_nan_stays_so(seed):
    """Whatever the second one is: a NaN's code is 0x7F (0xFF), and so is that of what a step makes of it."""
    import torch
    import laplace_prefix_scans_amd as lp
    n = 1500
    clean, x = state(n), state(n)
    for y in (clean, x):
        y["m"].fill_(0x30)  # 0.5 of the scale
        y["v"].fill_(0x38)
    where = torch.tensor([0, 31, 255, 256, 700, 1279, 1499], device="cuda")
    x["m"][where] = torch.tensor([0x7F, 0xFF, 0x7F, 0x7F, 0xFF, 0x7F, 0x7F], dtype=torch.uint8, device="cuda")
    step(clean, seed=seed)
    step(x, seed=seed)
    hit = torch.zeros(n, dtype=torch.bool, device="cuda")
    hit[where] = True
    m, v = lp.laplex_adamw_moments([x["m"]], [x["v"]], [x["m_scale"]], [x["v_scale"]])
    assert torch.isnan(m[0][hit]).all() and torch.isfinite(m[0][~hit]).all() and torch.isfinite(v[0]).all()
    assert torch.isnan(x["p"][hit]).all() and torch.equal(x["p"][~hit], clean["p"][~hit])
    # the second moments have nothing of it, and a block without one nothing at all
    assert torch.equal(x["v"], clean["v"]) and torch.equal(x["v_scale"], clean["v_scale"])
    blocks = torch.zeros(6, dtype=torch.bool, device="cuda")
    blocks[where // 256] = True
    rest = ~blocks.repeat_interleave(256)[:n]
    assert torch.equal(x["m"][rest], clean["m"][rest]) and torch.equal(x["m_scale"][~blocks], clean["m_scale"][~blocks])
