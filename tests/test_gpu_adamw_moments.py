"""8-bit moments of the AdamW step at values that are easy to get wrong: first moments that are NaN beside second ones that
are not, and values midway between two codes; and how far the step's quotient may be off."""
import numpy as np
import pytest

import train_ref as ref
from gpu_util import have_gpu, host

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


def test_values_midway_between_codes_round_away_from_zero():
    """To nearest, ties away from zero: gradients that are whole codes and the points midway between them, with a largest of
    448 in each block, whose scale is then (1 - b1) exactly, and b1 = 0."""
    import torch
    import laplace_prefix_scans_amd as lp
    c = np.arange(127)
    grid = np.where(c >> 3 == 0, (c & 7) * 2.0 ** -9, (1 + (c & 7) / 8.0) * 2.0 ** ((c >> 3) - 7.0))
    mid = (grid[1:] + grid[:-1]) / 2
    row = np.zeros(256)
    row[0] = 448.0
    row[1:127] = mid
    row[127:253] = -mid
    x = state(256)
    x["g"] = torch.from_numpy(row).float().cuda()
    x["p"].zero_()
    step(x, seed=None, step=1, betas=(0.0, 0.0))
    assert float(x["m_scale"]) == 1.0
    codes = host(x["m"]).astype(int)
    assert (codes[1:127] == np.arange(1, 127)).all() and (codes[127:253] == 128 + np.arange(1, 127)).all() and codes[0] == 126
    m, _ = lp.laplex_adamw_moments([x["m"]], [x["v"]], [x["m_scale"]], [x["v_scale"]])
    assert (host(m[0])[1:127] == grid[1:]).all()


@pytest.mark.parametrize("eps", [1e-8, 1e-3, 0.0])
def test_the_steps_quotient_is_off_by_a_few_roundings(eps):
    """p = keep p - rate m / d, d = sqrt(v) / sqrt(1 - beta2^step) + eps, from moments as they are stored: the root, the
    rounded correction and the fused sum put d off by 3 U, its reciprocal (a step, 2 U) and product the quotient by 6 U, the rate's
    own rounding and product 8 U; keep's rounding and product 2 U of p; the difference U."""
    import torch
    import laplace_prefix_scans_amd as lp
    g = torch.Generator().manual_seed(2)
    n, lr, b1, b2, t, wd = 100001, 3e-3, 0.9, 0.95, 3, 0.1
    p = torch.randn(n, generator=g) * torch.exp(4 * torch.randn(n, generator=g))
    grad = 1e-3 * torch.randn(n, generator=g)
    m, v = 1e-3 * torch.randn(n, generator=g), (1e-3 * torch.randn(n, generator=g)) ** 2 + 1e-12
    p0 = p.double().numpy()
    c = [y.cuda() for y in (p, grad, m, v)]
    lp.laplex_adamw(*[[y] for y in c], lr=lr, step=t, betas=(b1, b2), eps=eps, weight_decay=wd)
    new, _, m, v = (host(y).astype(np.float64) for y in c)
    move = lr / (1 - b1 ** t) * m / (np.sqrt(v) / np.sqrt(1 - b2 ** t) + eps)
    want = (1 - lr * wd) * p0 - move
    assert (np.abs(new - want) <= ref.U * (8.5 * np.abs(move) + 2 * np.abs(p0) + np.abs(want))).all()
