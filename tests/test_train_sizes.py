"""Sizes and workspaces of the training-step operators, on the host: what the header allows is served, what it does not is
refused.  No GPU work is started: every call fails a check before a launch."""
import ctypes
import os

import pytest

SIZE, WS = 2, 4
vp = ctypes.c_void_p
TB = 1 << 40


@pytest.fixture(scope="module")
def L():
    import laplace_prefix_scans_amd as lp
    from laplace_prefix_scans_amd import _training
    if not os.path.exists(lp.lib_path()):
        pytest.skip("liblaplex.so not built")
    return _training._lib()


def at(tb):
    return vp(tb * TB)  # never dereferenced


def calls(L, dtype, tokens, vocab, width):
    """The status of a forward and of a backward call, both with a workspace that is too small."""
    return (L.laplex_linear_cross_entropy(dtype, at(1), 8, tokens, at(2), at(200), vocab, width, 1.0, at(400), at(401), at(500), 256, None),
            L.laplex_linear_cross_entropy_backward(dtype, at(1), 8, tokens, at(2), at(200), vocab, width, 1.0, at(401), at(402), None, at(600), dtype,
                                                   at(800), at(500), 256, None))


# (tokens, vocab, width) at the limits of each alone, and of the products of two
INSIDE = [(300, 1 << 26, 1024), (1 << 28, 300, 256), (1, 1 << 26, 1 << 15), (1 << 21, 8, 1 << 20), (100, 1 << 21, 1 << 20), (1 << 28, 2, 1 << 13), (1, 1, 1 << 20)]
OUTSIDE = [(1 << 28, 300, 1 << 20), (300, 1 << 26, 1 << 20), (1 << 24, 8, 1 << 20), (300, 1 << 24, 1 << 20), (1 << 24, 1 << 20, 64), ((1 << 28) + 1, 2, 2),
           (2, (1 << 26) + 1, 2), (2, 2, (1 << 20) + 1)]


@pytest.mark.parametrize("dims", INSIDE, ids=str)
@pytest.mark.parametrize("dtype", [0, 1])
def test_cross_entropy_serves_what_the_header_allows(L, dtype, dims):
    size = [L.laplex_linear_cross_entropy_workspace_bytes(p, dtype, *dims) for p in (0, 1)]
    tokens, vocab, width = dims
    assert all(s > 0 and s % 256 == 0 for s in size)
    assert size[1] >= tokens * width * (2 if dtype else 4)  # (the backward's copy of x)
    assert calls(L, dtype, *dims) == (WS, WS)


@pytest.mark.parametrize("dims", OUTSIDE, ids=str)
@pytest.mark.parametrize("dtype", [0, 1])
def test_cross_entropy_refuses_what_it_does_not(L, dtype, dims):
    assert [L.laplex_linear_cross_entropy_workspace_bytes(p, dtype, *dims) for p in (0, 1)] == [0, 0]
    assert calls(L, dtype, *dims) == (SIZE, SIZE)
