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


# ------------------------------------------------------------------ workspaces without copies that are never made
OVERLAP = 7
GB = 1 << 30


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("dims", [(65536, 2048), (257, 513), (1000, 96), (131072, 4096), (77, 16384), (50001, 64)], ids=str)
def test_workspaces_of_aligned_tensors_have_no_copy_of_rows_that_are_whole(L, dtype, dims):
    """Rows of whole 128-byte pieces are read as they lie, but for x in the backward; other rows are copied, but for a few
    tokens' forward, which goes by the table as it lies."""
    vocab, width = dims
    e = 2 if dtype else 4
    whole = width * e % 128 == 0
    padded = -(-width * e // 128) * 128
    for p in (0, 1):
        last = 0
        for tokens in [*range(0, 40), 300, 2048, 2049, 5000, 1 << 16, 1 << 20]:
            least = L.laplex_linear_cross_entropy_workspace_bytes_aligned(p, dtype, tokens, vocab, width)
            most = L.laplex_linear_cross_entropy_workspace_bytes(p, dtype, tokens, vocab, width)
            assert last <= least <= most and least % 256 == 0, (p, tokens)  # (it serves fewer tokens too)
            last = least
            few = p == 0 and tokens <= (2 if whole else 4) and width <= 32768 // e  # (4 rows in 128 KB)
            if whole and not few:
                assert most - least >= vocab * padded + (0 if p else tokens * padded), (p, tokens)
            elif not few:
                assert least == most >= vocab * padded
            if few:  # statistics and the targets' logits of 64 entries' tiles or 1024 blocks
                assert most == least <= 4 * (8 * max(vocab // 64 + 1, 1024) + 4) + 1024, tokens


@pytest.mark.parametrize("dtype", [0, 1])
def test_calls_ask_for_what_their_own_pointers_need(L, dtype):
    tokens, vocab, width = 300, 5000, 256
    e = 2 if dtype else 4
    least = [L.laplex_linear_cross_entropy_workspace_bytes_aligned(p, dtype, tokens, vocab, width) for p in (0, 1)]
    most = [L.laplex_linear_cross_entropy_workspace_bytes(p, dtype, tokens, vocab, width) for p in (0, 1)]

    def both(x_off, table_off, sizes):
        # the last check, of overlaps, fails where the one of the workspace has passed
        x, table, y, lse = vp(2 * GB + x_off), vp(4 * GB + table_off), vp(GB), vp(6 * GB)
        return (L.laplex_linear_cross_entropy(dtype, y, 8, tokens, x, table, vocab, width, 1.0, lse, lse, vp(8 * GB), sizes[0], None),
                L.laplex_linear_cross_entropy_backward(dtype, y, 8, tokens, x, table, vocab, width, 1.0, lse, vp(7 * GB), None, vp(6 * GB), dtype,
                                                       vp(12 * GB), vp(8 * GB), sizes[1], None))
    assert both(0, 0, least) == (OVERLAP, OVERLAP) and both(0, 0, [s - 1 for s in least]) == (WS, WS)
    for off in ((e, 0), (0, e), (8, 0), (0, 8), (e, e)):
        assert both(*off, least) == (WS, WS) and both(*off, most) == (OVERLAP, OVERLAP) and both(*off, [s - 1 for s in most]) == (WS, WS)
    assert both(16, 48, least) == (OVERLAP, OVERLAP)
    assert [L.laplex_linear_cross_entropy_workspace_bytes_aligned(p, dtype, 10, 10, w) for p, w in ((2, 10), (0, 0))] == [0, 0]
