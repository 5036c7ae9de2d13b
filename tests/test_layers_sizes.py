"""What the sequence layers' binding makes of strides and sizes, and how workspaces grow (no GPU)."""
import pytest


def test_strides_of_batches():
    """A batch of single tokens may be a slice of longer sequences; a longer one has to lie sequence after sequence."""
    import torch
    from laplace_prefix_scans_amd._layers import _strides
    x = torch.empty(3, 10, 2, 8)
    for t, want in ((x, (16, 8)), (x[:, -1:], (160, 8)), (x[:, :1, 1:], (160, 8)), (x[:1, 3:7], (16, 8)), (x[:, :0], (16, 8)),
                    (x[:1, 4:5], (160, 8))):
        assert _strides(t, t.shape, "x", True) == want
    with pytest.raises(ValueError):
        _strides(x[:, 2:4], x[:, 2:4].shape, "x", True)


@pytest.fixture(scope="module")
def L():
    import os
    import laplace_prefix_scans_amd as lp
    from laplace_prefix_scans_amd import _layers
    if not os.path.exists(lp.lib_path()):
        pytest.skip("liblaplex.so not built")
    return _layers._lib()


SHAPES = [(8, 8, 128, 128, 1), (8, 2, 128, 128, 3), (1, 1, 64, 64, 1), (3, 3, 100, 66, 2), (16, 16, 256, 256, 1), (64, 64, 64, 128, 4),
          (8, 8, 33, 200, 1), (300, 1, 16, 16, 1), (257, 257, 64, 64, 1), (259, 259, 100, 128, 1)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("dtype", [0, 1])
def test_an_attention_workspace_serves_fewer_tokens(L, shape, backward, dtype):
    """Nothing a call needs shrinks as its tokens grow: steps of a token around every small size, coarser ones beyond."""
    import ctypes
    from laplace_prefix_scans_amd._layers import _Shape
    heads, kv, dk, dv, seqs = shape
    last = 0
    for tokens in list(range(0, 1200)) + list(range(1200, 40000, 13)) + list(range(40000, 400000, 331)) + [1 << 24, (1 << 31) - 1]:
        s = _Shape(dtype, seqs, heads, kv, dk, dv, tokens, None, None, 1.0, 0, 0, 0, 0, 0, 0)
        need = L.laplex_decay_attn_workspace_bytes(backward, ctypes.byref(s))
        assert need >= last, tokens
        last = need


@pytest.mark.parametrize("shape", [(65536, 2048), (250000, 8), (300000, 16), (5000, 64), (1, 1), (262144, 4096)], ids=str)
def test_an_embedding_workspace_serves_fewer_tokens(L, shape):
    vocab, width = shape
    last = 0
    steps = sorted(set(range(0, 3000, 7)) | set(range(3000, 400000, 211)) | {x + d for x in (1024, 4096, 16384, 32768, 131072) for d in (-1, 0, 1, 2)})
    for tokens in steps + [1 << 22, 1 << 28]:
        need = L.laplex_embedding_workspace_bytes(tokens, vocab, width)
        assert need >= last, tokens
        last = need


def test_sizes_past_32_bits_are_refused():
    import laplace_prefix_scans_amd as lp
    from laplace_prefix_scans_amd._layers import _u32
    _u32("x", 0 | 1 | (1 << 32) - 1)
    for n in (1 << 32, (1 << 32) + 8, -1):
        with pytest.raises(lp.LaplexError) as e:
            _u32("x", 4 | n)
        assert e.value.code == 2
