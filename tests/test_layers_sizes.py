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
