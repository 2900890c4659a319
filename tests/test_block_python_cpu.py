"""The block operators' Python side without a GPU."""
import pytest


def test_a_row_of_one_block_is_one_matrix():
    """However it came to be: its mode is what its layout says."""
    import torch

    import global_l2_norm_amd as G
    from global_l2_norm_amd import _lib
    for size in (1, 64, 128, 129, 300):
        x = torch.empty(4, size)
        for name, mode in (("row", _lib.GCLIP_SCALES_ROW), ("block", _lib.GCLIP_SCALES_BLOCK)):
            p = G.Packed8._new(x, size, mode)
            again = G.Packed8(p.values, p.scales)
            assert p.args.mode == again.args.mode and p.args.ld == again.args.ld, (size, name)


def test_one_scale_of_a_longer_row_is_refused_by_name():
    import torch

    from global_l2_norm_amd import _lib, block
    x = torch.empty(4, 129)
    with pytest.raises(ValueError, match="gate must have a scale for each 128 columns"):
        block._blocks(block.Packed8._new(x, 129, _lib.GCLIP_SCALES_ROW), x, "gate")
    block._blocks(block.Packed8._new(x, 129, _lib.GCLIP_SCALES_BLOCK), x, "gate")
