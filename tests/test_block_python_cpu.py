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


def polynomial():
    """(its coefficients as the source has them, rounded to binary32, highest
    first; the error that the comment states)"""
    import os
    import re

    import numpy as np

    import global_l2_norm_amd as G
    with open(os.path.join(os.path.dirname(G.__file__), "csrc", "gclip_activation.hpp"), encoding="utf-8") as f:
        part = re.search(r"KIND == GCLIP_ACT_GELU\) \{(.*?)h = e \* t \* h;", f.read(), re.S)[1]
    c = [float(np.float32(v)) for v in re.findall(r"(?:float h = |, t, )(-?[0-9.]+)f", part)]
    assert len(c) == 9
    return c, float(re.search(r"for z up to 10, (\S+) off", part)[1])


def test_the_activations_polynomial_is_as_good_as_its_comment_says():
    """P(t) / (e^(z^2) erfc(z) / (2 t)) with t = 1 / (1 + 0.3 z)."""
    import numpy as np
    from scipy.special import erfcx
    c, said = polynomial()
    z = np.linspace(0.0, 10.0, 200001)
    t = 1.0 / (1.0 + 0.3 * z)
    off = np.abs(np.polyval(c, t) * 2.0 * t / erfcx(z) - 1.0).max()
    assert said / 2 < off <= said <= 2.0 ** -24


def test_erfc_in_binary32_is_as_good_as_the_tolerances_take_it():
    """t P(t) step by step in binary32, with a t off by two half steps either
    way: within the 16 half steps that block_util.act_tolerances counts."""
    import numpy as np
    from scipy.special import erfcx
    u = 2.0 ** -24
    c, _ = polynomial()
    x = np.concatenate([np.linspace(0.0, 14.0, 200001), np.logspace(-6, 1.1, 100001)]).astype(np.float32).astype(np.float64)
    down = lambda v: v.astype(np.float32).astype(np.float64)  # noqa: E731  (of a product and a sum in binary64: one rounding)
    want = erfcx(x / np.sqrt(2.0)) / 2.0
    for off in (-2, 0, 2):
        t = down(1.0 / down(x * float(np.float32(0.212132034355964)) + 1.0) * (1.0 + off * u))
        h = np.full_like(x, c[0])
        for k in c[1:]:
            h = down(h * t + k)
        assert np.abs(down(t * h) / want - 1.0).max() <= 16 * u, off
