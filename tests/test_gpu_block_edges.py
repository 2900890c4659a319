"""The block operators on the GPU: what tests/test_gpu_block.py does not
reach."""
import numpy as np
import pytest

from tests import layers_util as lu
from tests.test_gpu_block import G, bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need an MI355X")
    import global_l2_norm_amd  # noqa: F401  (fails loudly when libgclip.so is missing)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [1, 7, 64, 127, 128])
def test_one_scale_of_a_row_of_one_block(size, dtype):
    """It is a block's scale too, however the matrix came to be."""
    g, rng = G(), np.random.default_rng(size)
    x, up, dy = (lu.matrix(rng.standard_normal((9, size)), dtype) for _ in range(3))
    block = [g.pack8(t, "block") for t in (x, up)]
    want = g.activation_backward(dy, *block, "gelu", recompute=True)
    row = [g.pack8(t, "row") for t in (x, up)]
    assert bits(*row) == bits(*block)
    for made in (row, [g.Packed8(p.values, p.scales) for p in row]):
        assert bits(*g.activation_backward(dy, *made, "gelu", recompute=True)) == bits(*want)
        assert [p.args.mode for p in made] == [p.args.mode for p in block]
    # y in 8 bits as it was written: value and scale stand for it in every reader
    y8 = g.rms_norm_forward(x, packed="row")[0]
    again = g.Packed8(y8.values, y8.scales)
    assert bits(*g.activation_backward(dy, y8)) == bits(*g.activation_backward(dy, again))
    assert bits(g.unpack8(y8)) == bits(g.unpack8(again))


def test_one_scale_of_a_longer_row_is_refused_by_name():
    import torch
    g = G()
    x = torch.ones(4, 129, device="cuda")
    row, block = g.pack8(x, "row"), g.pack8(x)
    with pytest.raises(ValueError, match="gate must have a scale for each 128 columns"):
        g.activation_backward(x, row)
    with pytest.raises(ValueError, match="up must have a scale for each 128 columns"):
        g.activation_backward(x, block, row)
