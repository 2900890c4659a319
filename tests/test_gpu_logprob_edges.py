"""Log probabilities on the GPU: what tests/test_gpu_logprob.py does not reach,
to the same tolerances."""
import numpy as np
import pytest

from oracle import block as B
from tests import block_util as bu
from tests import layers_util as lu
from tests import logprob_util as lp
from tests.test_gpu_block import bits
from tests.test_gpu_logprob import G, chain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need an MI355X")
    import global_l2_norm_amd  # noqa: F401  (fails loudly when libgclip.so is missing)


@pytest.mark.parametrize("rows,size,dtype", [c[:3] for c in lp.CROWDED])
def test_crowded_rows(rows, size, dtype):
    """Few lanes with more candidates than there is room for, among which the
    first columns of those that cannot come are put."""
    import torch
    x = lu.matrix(lp.crowded(rows, size, dtype), dtype)
    few = min(rows, 4)
    row = torch.arange(rows, device="cuda") % 4
    t = x[row]
    xv = lu.values(x[:few])
    m, s, z, p, h = B.log_probs(xv)
    ids = B.top(xv, 32)
    for top in (1, 20, 32):
        r = G().token_log_probs_forward(t, top=top, stats=False)
        tops = np.take_along_axis(z, ids[:, :top], 1)
        tol = bu.log_prob_tolerances(xv, chain(size, dtype))[1]
        with np.errstate(invalid="ignore"):
            lu.within(lu.values(r.top_logp[:few]), tops, tol[:, None] + 2 * lu.U * np.abs(tops), f"top {top}")
        assert np.array_equal(r.top_ids[:few].cpu().numpy(), ids[:, :top]), top
        assert bits(r.top_ids) == bits(r.top_ids[row]) and bits(r.top_logp) == bits(r.top_logp[row])
