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


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,size", [(6, 1), (7, 40), (9, 300), (600, 382), (8200, 100), (8200, 600), (40, 1000),
                                       (8200, 1025), (9, 2048), (600, 3000), (1600, 2500), (6, 70000), (300, 20000)])
def test_rows_that_count_for_nothing_may_hold_anything(rows, size, dtype):
    """NaNs and infinities of ignored rows, in the logits and in what the
    backward pass is given of them, have no effect."""
    import torch
    g, rng = G(), np.random.default_rng([rows, size])
    x = lu.matrix(rng.standard_normal((rows, size)), dtype)
    t = torch.from_numpy(rng.integers(0, size, rows)).cuda()
    none = torch.arange(rows, device="cuda") % 3 == 1
    t[none] = -100
    dl, dh = (torch.from_numpy(rng.standard_normal(rows)).float().cuda() for _ in range(2))
    spoilt = x.clone()
    spoilt[none] = float("nan")
    spoilt[none.nonzero()[0]] = float("inf")
    for top in (min(5, size), 0):
        clean = g.token_log_probs_forward(x, t, entropy=True, top=top)
        r = g.token_log_probs_forward(spoilt, t, entropy=True, top=top)
        assert bits(r.logp, r.entropy, r.stats) == bits(clean.logp, clean.entropy, clean.stats)
        assert not r.logp[none].any() and not r.entropy[none].any() and not r.stats[none].any()
        if top:
            assert (r.top_ids[none] == -1).all() and torch.isneginf(r.top_logp[none]).all()
    bad = lambda v: torch.where(none.reshape(-1, *[1] * (v.dim() - 1)), float("nan"), v)  # noqa: E731
    for de in (None, dh):
        want = g.token_log_probs_backward(dl, de, x, t, clean.stats, clean.entropy)
        d = g.token_log_probs_backward(bad(dl), None if de is None else bad(de), spoilt, t, bad(clean.stats), bad(clean.entropy))
        assert bits(d) == bits(want) and not d[none].any()


def test_forward_over_reverse_is_refused():
    import torch
    import torch.autograd.forward_ad as forward_ad
    g = G()
    x = torch.randn(3, 50, device="cuda").requires_grad_()
    t, one = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.ones(3, device="cuda")
    r = g.token_log_probs(x, t, entropy=True)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(one, one)
        for out in (r.logp, r.entropy):
            with pytest.raises(NotImplementedError):
                torch.autograd.grad(out, x, dual, retain_graph=True)
        assert torch.autograd.grad(r.logp, x, one)[0].shape == x.shape


def test_the_largest_rows_of_equal_logits_far_below_another():
    """Rows of the largest extent, one workgroup each: a wave's sum of equal
    logits, half a billion of them, is dropped where another wave has a far
    larger one.  All rows are the same memory."""
    import torch
    rows, size = 257, 0x7ffffff0
    assert lp.cut(rows, size, "bf16")[::2] == (1, 256)
    x = torch.full((1, size), -2e30, dtype=torch.bfloat16, device="cuda")
    x[0, -1] = 0.0
    t = torch.full((rows,), size - 1, device="cuda")
    r = G().token_log_probs_forward(x.expand(rows, size), t, entropy=True)
    for got in (r.logp, r.entropy, r.stats):
        assert not got.any(), got.flatten()[:4]
    x[0, -1] = -2e30
    r = G().token_log_probs_forward(x.expand(rows, size), t, entropy=True)
    # a lane adds 2^31 / 256 ones, 32 at a time
    want, tol = np.log(size), (size // (256 * 32) + 100) * lu.U
    for got in (-lu.values(r.logp), lu.values(r.entropy), lu.values(r.stats[:, 1])):
        assert np.abs(got - want).max() <= tol
