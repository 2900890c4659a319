"""Log probabilities without a GPU: how the sources store a candidate, and that
the inputs of tests/test_gpu_logprob_edges.py reach the ways that they are
for."""
import os
import re

import numpy as np
import pytest

from tests import logprob_util as lp

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "global_l2_norm_amd", "csrc")


def test_every_store_of_a_candidate_is_bounded():
    """More of a row's logits than there is room for may reach the threshold,
    in whatever order the waves come."""
    with open(os.path.join(CSRC, "gclip_logprob.hip"), encoding="utf-8") as f:
        code = f.read()
    stores = [m.start() for m in re.finditer(r"candidate\[[^;]*\]\s*=[^=]", code)]
    assert len(stores) == 1
    assert re.search(r"if \(at >= kCandidates\) return false;\s*\S*$", code[:stores[0]])
    assert f"kCandidates = {lp.CANDIDATES};" in code


@pytest.mark.parametrize("rows,size,dtype", [c[:3] for c in lp.CROWDED])
def test_crowded_rows_pass_the_room_from_other_waves(rows, size, dtype):
    """Rows of which little can come in few lanes, and much in those."""
    segments, turns, threads = lp.cut(rows, size, dtype)
    assert (segments, threads) == next(c[3:] for c in lp.CROWDED if c[:3] == (rows, size, dtype))
    x = lp.crowded(rows, size, dtype)
    columns = turns * threads * lp.UNIT[dtype]
    for row in x[:2]:
        scarce, n, elsewhere, nothing = lp.candidates(row[:columns], 20, dtype, turns, threads)
        assert scarce and nothing > 0 and (elsewhere > lp.CANDIDATES if threads > 64 else n > lp.CANDIDATES)
    # the last two: as much as there is room for, but for one and with one more
    got = [lp.candidates(row[:columns], 20, dtype, turns, threads) for row in x[2:]]
    assert all(g[0] for g in got) and [g[1] + g[3] for g in got] == [lp.CANDIDATES, lp.CANDIDATES + 1]


def test_no_targets_are_refused_by_name():
    import torch

    import global_l2_norm_amd as G
    x = torch.ones(4, 16)
    for arg in (x, x.clone().requires_grad_()):
        with pytest.raises(TypeError, match="needs targets"):
            G.token_log_probs(arg, None, entropy=True)


def test_tangents_of_the_results_gradients_are_refused():
    """As the other operators do: without a check the logits' gradient would
    come back without a tangent, as if it were constant."""
    import types

    import torch
    import torch.autograd.forward_ad as forward_ad

    from global_l2_norm_amd import logprob
    x, one, stats = torch.ones(4, 16), torch.ones(4), torch.ones(4, 2)
    ctx = types.SimpleNamespace(saved_tensors=(x, torch.zeros(4, dtype=torch.int64), stats, one), ignore=-100)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(one, one)
        for grads in ((dual, None), (None, dual), (one, dual), (dual, one)):
            with pytest.raises(NotImplementedError):
                logprob._TokenLogProbs.backward(ctx, *grads, None, None, None)
        with pytest.raises(ValueError, match="device"):  # no tangent: only that no GPU sees it
            logprob._TokenLogProbs.backward(ctx, one, one, None, None, None)


def test_rows_at_two_distances_are_refused_with_what_to_do():
    """Logits shifted by one position, of more than one sequence."""
    import torch

    from global_l2_norm_amd import layers
    logits = torch.ones(2, 5, 7)
    with pytest.raises(ValueError, match=r"logits: .* a contiguous\(\) copy is"):
        layers._ld(logits[:, :-1], "logits")
    assert layers._ld(logits[:, :-1].contiguous(), "logits") == 7
    assert layers._ld(logits[:1, :-1], "logits") == 7
