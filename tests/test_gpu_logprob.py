"""Log probabilities on the GPU against their binary64 oracle (oracle/block.py)
to the tolerances that tests/block_util.py derives; the alternatives' columns
exactly."""
import numpy as np
import pytest

from oracle import block as B
from tests import block_util as bu
from tests import layers_util as lu
from tests.test_gpu_block import bits

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "f16", "bf16"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need an MI355X")
    import global_l2_norm_amd  # noqa: F401  (fails loudly when libgclip.so is missing)


def G():
    import global_l2_norm_amd
    return global_l2_norm_amd


def chain(size, dtype):
    """Additions that a term goes through: 32 in a lane, the lane's sums (one
    for every 4 units of 16 bytes, of which 256 lanes share a row), the lanes,
    the waves, the segments; and as many rescalings, of two roundings each."""
    turns = -(-size // (256 * (4 if dtype == "f32" else 8) * 4))
    return 3 * (turns + 6 + 4 + 64) + 32


def logits(rows, size, seed, spread=3.0):
    rng = np.random.default_rng([rows, size, seed])
    x = spread * rng.standard_normal((rows, size))
    x[np.arange(rows), rng.integers(0, size, rows)] += 6.0
    return x, rng


def check(x, targets, top, dtype, what, layout="plain", entropy=True, ignore=-100, gradient=True):
    import torch
    g = G()
    print(what, flush=True)
    t = lu.matrix(x, dtype, layout)
    xv = lu.values(t)
    rows, size = xv.shape
    tt = torch.from_numpy(np.asarray(targets, dtype=np.int64)).cuda()
    r = g.token_log_probs_forward(t, tt, entropy=entropy, top=top, ignore_index=ignore)
    m, s, z, p, h = B.log_probs(xv)
    ts, tz, th = bu.log_prob_tolerances(xv, chain(size, dtype))
    counted = targets != ignore
    valid = (targets >= 0) & (targets < size)
    want = np.where(valid, z[np.arange(rows), np.where(valid, targets, 0)], np.nan)
    want = np.where(counted, np.where(np.isneginf(m) & valid, -np.inf, want), 0.0)
    with np.errstate(invalid="ignore"):
        lu.within(lu.values(r.logp), want, tz + 2 * lu.U * np.abs(want), what + " logp")
        stats = lu.values(r.stats)
        assert np.array_equal(stats[:, 0], np.where(counted, m, 0.0)), what + " m"
        lu.within(stats[:, 1], np.where(counted, s, 0.0), ts, what + " s")
        if entropy:
            lu.within(lu.values(r.entropy), np.where(counted, h, 0.0), th, what + " entropy")
        if top:
            ids = B.top(xv, top)
            assert np.array_equal(r.top_ids.cpu().numpy(), np.where(counted[:, None], ids, -1)), what + " ids"
            tops = np.where(counted[:, None], np.take_along_axis(z, ids, 1), -np.inf)
            lu.within(lu.values(r.top_logp), tops, tz[:, None] + 2 * lu.U * np.abs(tops), what + " top")
    if not gradient:
        return r
    rng = np.random.default_rng(7)
    dl, dh = (torch.from_numpy(rng.standard_normal(rows)).float().cuda() for _ in range(2))
    for de in (None, dh) if entropy else (None,):
        d = g.token_log_probs_backward(dl, de, t, tt, r.stats, r.entropy, ignore_index=ignore)
        dlv, dev = lu.values(dl), lu.values(dh) if de is not None else np.zeros(rows)
        ev = lu.values(r.entropy) if de is not None else np.zeros(rows)
        want = B.log_probs_gradient(xv, targets, dlv, dev, stats[:, 0], stats[:, 1], ev, ignore)
        with np.errstate(invalid="ignore", over="ignore"):
            zz = xv - stats[:, :1] - stats[:, 1:]
            pp = np.where(np.isfinite(zz), np.exp(zz), 0.0)
            a = np.where(pp > 0, np.abs(zz), 0.0)
            # p by two differences, the product and the power; the factor by
            # three roundings of its terms; the product and the target's sum
            rel = (2 * (a + np.abs(stats[:, 1:])) + 1.5 * a + 4) * lu.U
            f = np.abs(dlv[:, None]) + np.abs(dev[:, None]) * (a + np.abs(ev[:, None]))
            tol = np.nan_to_num(pp * f * (rel + 5 * lu.U)) + 2 * lu.U * np.nan_to_num(np.abs(want)) + 2.0 ** -126 * (1 + np.nan_to_num(f))
            lu.within(lu.values(d), want, bu.stored(np.nan_to_num(want), dtype, tol), what + f" gradient {de is not None}")
    return r


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [1, 2, 3, 7, 8, 9, 31, 64, 100, 255, 257, 1000, 1024, 2047, 2048, 2049, 4096, 8192, 8193,
                                  8449, 20000, 50304, 65537, 131072, 200001])
def test_every_row_length(size, dtype):
    for rows, layout, top in ((1, "plain", 20), (3, "padded", 1), (9, "shifted", 32), (5, "one row", 5)):
        x, rng = logits(rows, size, 0)
        check(x, rng.integers(0, size, rows), min(top, size), dtype, f"{rows} x {size} {dtype} {layout} top {top}", layout)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,size", [(2, 100), (17, 2000), (64, 8449), (255, 4097), (257, 1000), (513, 5000), (700, 8449),
                                       (2049, 300), (5000, 33)])
def test_every_number_of_rows(rows, size, dtype):
    x, rng = logits(rows, size, 1)
    targets = rng.integers(0, size, rows)
    targets[::5] = -100
    check(x, targets, 0, dtype, f"{rows} x {size} {dtype}", "padded" if rows % 2 else "plain")
    check(x, targets, min(7, size), dtype, f"{rows} x {size} {dtype} top", entropy=False, gradient=False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,size", [(1536, 2049), (1600, 2500), (1535, 2500), (1537, 8449), (1536, 16384), (1536, 16385)])
def test_many_rows_by_a_wave_each(rows, size, dtype):
    """As many as have a wave each and one fewer; rows at a lane's last turn
    and one column past it."""
    x, rng = logits(rows, size, 8)
    targets = rng.integers(0, size, rows)
    targets[::7] = -100
    x[3, size // 3:] = -np.inf
    x[4, :] = -np.inf
    x[5, :-1] = -np.inf
    targets[3], targets[4], targets[5] = 0, 1, size - 1
    layout = ("plain", "padded", "shifted")[size % 3]
    check(x, targets, 20, dtype, f"{rows} x {size} {dtype} top", layout, gradient=False)
    check(x, targets, 0, dtype, f"{rows} x {size} {dtype}", layout, entropy=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,size", [(63, 65536), (64, 65537), (96, 90001), (128, 131072), (128, 131080), (255, 50304),
                                       (256, 131072), (257, 40000), (200, 200001)])
def test_few_long_rows(rows, size, dtype):
    """A workgroup a row, of more turns with more rows, and in segments."""
    x, rng = logits(rows, size, 12)
    targets = rng.integers(0, size, rows)
    targets[::9] = -100
    x[1, 5:] = -np.inf
    x[2, :] = -np.inf
    targets[1], targets[2] = 3, 0
    layout = "plain" if rows % 2 else "padded"
    check(x, targets, 20, dtype, f"{rows} x {size} {dtype} top", layout, gradient=False)
    check(x, targets, 0, dtype, f"{rows} x {size} {dtype}", layout, entropy=False, gradient=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows_by_a_wave_each_streamed(dtype):
    x, rng = logits(4500 if dtype == "f32" else 9001, 8449, 9)
    check(x, rng.integers(0, 8449, len(x)), 3, dtype, f"streamed by waves {dtype}", gradient=False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [1, 4, 5, 16, 17, 31, 33, 64, 65, 127, 129, 250, 256, 257, 500, 513, 1000, 1025])
def test_many_short_rows(size, dtype):
    """8192 rows and more, where a row has fewer lanes."""
    for rows in (8192, 8201):
        x, rng = logits(rows, size, 10)
        targets = rng.integers(0, size, rows)
        targets[::11] = -100
        x[2, size // 2:] = -np.inf
        x[rows - 1, :] = -np.inf
        check(x, targets, 0, dtype, f"{rows} x {size} {dtype}", "padded" if rows % 2 else "plain")
        check(x, targets, min(3, size), dtype, f"{rows} x {size} {dtype} top", entropy=False, gradient=False)


@pytest.mark.parametrize("dtype", DTYPES)
def test_streamed(dtype):
    x, rng = logits(2100, 20011 if dtype == "f32" else 40011, 2)
    check(x, rng.integers(0, x.shape[1], len(x)), 3, dtype, f"streamed {dtype}")


@pytest.mark.parametrize("rows", [6, 600])
@pytest.mark.parametrize("size", [5, 40, 3000, 70000])
def test_masks(size, rows):
    """Padding, few allowed tokens, one, none; by -infinity and by the lowest
    finite number; of every type."""
    if rows * size > 10 ** 7:
        rows = 100
    for dtype in DTYPES:
        import torch
        low = float(torch.finfo(lu.torch_type(dtype)).min)
        for mask in (-np.inf, low):
            x, rng = logits(rows, size, 3)
            x[:, size - size // 5:] = mask
            x[1, np.arange(size) % 4 != 1] = mask
            x[2, :] = mask
            x[2, size // 2] = 1.0
            x[3, :] = mask
            x[rows - 1, :-1] = mask
            x[rows - 1, -1] = 2.0
            targets = rng.integers(0, max(1, size - size // 5), rows)
            targets[1], targets[2], targets[3], targets[rows - 1] = 1, size // 2, 0, size - 1
            check(x, targets, min(4, size), dtype, f"{rows} x {size} {dtype} mask {mask}")


@pytest.mark.parametrize("rows", [5, 600])
@pytest.mark.parametrize("size", [6, 3000, 70000])
def test_nans_and_infinities_stay_in_their_rows(size, rows):
    if rows * size > 10 ** 7:
        rows = 100
    for dtype in DTYPES:
        x, rng = logits(rows, size, 4)
        x[1, size // 2] = np.nan
        x[2, 3] = np.inf
        x[3, [0, 4]] = np.nan
        x[3, 2] = np.inf
        targets = rng.integers(0, size, rows)
        r = check(np.delete(x, [2, 3], 0), np.delete(targets, [2, 3]), 3, dtype, f"{rows} x {size} {dtype}")
        import torch
        t = lu.matrix(x, dtype)
        tt = torch.from_numpy(targets).cuda()
        q = G().token_log_probs_forward(t, tt, entropy=True, top=3)
        for i in (1, 2, 3):
            assert np.isnan([float(q.logp[i]), float(q.entropy[i]), float(q.stats[i, 1])]).all() and torch.isnan(q.top_logp[i]).all()
        assert q.top_ids[1:4].tolist() == B.top(lu.values(t)[1:4], 3).tolist()
        one = torch.ones(rows, device="cuda")
        d = G().token_log_probs_backward(one, one, t, tt, q.stats, q.entropy)
        assert torch.isnan(d[1:4]).all() and torch.isfinite(d[[0, *range(4, rows)]]).all()
        assert bits(q.logp[[0]]) == bits(r.logp[[0]])


@pytest.mark.parametrize("rows", [3, 600])
@pytest.mark.parametrize("size", [1, 6, 2048, 3000, 70000])
def test_rows_of_nans_and_nothing_that_can_come(size, rows):
    """A NaN is in the gradient though no number is the row's largest."""
    import torch
    if rows * size > 10 ** 7:
        rows = 100
    for dtype in DTYPES:
        x, rng = logits(rows, size, 11)
        x[0] = np.nan
        x[1] = -np.inf
        x[1, -1] = np.nan
        t, tt = lu.matrix(x, dtype), torch.zeros(rows, dtype=torch.int64, device="cuda")
        q = G().token_log_probs_forward(t, tt, entropy=True, top=1)
        one = torch.ones(rows, device="cuda")
        for de in (None, one):
            d = G().token_log_probs_backward(one, de, t, tt, q.stats, q.entropy if de is not None else None)
            assert torch.isnan(d[:2]).all() and torch.isfinite(d[2:]).all()
        for got in (q.logp, q.entropy, q.stats[:, 1], q.top_logp[:, 0]):
            assert torch.isnan(got[:2]).all() and torch.isfinite(got[2:]).all()
        assert q.top_ids[:2, 0].tolist() == [0, size - 1]


@pytest.mark.parametrize("size", [40, 2048, 5000, 131072])
def test_equal_logits_take_the_lowest_columns(size):
    """Rows of one value, of two, of halves of a step, in falling and rising
    order: more candidates than there is room for."""
    for dtype in DTYPES:
        for rows in (1, 4, 520 if size <= 5000 else 5):
            x = np.zeros((rows, size))
            if rows >= 4:
                x[1] = np.arange(size) % 2
                x[2] = -np.arange(size) / 64
                x[3] = np.arange(size) / 64
            x[0, 1::2] = -0.0
            check(x, np.zeros(rows, dtype=np.int64), 32, dtype, f"{rows} x {size} {dtype} equal", gradient=False)


@pytest.mark.parametrize("offset", [1e4, -3e5, 1e30])
def test_logits_of_large_magnitude(offset):
    """m and s apart keep what their sum would lose."""
    for rows, size in ((3, 1000), (600, 500)):
        x, rng = logits(rows, size, 5)
        step = np.spacing(np.float32(abs(offset))).astype(np.float64)
        x = offset + np.round(x) * step
        check(x, rng.integers(0, size, rows), 5, "f32", f"{offset} {rows} x {size}")


def test_targets_that_are_no_column():
    import torch
    x, rng = logits(6, 700, 6)
    t = np.array([0, 700, -1, 699, 1 << 40, -100])
    for ignore in (-100, 700, -1):
        check(x, t, 2, "bf16", f"ignore {ignore}", ignore=ignore)
    for x in (x, logits(2, 70000, 6)[0]):
        n = len(x)
        check(x, np.array([-5, x.shape[1] + 7, 3, 0, 1, 2])[:n], 2, "f32", "no column")


def test_without_targets_and_what_is_not_asked_for():
    import torch
    for rows, size in ((2, 50000), (700, 900)):
        x = lu.matrix(logits(rows, size, 8)[0], "bf16")
        t = torch.zeros(rows, dtype=torch.int64, device="cuda")
        full = G().token_log_probs_forward(x, t, entropy=True, top=4)
        part = G().token_log_probs_forward(x, top=4, stats=False)
        assert part.logp is None and part.entropy is None and part.stats is None
        assert bits(part.top_logp, part.top_ids) == bits(full.top_logp, full.top_ids)
        assert bits(G().token_log_probs_forward(x, t).logp) == bits(full.logp)
        assert bits(G().token_log_probs_forward(x, entropy=True).entropy) == bits(full.entropy)


def test_refusals():
    import torch
    g = G()
    x, t = torch.zeros(4, 50, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    r = g.token_log_probs_forward(x, t, entropy=True)
    one = torch.ones(4, device="cuda")
    for error, call in ((TypeError, lambda: g.token_log_probs_forward(x, t.int())), (ValueError, lambda: g.token_log_probs_forward(x, t[:3])),
                        (ValueError, lambda: g.token_log_probs_forward(x, t.cpu())), (ValueError, lambda: g.token_log_probs_forward(x, t, top=33)),
                        (ValueError, lambda: g.token_log_probs_forward(x, t, top=-1)), (ValueError, lambda: g.token_log_probs_forward(x[:, :3], t, top=4)),
                        (g.GclipError, lambda: g.token_log_probs_forward(x[:, :0], t)), (ValueError, lambda: g.token_log_probs_forward(x.t(), t)),
                        (ValueError, lambda: g.token_log_probs_backward(one, one, x, t, r.stats)),
                        (TypeError, lambda: g.token_log_probs_backward(one.double(), None, x, t, r.stats)),
                        (ValueError, lambda: g.token_log_probs_backward(one, None, x, t, r.stats[:, 0])),
                        (ValueError, lambda: g.token_log_probs_backward(one[:2], None, x, t, r.stats)),
                        (TypeError, lambda: g.token_log_probs_backward(one, None, x, t, r.stats, out=x.half()))):
        with pytest.raises(error):
            call()
    none = g.token_log_probs_forward(x[:0], t[:0], entropy=True, top=3)
    assert none.logp.shape == (0,) and none.top_ids.shape == (0, 3)
    assert g.token_log_probs_backward(one[:0], one[:0], x[:0], t[:0], none.stats, none.entropy).shape == (0, 50)


def test_numbers_that_are_none_are_refused():
    import torch
    g, x, t = G(), torch.zeros(4, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    for bad, error in ((1.0, TypeError), ("1", TypeError), (1 << 63, ValueError), (-(1 << 63) - 1, ValueError)):
        with pytest.raises(error):
            g.token_log_probs_forward(x, t, ignore_index=bad)
    r = g.token_log_probs_forward(x, t, ignore_index=-(1 << 63))
    for bad, error in ((1.0, TypeError), (1 << 63, ValueError)):
        with pytest.raises(error):
            g.token_log_probs_backward(r.logp, None, x, t, r.stats, ignore_index=bad)
    for bad, error in ((None, TypeError), ("x", ValueError), (0, g.GclipError)):
        with pytest.raises(error):
            g.rms_norm_forward(x, eps=bad)


@pytest.mark.parametrize("dtype", DTYPES)
def test_in_place_and_between_guards(dtype):
    import torch
    g = G()
    for rows, size in ((5, 9), (7, 1001), (300, 4099)):
        x, rng = logits(rows, size, 9)
        a = lu.matrix(x, dtype, "padded")
        t = torch.from_numpy(rng.integers(0, size, rows)).cuda()
        r = g.token_log_probs_forward(a, t, entropy=True)
        d = g.token_log_probs_backward(r.logp, r.entropy, a, t, r.stats, r.entropy)
        guard = torch.full((rows + 2, size + 9), 7.0, dtype=a.dtype, device="cuda")
        g.token_log_probs_backward(r.logp, r.entropy, a, t, r.stats, r.entropy, out=guard[1:-1, 3:3 + size])
        assert bits(guard[1:-1, 3:3 + size]) == bits(d)
        guard[1:-1, 3:3 + size] = 7.0
        assert (guard == 7.0).all()
        assert bits(g.token_log_probs_backward(r.logp, r.entropy, a, t, r.stats, r.entropy, out=a)) == bits(d)


def test_captured_replayed_and_on_two_streams():
    import torch
    g = G()
    shapes = ((4, 100000, 20), (600, 3000, 0))
    xs = [lu.matrix(logits(r, n, 10)[0], "bf16") for r, n, _ in shapes]
    ts = [torch.zeros(r, dtype=torch.int64, device="cuda") for r, _, _ in shapes]

    def step(i, stream=None):
        r = g.token_log_probs_forward(xs[i], ts[i], entropy=True, top=shapes[i][2], stream=stream)
        return (*r, g.token_log_probs_backward(r.logp, r.entropy, xs[i], ts[i], r.stats, r.entropy, stream=stream))

    want = [bits(*step(i)) for i in (0, 1)]
    streams = [torch.cuda.Stream() for _ in (0, 1)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [step(i, streams[i]) for i in (0, 1)]
        torch.cuda.synchronize()
        assert [bits(*o) for o in got] == want
    graphs = []
    for i in (0, 1):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(i)
        graphs.append((graph, out))
    for n in range(3):
        for x in xs:
            x.mul_(0.9)
        for i, (graph, out) in enumerate(graphs):
            eager = bits(*step(i))
            graph.replay()
            torch.cuda.synchronize()
            assert bits(*out) == eager, (n, i)


def test_large():
    """A matrix past 4 GiB, and a row of over 2^30 columns."""
    import torch
    g = G()
    rows, size = 20001, 131072
    x = torch.empty(rows, size, dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 5000):
        x[i:i + 5000].normal_(generator=torch.Generator("cuda").manual_seed(i))
    t = torch.full((rows,), size - 1, dtype=torch.int64, device="cuda")
    r = g.token_log_probs_forward(x, t, entropy=True, top=2)
    last = lu.values(x[-2:])
    m, s, z, p, h = B.log_probs(last)
    ts, tz, th = bu.log_prob_tolerances(last, chain(size, "bf16"))
    lu.within(lu.values(r.logp[-2:]), z[:, -1], tz + 2 * lu.U * np.abs(z[:, -1]), "logp")
    lu.within(lu.values(r.entropy[-2:]), h, th, "entropy")
    assert r.top_ids[-2:].tolist() == B.top(last, 2).tolist()
    tail = x[-2:].clone()
    g.token_log_probs_backward(r.logp, r.entropy, x, t, r.stats, r.entropy, out=x)
    assert bits(x[-2:]) == bits(g.token_log_probs_backward(r.logp[-2:], r.entropy[-2:], tail, t[-2:], r.stats[-2:], r.entropy[-2:]))
    del x
    torch.cuda.empty_cache()
    size = (1 << 30) + 1027
    x = torch.zeros(1, size, dtype=torch.bfloat16, device="cuda")
    x[0, size - 1], x[0, 1 << 30] = 20.0, 19.0
    t = torch.tensor([size - 1], device="cuda")
    r = g.token_log_probs_forward(x, t, entropy=True, top=3)
    assert r.top_ids.tolist() == [[size - 1, 1 << 30, 0]]
    total = (size - 2) + np.exp(20.0) + np.exp(19.0)
    want = 20.0 - np.log(total)
    # a lane adds 2^30 / (64 segments 256 lanes) logits, 32 at a time
    tol = (3 * ((1 << 30) // (64 * 256 * 32) + 100) + 32 + 40) * lu.U
    assert abs(float(r.logp) - want) <= tol
    d = g.token_log_probs_backward(torch.ones(1, device="cuda"), None, x, t, r.stats, out=x)
    assert abs(float(d[0, -1]) - (1 - np.exp(want))) <= tol + 2.0 ** -8


@pytest.mark.parametrize("dtype", DTYPES)
def test_under_autograd(dtype):
    import torch
    g, rng = G(), np.random.default_rng(11)
    x = torch.from_numpy(rng.standard_normal((2, 3, 500))).to(lu.torch_type(dtype)).cuda()
    t = torch.randint(0, 500, (2, 3), device="cuda")
    t[0, 1] = -100
    dl, dh = (torch.randn(2, 3, device="cuda") for _ in range(2))
    f = g.token_log_probs_forward(x, t, entropy=True, top=2)
    for use_logp, use_entropy in ((True, True), (True, False), (False, True)):
        a = x.clone().requires_grad_()
        r = g.token_log_probs(a, t, entropy=True, top=2)
        assert bits(*r) == bits(*f) and not r.top_logp.requires_grad and not r.stats.requires_grad
        loss = 0.0
        if use_logp:
            loss = loss + (r.logp * dl).sum()
        if use_entropy:
            loss = loss + (r.entropy * dh).sum()
        loss.backward()
        want = g.token_log_probs_backward(dl if use_logp else torch.zeros_like(dl), dh if use_entropy else None, x, t, f.stats, f.entropy)
        assert bits(a.grad) == bits(want)
    with torch.no_grad():
        assert g.token_log_probs(a, t).logp.grad_fn is None


def test_gradient_against_differences():
    """Of the forward pass itself, in binary32: a difference of logp over 2 h
    is off by its results' error over h and h^2."""
    import torch
    g, rng = G(), np.random.default_rng(12)
    x = rng.standard_normal((4, 12))
    t = torch.tensor([0, 5, 11, 3], device="cuda")
    dl, dh = rng.standard_normal(4), rng.standard_normal(4)

    def loss(v):
        r = g.token_log_probs_forward(torch.from_numpy(v).float().cuda(), t, entropy=True)
        return (lu.values(r.logp) * dl + lu.values(r.entropy) * dh).sum()
    h = 2.0 ** -7
    a = torch.from_numpy(x).float().cuda()
    r = g.token_log_probs_forward(a, t, entropy=True)
    got = lu.values(g.token_log_probs_backward(torch.from_numpy(dl).float().cuda(), torch.from_numpy(dh).float().cuda(), a, t, r.stats, r.entropy))
    ts, tz, th = bu.log_prob_tolerances(lu.values(a), chain(12, "f32"))
    tol = (np.abs(dl) * (tz + 8 * lu.U) + np.abs(dh) * th) / h
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        # the third derivatives of log p and of the entropy are at most 1 and 8
        assert abs((loss(up) - loss(down)) / (2 * h) - got[i]) <= tol.sum() + h * h / 6 * (np.abs(dl).sum() + 8 * np.abs(dh).sum()), i
