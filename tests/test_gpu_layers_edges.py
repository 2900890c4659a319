"""The layers on the GPU where values, shapes or numbers of rows are at an
edge: rows without spread, values near the formats' ends, and every shape of
the kernels with many rows.  Oracle and tolerances as in test_gpu_layers.py."""
import numpy as np
import pytest

from oracle import layers as L
from tests import layers_util as lu
from tests.test_gpu_layers import EPS, G, _need_gpu, factors, mask, vectors  # noqa: F401  (_need_gpu: a fixture)

pytestmark = pytest.mark.gpu


def f32(v, device="cuda"):
    import torch
    return torch.from_numpy(np.asarray(v, dtype=np.float32)).to(device)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size,rows", [(size, rows) for size in (5, 8, 64, 100, 771, 1111, 2049, 5000, 8192, 9001, 33001)
                                       for rows in (3, 37, 600, 2085) if rows * size < 5_000_000])
def test_gradients_of_rows_without_spread(size, rows, dtype):
    """n is 0 in every column, however large |mean| * rstd is, so dx is
    rstd (g - sum(g) / size) and dweight 0: lanes past a row's end and rows
    past the last one add nothing to either."""
    import torch
    g, rng = G(), np.random.default_rng([rows, size])
    for value, rstd in ((3e38, EPS ** -0.5), (-1e30, 3e9), (2.0, EPS ** -0.5)):
        what = f"{rows} x {size} {dtype} of {value} rstd {rstd}"
        print(what, flush=True)
        x = torch.full((rows, size), value, dtype=lu.torch_type(dtype), device="cuda")
        dy, dh = (lu.matrix(rng.standard_normal((rows, size)), dtype) for _ in range(2))
        w, _ = vectors(size, "f32", rng)
        mean, rs = x[:, 0].float().contiguous(), torch.full((rows,), rstd, device="cuda")
        xv, dyv, dhv, mv, sv, wv = (lu.values(t) for t in (x, dy, dh, mean, rs, w))
        dx, dw, db = g.layer_norm_backward(dy, x, mean, rs, w)
        assert not dw.any(), what + " dweight"
        lu.check_norm_gradient(lu.values(dx), lu.values(dw), lu.values(db), dyv, xv, mv, sv, wv, dtype, "f32", what)
        f = factors(rows, size)
        dx, dres, dw, db = g.residual_norm_backward(dy, dh, x, mean, rs, w, mask())
        assert not dw.any(), what + " residual dweight"
        lu.check_norm_gradient(lu.values(dx), lu.values(dw), lu.values(db), dyv, xv, mv, sv, wv, dtype, "f32",
                               what + " residual", dhv, f, lu.values(dres))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [9, 40, 64, 300, 1000, 2500, 5000, 9001, 16000])
def test_some_rows_overflow_among_many(size, dtype):
    """Rows whose squares leave binary32 and rows with a NaN among thousands,
    so that they share a wave or a workgroup with rows that do neither, over
    several turns: those keep their bits, the former are right."""
    import torch
    g, rng = G(), np.random.default_rng(size)
    rows = max(2100, min(20000, 12_000_000 // size))
    gen = torch.Generator(device="cuda").manual_seed(size)
    good = torch.randn(rows, size, generator=gen, device="cuda").to(lu.torch_type(dtype))
    x = good.clone()
    big = torch.from_numpy(rng.permutation(rows)[:rows // 5]).cuda()
    x[big] *= 2.0 ** 90
    bad = torch.from_numpy(rng.permutation(rows)[:rows // 50]).cuda()
    x[bad, size // 2] = float("nan")
    w, b = vectors(size, "f32", rng)
    y0, m0, s0 = g.layer_norm_forward(good, w, b, EPS)
    y, m, s = g.layer_norm_forward(x, w, b, EPS)
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[big] = rest[bad] = False
    assert torch.equal(y[rest], y0[rest]) and torch.equal(m[rest], m0[rest]) and torch.equal(s[rest], s0[rest])
    assert y[bad].isnan().all() and m[bad].isnan().all()
    kept = torch.zeros_like(rest)
    kept[big] = True
    kept[bad] = False
    at = kept.nonzero()[:, 0][:300]
    lu.check_norm(lu.values(x[at]), lu.values(y[at]), lu.values(m[at]), lu.values(s[at]), lu.values(w), lu.values(b),
                  EPS, dtype, f"{rows} x {size} {dtype}")


@pytest.mark.parametrize("size,lanes,chain", [(768, 64, 12), (64, 16, 4), (512, 64, 8)])
def test_mean_of_binary32_rows_around_zero(size, lanes, chain):
    """A row's mean is off by the roundings of its sum alone.  Each of them is
    at most u times its partial sum and taken as uniform there, so their
    root mean square is at most that of all the partial sums times u / sqrt 3
    (lanes add `chain` elements each, then pairs); the division adds one.
    4000 rows give the root mean square to 1.1 % (one deviation): 1.06 stands
    for five of them."""
    g, rng = G(), np.random.default_rng(size)
    rows = 4000
    x = lu.matrix(rng.standard_normal((rows, size)), "f32")
    _, mean, _ = g.layer_norm_forward(x, eps=EPS)
    v = lu.values(x)
    part = np.cumsum(v.reshape(rows, chain // 4, lanes, 4).transpose(0, 2, 1, 3).reshape(rows, lanes, chain), axis=2)
    squares = (part[:, :, 1:] ** 2).sum((1, 2))
    s = part[:, :, -1]
    while s.shape[1] > 1:
        s = s[:, 0::2] + s[:, 1::2]
        squares += (s ** 2).sum(1)
    exact = v.mean(1)
    unit = lu.U * np.sqrt(squares / size ** 2 + exact ** 2)
    ratio = np.sqrt((((lu.values(mean) - exact) / unit) ** 2).mean())
    assert ratio <= 1.06 / np.sqrt(3), ratio


@pytest.mark.parametrize("rows", [3, 600])
@pytest.mark.parametrize("size", [5, 8, 64, 100, 771, 1111, 2500, 8192, 10001, 40000])
def test_spread_of_almost_constant_rows(size, rows):
    """Binary32 rows whose elements are 0 to 3 steps above a large value.  The
    stored mean is its nearest neighbour and off by half a step at most, the
    subtractions from it are exact, and the squares are taken about the mean
    that they have themselves, so rstd is off by the sum's roundings as of any
    row (twice: the squares about the stored mean are at most twice those
    about the mean, for a deviation of half a step or more).  A row without
    spread has rstd = 1 / sqrt(eps) to four roundings."""
    import torch
    g, rng = G(), np.random.default_rng([size, rows])
    for value, step in ((1e9, 64.0), (-123456.0, 2.0 ** -7), (1e30, 2.0 ** 76)):
        base = np.full((rows, size), np.float64(np.float32(value)))
        x = base + step * rng.integers(0, 4, (rows, size))
        x[0] = base[0]
        t = lu.matrix(x, "f32")
        assert np.array_equal(lu.values(t), x)
        _, mean, rstd = g.layer_norm_forward(t, eps=EPS)
        _, wm, wr = L.norm(x, 1.0, 0.0, EPS)
        lu.within(lu.values(mean), wm, step / 2 * (1 + 1e-6), f"{value} {size} mean")
        spread = x.std(1)
        ok = (spread >= step / 2) | (spread == 0)
        tol = np.where(spread == 0, 4 * lu.U, (lu.PATH + 10) * lu.U) * wr
        lu.within(lu.values(rstd)[ok], wr[ok], tol[ok], f"{value} {size} rstd")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [5, 8, 64, 100, 771, 3000, 8192, 16000, 40000])
def test_elements_further_from_the_mean_than_binary32_reaches(size, dtype):
    """All of a row at one end of the format but for one element at the other:
    x - mean is above the largest binary32 value, y and the gradients are
    not."""
    g, rng = G(), np.random.default_rng(size)
    for rows in (3, 600):
        what = f"{rows} x {size} {dtype}"
        print(what, flush=True)
        x = np.full((rows, size), -3e38)
        x[np.arange(rows), rng.integers(0, size, rows)] = 3e38
        x[0] = -x[0]
        x = lu.matrix(x, dtype)
        w, b = vectors(size, "f32", rng)
        xv, wv, bv = lu.values(x), lu.values(w), lu.values(b)
        y, mean, rstd = g.layer_norm_forward(x, w, b, EPS)
        lu.check_norm(xv, lu.values(y), lu.values(mean), lu.values(rstd), wv, bv, EPS, dtype, what)
        dy = lu.matrix(rng.standard_normal((rows, size)), dtype)
        # the exact statistics: the mean's own error is not the gradient's
        _, m, r = L.norm(xv, 1.0, 0.0, EPS)
        mean, rstd = f32(m), f32(r)
        dx, dw, db = g.layer_norm_backward(dy, x, mean, rstd, w)
        lu.check_norm_gradient(lu.values(dx), lu.values(dw), lu.values(db), lu.values(dy), xv, lu.values(mean),
                               lu.values(rstd), wv, dtype, "f32", what)


@pytest.mark.parametrize("size", [5, 8, 64, 100, 771, 3000, 8192, 16000, 40000])
def test_variance_and_eps_whose_sum_leaves_binary32(size):
    g, rng = G(), np.random.default_rng(size)
    for eps, scale in ((3e38, 1.4e19), (3.4e38, 1.0e18), (2e38, 2e19)):
        for rows in (3, 600):
            x = lu.matrix(scale * rng.choice([-1.0, 1.0], (rows, size)), "f32")
            y, mean, rstd = g.layer_norm_forward(x, eps=eps)
            lu.check_norm(lu.values(x), lu.values(y), lu.values(mean), lu.values(rstd), np.ones(size), np.zeros(size),
                          float(np.float32(eps)), "f32", f"{size} {eps} {scale}")


MOST = 0x7ffffff0  # the largest extent of a matrix


def test_gradients_of_the_longest_row():
    """One row of 2^31 - 16 columns: more columns than a dispatch of a lane a
    column could count.  With mean 0 and rstd 1, n is x: dbias is dy and
    dweight dy * x exactly, and the two means are at most 2^-11 here, so dx is
    dy - c1 - x c2 to a few roundings."""
    import torch
    g = G()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randn(1, MOST, generator=gen, device="cuda") for _ in range(2))
    mean, rstd = torch.zeros(1, device="cuda"), torch.ones(1, device="cuda")
    dx, dw, db = g.layer_norm_backward(dy, x, mean, rstd, weight_grad=True, bias_grad=True)
    assert torch.equal(db, dy[0])
    part = 1 << 28
    c1 = c2 = 0.0
    for i in range(0, MOST, part):
        u, v = x[0, i:i + part], dy[0, i:i + part]
        assert torch.equal(dw[i:i + part], u * v), i
        c1 += float(v.sum(dtype=torch.float64)) / MOST
        c2 += float((u.double() * v.double()).sum()) / MOST
    assert abs(c1) < 2.0 ** -11 and abs(c2) < 2.0 ** -11
    for i in range(0, MOST, part):
        u, v = x[0, i:i + part].double(), dy[0, i:i + part].double()
        off = (dx[0, i:i + part].double() - (v - c1 - u * c2)).abs()
        # dx, dy - c1 and the product and sum with c2 round; c1 and c2 are
        # binary64 sums of units' binary32 sums
        assert bool((off <= 4 * lu.U * (v.abs() + u.abs() * 2.0 ** -11 + 2.0 ** -11)).all()), i


def test_dropout_of_more_units_than_32_bits_count():
    """In place over 17 rows of 2^31 - 16 bfloat16 elements, 68 GiB: the
    groups at both ends of each row, and those about the 2^32nd unit."""
    import torch
    g = G()
    rows = 17
    x = torch.ones(rows, MOST, dtype=torch.bfloat16, device="cuda")
    g.dropout_forward(x, mask(0.5), out=x)
    units = MOST // 8
    at = [(r, u) for r in range(rows) for u in (0, 1, units - 2, units - 1)]
    at += [divmod((1 << 32) + k, units) for k in range(-300, 300) if (1 << 32) + k < rows * units]
    at += [divmod((1 << 28) * k, units) for k in range(1, 17)]
    r, u = (np.array(v) for v in zip(*at))
    w = L.philox_words([u, r, np.full_like(u, 3), np.full_like(u, 7)], [0x90ABCDEF, 0x12345678])
    half = np.stack([v for k in w for v in (k & 0xFFFF, k >> 16)], 1)
    rt, ut = torch.from_numpy(r).cuda(), torch.from_numpy(u).cuda()
    got = x.view(rows, units, 8)[rt, ut]
    assert np.array_equal(lu.values(got), np.where(half >= 32768, 2.0, 0.0))


def test_written_buffers_are_seen_by_autograd():
    """A tensor that autograd saved and that a pass then writes fails its
    backward, as after any in-place operation; tensors that are only read keep
    their version."""
    import torch
    g = G()
    x, w = torch.randn(6, 32, device="cuda"), torch.ones(32, device="cuda")
    side = torch.cuda.Stream()
    y, mean, rstd = g.layer_norm_forward(x, w)
    h = x.clone()
    calls = [
        (lambda t, s: g.dropout_forward(x, mask(), out=t, stream=s), x),
        (lambda t, s: g.dropout_backward(x, mask(), out=t, stream=s), x),
        (lambda t, s: g.layer_norm_forward(x, w, out=t, stream=s), x),
        (lambda t, s: g.residual_norm_forward(x, h, w, out_h=t, stream=s), x),
        (lambda t, s: g.residual_norm_forward(x, h, w, out=t, stream=s), x),
        (lambda t, s: g.layer_norm_backward(x, h, mean, rstd, w, out=t, stream=s), x),
        (lambda t, s: g.residual_norm_backward(x, None, h, mean, rstd, w, mask(), out=t, stream=s), x),
        (lambda t, s: g.residual_norm_backward(x, None, h, mean, rstd, w, mask(), out_residual=t, stream=s), x),
        (lambda t, s: g.layer_norm_backward(x, h, mean, rstd, w, dweight=t, stream=s), w),
        (lambda t, s: g.layer_norm_backward(x, h, mean, rstd, w, dbias=t, weight_grad=False, stream=s), w),
    ]
    for stream in (None, side):
        for i, (call, like) in enumerate(calls):
            leaf = torch.ones_like(like).requires_grad_()
            saved = torch.zeros_like(like)
            read = [t._version for t in (x, h, w, mean, rstd)]
            loss = (leaf * saved).sum()
            torch.cuda.synchronize()
            call(saved, stream)
            torch.cuda.synchronize()
            with pytest.raises(RuntimeError, match="inplace"):
                loss.backward()
            assert read == [t._version for t in (x, h, w, mean, rstd)], i


def test_a_counter_that_moved_is_refused():
    """A mask holds its counter's address; another storage behind the same
    tensor would leave it pointing to memory that may be given out again."""
    import torch
    g = G()
    x = torch.ones(4, 64, device="cuda")
    for change in (lambda t: t.set_(torch.tensor([9], dtype=torch.int32, device="cuda")),
                   lambda t: setattr(t, "data", torch.tensor([9], dtype=torch.int32, device="cuda")),
                   lambda t: t.resize_(0)):
        counter = torch.zeros(1, dtype=torch.int32, device="cuda")
        m = mask(counter=counter)
        g.dropout_forward(x, m)
        counter.add_(1)
        assert np.array_equal(lu.values(g.dropout_forward(x, m)), factors(4, 64, step=8))
        old = counter.untyped_storage()  # kept: the address stays taken
        change(counter)
        for call in (lambda: g.dropout_forward(x, m), lambda: g.residual_norm_forward(x, x, mask=m),
                     lambda: g.dropout(x, m)):
            with pytest.raises(ValueError, match="storage"):
                call()
        del old


def test_probabilities_next_to_a_step():
    """t = floor(65536 p + 1/2) for the neighbours of its steps, from exact
    fractions: the scale 65536 / (65536 - t) tells t, or 0 for all dropped."""
    from fractions import Fraction
    from math import floor

    import torch
    g = G()
    x = torch.ones(64, 512, device="cuda")
    for k in (0, 1, 2, 3, 4, 1000, 32767, 32768, 65534, 65535):
        step = (k + 0.5) / 65536
        for p in (np.nextafter(step, 0.0), step, np.nextafter(step, 1.0)):
            t = floor(Fraction(p) * 65536 + Fraction(1, 2))
            y = lu.values(g.dropout_forward(x, mask(p)))
            scale = np.float64(np.float32(65536 / (65536 - t))) if t < 65536 else 0.0
            assert set(np.unique(y)) <= {0.0, scale}, (p, t)
            assert t > 65000 or scale in y, (p, t)
            assert mask(p).drops == (t > 0)


def test_a_frozen_input_costs_no_dropout(monkeypatch):
    """The backward pass of a residual step whose x needs no gradient runs
    without the mask: one matrix less, the same other gradients."""
    import torch
    from global_l2_norm_amd import layers
    g, rng = G(), np.random.default_rng(3)
    x, r, dy, dh = (lu.matrix(rng.standard_normal((40, 300)), "bf16") for _ in range(4))
    w, b = vectors(300, "f32", rng)
    m = mask()
    h, y, mean, rstd = g.residual_norm_forward(x, r, w, b, EPS, m)
    want = g.residual_norm_backward(dy, dh, h, mean, rstd, w, m)
    drops = []
    call, apply = layers.gclip_residual_backward, layers.gclip_dropout_apply
    monkeypatch.setattr(layers, "gclip_residual_backward",
                        lambda args, drop, stream: (drops.append(drop is not None), call(args, drop, stream)))
    monkeypatch.setattr(layers, "gclip_dropout_apply", lambda *args: (drops.append(True), apply(*args)))
    leaf = [t.clone().requires_grad_() for t in (x, r, w, b)]
    for frozen, expected in ((0, False), (1, True)):
        part = [t.detach() if i == frozen else t for i, t in enumerate(leaf)]
        rest = [t for i, t in enumerate(leaf) if i != frozen]
        drops.clear()
        got = torch.autograd.grad(g.residual_norm(*part, EPS, m), rest, [dh, dy])
        assert drops == [expected]
        assert all(torch.equal(p, q) for p, q in zip(got, [t for i, t in enumerate(want) if i != frozen]))
        drops.clear()
        got = torch.autograd.grad(g.residual_norm(*part, EPS, m)[0], rest[0], dh)[0]
        assert drops == [True] * expected
        assert torch.equal(got, dh if frozen == 0 else g.dropout_backward(dh, m))


def test_weights_of_another_shape_get_gradients_of_it():
    """weight and bias are taken by their elements in any shape."""
    import torch
    g, rng = G(), np.random.default_rng(4)
    x, dy = (lu.matrix(rng.standard_normal((20, 48)), "f32") for _ in range(2))
    w, b = vectors(48, "f32", rng)
    y, mean, rstd = g.layer_norm_forward(x, w, b, EPS)
    want = g.layer_norm_backward(dy, x, mean, rstd, w)
    for shape in ((48,), (1, 48), (6, 8)):
        leaf = [w.view(shape).clone().requires_grad_(), b.view(shape).clone().requires_grad_()]
        for out in (g.layer_norm(x, *leaf, EPS), g.residual_norm(x, torch.zeros_like(x), *leaf, EPS)[1]):
            got = torch.autograd.grad(out, leaf, dy)
            assert all(p.shape == shape and torch.equal(p.reshape(-1), q) for p, q in zip(got, want[1:]))


@pytest.mark.parametrize("dtype,size", [("f32", 10001), ("f32", 16001), ("bf16", 10001), ("bf16", 16001), ("f16", 2500),
                                        ("f16", 4001), ("f16", 5000), ("f16", 7001), ("f16", 10001), ("f16", 16001)])
def test_the_longest_shapes_of_many_rows(size, dtype):
    """Above the number of rows that takes other shapes, against the oracle."""
    from tests.test_gpu_layers import run_all
    run_all(521, size, dtype, "f32", "padded" if size % 2 else "plain", seed=9)


# a size for each shape of the kernels with rows in registers (the longest
# row of a shape is as long in every format), and one of the kernels beyond
SHAPES = [8, 13, 30, 61, 120, 190, 250, 380, 511, 700, 1001, 1500, 2041, 2900, 4001, 6001, 8100, 12001, 16001, 20001]
STREAM = 144 << 20  # bytes that a call moves, above which it streams


def normals(gen, rows, size, t):
    import torch
    return torch.randn(rows, size, generator=gen, device="cuda").to(t)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", SHAPES)
def test_every_shape_streams(size, dtype):
    """Calls that stream against calls on a quarter of the rows, which do not
    and have the same shape: the same bits.  With dropout the sum is that of
    the mask, its norm the norm's, and a sample of the gradients the oracle's;
    the weights' gradients are sums in any order."""
    import torch
    g = G()
    t, es = lu.torch_type(dtype), 4 if dtype == "f32" else 2
    part = max(2085 if es == 2 and size <= 2048 else 521, STREAM // (6 * size * es))
    rows = 4 * part
    assert size > 16384 or 2 * rows * size * es > STREAM >= 4 * part * size * es  # longer rows never stream
    gen = torch.Generator(device="cuda").manual_seed(size)
    x, r, dy, dh = (normals(gen, rows, size, t) for _ in range(4))
    w, b = vectors(size, "f32", np.random.default_rng(size))
    h, y, mean, rstd = g.residual_norm_forward(x, r, w, b, EPS)
    yn, mn, sn = g.layer_norm_forward(h, w, b, EPS)
    assert torch.equal(yn, y) and torch.equal(mn, mean) and torch.equal(sn, rstd)
    dres, _, dw, db = g.residual_norm_backward(dy, dh, h, mean, rstd, w)
    dn, dwn, dbn = g.layer_norm_backward(dy, h, mean, rstd, w)
    assert torch.equal(dwn, dw) and torch.equal(dbn, db)
    for at in range(0, rows, part):
        p = slice(at, at + part)
        for got, want in zip(g.residual_norm_forward(x[p], r[p], w, b, EPS), (h, y, mean, rstd)):
            assert torch.equal(got, want[p]), at
        got = g.layer_norm_forward(h[p], w, b, EPS)[0]
        assert torch.equal(got, y[p]), at
        if 5 * part * size * es <= STREAM or size > 8192:  # longer rows' gradients do not stream
            assert torch.equal(g.residual_norm_backward(dy[p], dh[p], h[p], mean[p], rstd[p], w)[0], dres[p]), at
            assert torch.equal(g.layer_norm_backward(dy[p], h[p], mean[p], rstd[p], w)[0], dn[p]), at
    for got, terms in ((dw, lambda p: dy[p].double() * (h[p].double() - mean[p].double()[:, None])
                        * rstd[p].double()[:, None]), (db, lambda p: dy[p].double())):
        total, size_of = torch.zeros(2, size, dtype=torch.float64, device="cuda")
        for at in range(0, rows, part):
            v = terms(slice(at, at + part))
            total += v.sum(0)
            size_of += v.abs_().sum(0)
        assert ((got.double() - total).abs() <= (rows + 4) * lu.U * size_of).all()
    # with dropout
    m = mask()
    f = g.dropout_forward(torch.ones(rows, size, device="cuda"), m)
    hd, yd, md, sd = g.residual_norm_forward(x, r, w, b, EPS, m)
    assert torch.equal(hd, (r.float() + torch.where(f != 0, x.float() * f, 0)).to(t))
    yn, mn, sn = g.layer_norm_forward(hd, w, b, EPS)
    assert torch.equal(yn, yd) and torch.equal(mn, md) and torch.equal(sn, sd)
    dx, dd, dwd, dbd = g.residual_norm_backward(dy, dh, h, mean, rstd, w, m)
    assert torch.equal(dd, dres) and torch.equal(dwd, dw) and torch.equal(dbd, db) and not dx[f == 0].any()
    some = slice(3, None, max(1, rows // max(2, 200_000 // size)))
    lu.check_norm_gradient(lu.values(dx[some]), None, None, lu.values(dy[some]), lu.values(h[some]),
                           lu.values(mean[some]), lu.values(rstd[some]), lu.values(w), dtype, "f32",
                           f"{rows} x {size} {dtype}", lu.values(dh[some]), lu.values(f[some]), lu.values(dres[some]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [5, 48, 257, 768, 2041, 2500, 5000, 9001, 16001, 40000])
def test_in_place_over_several_turns(size, dtype):
    """So many rows that a workgroup loads its next one before it has stored
    the present one."""
    import torch
    g = G()
    t = lu.torch_type(dtype)
    rows = 24_000_000 // size
    gen = torch.Generator(device="cuda").manual_seed(size)
    x, r, dy, dh = (normals(gen, rows, size, t) for _ in range(4))
    w, b = vectors(size, "f32", np.random.default_rng(size))
    m = mask()
    h, y, mean, rstd = g.residual_norm_forward(x, r, w, b, EPS, m)
    want = g.residual_norm_backward(dy, dh, h, mean, rstd, w, m)
    for over in (("x", "r"), ("r", "x")):
        s = dict(x=x.clone(), r=r.clone())
        got = g.residual_norm_forward(s["x"], s["r"], w, b, EPS, m, out_h=s[over[0]], out=s[over[1]])
        assert all(torch.equal(p, q) for p, q in zip(got, (h, y, mean, rstd))), over
    for over in (("dy", "dh"), ("dh", "h"), ("h", "dy")):
        s = dict(dy=dy.clone(), dh=dh.clone(), h=h.clone())
        got = g.residual_norm_backward(s["dy"], s["dh"], s["h"], mean, rstd, w, m, out=s[over[0]],
                                       out_residual=s[over[1]])
        assert all(torch.equal(p, q) for p, q in zip(got, want)), over
    s = h.clone()
    assert torch.equal(g.layer_norm_forward(s, w, b, EPS, out=s)[0], y)
    want = g.layer_norm_backward(dy, h, mean, rstd, w)
    for over in ("dy", "h"):
        s = dict(dy=dy.clone(), h=h.clone())
        got = g.layer_norm_backward(s["dy"], s["h"], mean, rstd, w, out=s[over])
        assert all(torch.equal(p, q) for p, q in zip(got, want)), over
    s = x.clone()
    assert torch.equal(g.dropout_forward(s, m, out=s), g.dropout_forward(x, m))


def test_the_readme_runs():
    """README.md's examples of the layers, each by itself."""
    import os
    import re

    import torch
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        blocks = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "residual_norm" in b]
    assert len(blocks) == 2
    g, rng = G(), np.random.default_rng(5)
    x, residual, dy, dh = (lu.matrix(rng.standard_normal((20, 64)), "bf16") for _ in range(4))
    for block in blocks:
        weight, bias = vectors(64, "f32", rng)
        for t in (weight, bias):
            t.grad = torch.ones_like(t)
        env = dict(G=g, seed=1, step=2, layer=3, mask=mask(), x=x, residual=residual, weight=weight, bias=bias, dy=dy,
                   dh=dh)
        exec(block, env)
        m = env["mask"]
        h, y, mean, rstd = g.residual_norm_forward(x, residual, weight, bias, mask=m)
        assert torch.equal(env["h"], h) and torch.equal(env["y"], y)
        if "dx" in env:
            want = g.residual_norm_backward(dy, dh, h, mean, rstd, weight, m)
            assert torch.equal(env["dx"], want[0]) and torch.equal(env["dresidual"], want[1])
            assert env["dw"] is weight.grad and torch.equal(weight.grad, 1 + want[2])
