"""The layers on the GPU against their binary64 oracle (oracle/layers.py), to
the tolerances that tests/layers_util.py derives; the mask and the stored sum
exactly."""
import numpy as np
import pytest

from oracle import layers as L
from tests import layers_util as lu

pytestmark = pytest.mark.gpu
EPS = 1e-5
P, SEED, STEP, SITE = 0.3, 0x1234567890ABCDEF, 7, 3


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need an MI355X")
    import global_l2_norm_amd  # noqa: F401  (fails loudly when libgclip.so is missing)


def G():
    import global_l2_norm_amd
    return global_l2_norm_amd


def mask(p=P, **over):
    return G().DropoutMask(p, SEED, **{"step": STEP, "site": SITE, **over})


def factors(rows, size, p=P, **over):
    """The factor of each element, rounded to binary32 as the kernels use it."""
    k = {"step": STEP, "site": SITE, **over}
    return L.kept(rows, size, p, SEED, **k) * float(np.float32(L.dropout_scale(p)))


def stored_sum(r, x, f, dtype):
    """h: the product rounded to binary32, the sum too, then to the format."""
    drop = np.where(f != 0, (x * f).astype(np.float32), np.float32(0))
    return lu.rounded(r.astype(np.float32) + drop, dtype)


def vectors(size, wt, rng):
    import torch
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(size)).to(lu.torch_type(wt)).cuda()
    b = torch.from_numpy(0.3 * rng.standard_normal(size)).to(lu.torch_type(wt)).cuda()
    return w, b


def run_all(rows, size, dtype, wt, layout="plain", p=P, seed=0, scale=1.0, shift=0.5, eps=EPS):
    """Every pass at one shape."""
    g, rng = G(), np.random.default_rng([rows, size, seed])
    what = f"{rows} x {size} {dtype} weights {wt} {layout}"
    print(what, flush=True)
    mk = lambda s=1.0, o=0.0: lu.matrix(s * rng.standard_normal((rows, size)) + o, dtype, layout)  # noqa: E731
    x, r, dy, dh = mk(scale, shift), mk(scale, shift), mk(), mk()
    w, b = vectors(size, wt, rng)
    xv, rv, dyv, dhv, wv, bv = (lu.values(t) for t in (x, r, dy, dh, w, b))
    m, f = mask(p), factors(rows, size, p)

    # dropout, exactly
    y = g.dropout_forward(x, m)
    want = np.where(f != 0, (xv * f).astype(np.float32), np.float32(0))
    assert np.array_equal(lu.values(y), lu.rounded(want, dtype)), what + " dropout"

    # the norm
    y, mean, rstd = g.layer_norm_forward(x, w, b, eps)
    y1, none, _ = g.layer_norm_forward(x, w, b, eps, stats=False)
    assert none is None and lu.values(y1).tobytes() == lu.values(y).tobytes()
    mv, sv = lu.values(mean), lu.values(rstd)
    lu.check_norm(xv, lu.values(y), mv, sv, wv, bv, eps, dtype, what)
    dx, dw, db = g.layer_norm_backward(dy, x, mean, rstd, w)
    assert dw.dtype == w.dtype
    lu.check_norm_gradient(lu.values(dx), lu.values(dw), lu.values(db), dyv, xv, mv, sv, wv, dtype, wt, what)

    # the residual step, with and without dropout
    for mm, ff in ((m, f), (None, np.ones((rows, size)))):
        h, y, mean, rstd = g.residual_norm_forward(x, r, w, b, eps, mm)
        hv, mv, sv = lu.values(h), lu.values(mean), lu.values(rstd)
        assert np.array_equal(hv, stored_sum(rv, xv, ff, dtype)), what + " h"
        lu.check_norm(hv, lu.values(y), mv, sv, wv, bv, eps, dtype, what + " residual")
        acc = vectors(size, "f32", rng)
        start = [lu.values(t) for t in acc]
        dx, dres, dw, db = g.residual_norm_backward(dy, dh, h, mean, rstd, w, mm, dweight=acc[0], dbias=acc[1],
                                                    accumulate=True)
        assert dw is acc[0] and db is acc[1] and (mm is not None or dx is dres)
        lu.check_norm_gradient(lu.values(dx), lu.values(dw), lu.values(db), dyv, hv, mv, sv, wv, dtype, "f32",
                               what + " residual", dhv, ff, lu.values(dres), *start)


SIZES = [1, 2, 7, 8, 9, 31, 63, 64, 65, 120, 128, 129, 250, 256, 257, 511, 512, 520, 768, 769, 1000, 1024, 1111, 1536,
         2040, 2047, 2048, 2049, 4096, 4100, 5000, 8192, 8200, 12288, 16384, 16400, 24000, 32768, 33001, 70001]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", SIZES)
def test_every_row_length(size, dtype):
    for rows, layout, wt in ((1, "plain", dtype), (5, "padded", "f32"), (3, "shifted", dtype)):
        run_all(rows, size, dtype, wt, layout)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,size", [(2, 64), (15, 768), (16, 96), (17, 8), (64, 300), (255, 64), (257, 33),
                                       (1000, 17), (513, 768), (4099, 8), (2053, 128), (300, 2048), (100, 5000),
                                       (40, 16384)])
def test_every_number_of_rows(rows, size, dtype):
    run_all(rows, size, dtype, "f32", "plain" if rows % 2 else "padded", seed=1)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [8, 16, 32, 64, 128, 192, 256, 384, 512, 768, 1024, 1536, 2048, 4096, 6144, 8192,
                                   12288])
def test_ragged_ends_in_every_wave(shape, dtype):
    """Rows that a few columns make too long for a register shape: the end of
    each lies alone in a unit, in every wave of a workgroup."""
    for extra in (1, 3, 6):
        run_all(37, shape + extra, dtype, "f32", "padded", seed=6)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [8, 15, 24, 33, 64, 97, 128, 129, 190, 193, 256, 257, 380, 385, 512, 513, 700, 768, 769,
                                  1024, 1025, 1300, 1537, 2040])
def test_shapes_of_many_rows(size, dtype):
    """Above the numbers of rows that take other shapes."""
    run_all(2085, size, dtype, "f32", "padded" if size % 2 else "plain", seed=7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [2049, 2500, 3100, 4097, 5001, 6145, 8192])
def test_long_shapes_of_many_rows(size, dtype):
    run_all(530, size, dtype, dtype, "padded" if size % 2 else "plain", seed=8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_short_rows(dtype):
    run_all(150001, 9, dtype, "f32", "plain", seed=2)
    run_all(70003, 64, dtype, "f32", "plain", seed=2)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,size", [(4, 3), (5, 70), (33, 768), (6, 4100), (3, 40000)])
def test_one_row_for_all(rows, size, dtype):
    run_all(rows, size, dtype, "f32", "one row", seed=3)


@pytest.mark.parametrize("seed", range(60))
def test_random_cases(seed):
    """Seeded shapes, formats, layouts and probabilities over the whole range;
    the weights' gradients also into buffers of the rows' format, added to."""
    rng = np.random.default_rng(1000 + seed)
    size = int(round(np.exp(rng.uniform(0, np.log(20000)))))
    rows = int(round(np.exp(rng.uniform(0, np.log(min(60000, max(2, 600000 // size)))))))
    dtype = str(rng.choice(["f32", "f16", "bf16"]))
    layout = str(rng.choice(["plain", "padded", "shifted", "one row"]))
    run_all(rows, size, dtype, str(rng.choice(["f32", dtype])), layout, p=float(rng.uniform(0, 1)), seed=seed,
            scale=float(rng.uniform(0.2, 3)), shift=float(rng.uniform(-3, 3)))
    g = G()
    x, dy = (lu.matrix(rng.standard_normal((rows, size)), dtype, layout) for _ in range(2))
    w, b = vectors(size, dtype, rng)
    y, mean, rstd = g.layer_norm_forward(x, w, b, EPS)
    buf = vectors(size, dtype, rng)
    start = [lu.values(t) for t in buf]
    dx, dw, db = g.layer_norm_backward(dy, x, mean, rstd, w, dweight=buf[0], dbias=buf[1], accumulate=True)
    lu.check_norm_gradient(lu.values(dx), lu.values(dw), lu.values(db), lu.values(dy), lu.values(x), lu.values(mean),
                           lu.values(rstd), lu.values(w), dtype, dtype, "added", dw0=start[0], db0=start[1])


@pytest.mark.parametrize("p", [0.0, 1e-6, 2.0 ** -16, 0.5, 0.999999, 1.0])
def test_probabilities(p):
    for size in (100, 3001):
        run_all(9, size, "f32", "f32", p=p, seed=4)
        run_all(9, size, "bf16", "bf16", p=p, seed=4)


@pytest.mark.parametrize("size", [8, 768, 2048, 5000, 40000])
def test_offset_far_above_the_spread(size):
    """Values around 300 with a spread of 1: the mean comes off first."""
    run_all(7, size, "f32", "f32", scale=1.0, shift=300.0, seed=5)


@pytest.mark.parametrize("dtype,scale", [("f32", 1e25), ("bf16", 1e25), ("f32", 1e37), ("f32", 1e-25), ("f16", 1e4)])
@pytest.mark.parametrize("size", [5, 64, 768, 3000, 40000])
def test_values_whose_squares_leave_binary32(dtype, scale, size):
    g, rng = G(), np.random.default_rng(size)
    x = lu.matrix(scale * rng.uniform(-1, 1, (6, size)), dtype)
    w, b = vectors(size, "f32", rng)
    y, mean, rstd = g.layer_norm_forward(x, w, b, EPS)
    lu.check_norm(lu.values(x), lu.values(y), lu.values(mean), lu.values(rstd), lu.values(w), lu.values(b), EPS, dtype,
                  f"{dtype} {scale} {size}")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [1, 3, 64, 768, 5000, 40000])
def test_rows_without_spread(dtype, size):
    """A constant row of a power of two: n is 0 exactly, y the bias, dx 0."""
    import torch
    g = G()
    x = torch.full((4, size), 2.0, dtype=lu.torch_type(dtype), device="cuda")
    w, b = vectors(size, "f32", np.random.default_rng(0))
    y, mean, rstd = g.layer_norm_forward(x, w, b, EPS)
    assert torch.equal(y, b.to(y.dtype).expand_as(y)) and (mean == 2.0).all()
    lu.within(lu.values(rstd), np.float64(EPS) ** -0.5, 316.3 * 4 * lu.U, "rstd")
    dx, dw, db = g.layer_norm_backward(torch.ones_like(x), x, mean, rstd, torch.ones_like(w))
    assert not dx.any() and not dw.any() and (db == 4).all()


@pytest.mark.parametrize("value", [0.1, 12345.678, -1e6 / 3, 3e38])
@pytest.mark.parametrize("size", [5, 64, 100, 768, 3001, 8192, 40000])
def test_constant_rows_of_any_value(value, size):
    """The mean is the value itself, whatever its binary32 sums round to, so y
    is the bias exactly."""
    import torch
    g = G()
    w, b = vectors(size, "f32", np.random.default_rng(2))
    for rows in (3, 600):
        x = torch.full((rows, size), value, device="cuda")
        y, mean, _ = g.layer_norm_forward(x, w, b, EPS)
        assert torch.equal(y, b.expand_as(y)) and (mean == x[0, 0]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("value", [0.1, 333.25, 60000.0])
@pytest.mark.parametrize("size", [5, 100, 768, 2047, 8192, 12287, 16384, 40000])
def test_constant_rows_of_16_bits(value, dtype, size):
    import torch
    g = G()
    w, b = vectors(size, "f32", np.random.default_rng(2))
    for rows in (3, 600):
        x = torch.full((rows, size), value, dtype=lu.torch_type(dtype), device="cuda")
        y, mean, _ = g.layer_norm_forward(x, w, b, EPS)
        assert torch.equal(y, b.to(y.dtype).expand_as(y)) and (mean == x[0, 0].float()).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [9, 64, 777, 3000, 40000])
def test_nan_and_infinity_stay_in_their_rows(dtype, size):
    import torch
    g, rng = G(), np.random.default_rng(size)
    base = rng.standard_normal((8, size))
    bad = base.copy()
    bad[1, size // 2], bad[3, 0], bad[5, size - 1] = np.nan, np.inf, -np.inf
    w, b = vectors(size, "f32", rng)
    good, x = lu.matrix(base, dtype), lu.matrix(bad, dtype)
    dy = lu.matrix(rng.standard_normal((8, size)), dtype)
    rows = [0, 2, 4, 6, 7]
    y0, m0, s0 = g.layer_norm_forward(good, w, b, EPS)
    y1, m1, s1 = g.layer_norm_forward(x, w, b, EPS)
    assert torch.equal(y0[rows], y1[rows]) and torch.equal(m0[rows], m1[rows])
    assert y1[[1, 3, 5]].isnan().all()
    d0, _, b0 = g.layer_norm_backward(dy, good, m0, s0, w)
    d1, w1, b1 = g.layer_norm_backward(dy, x, m1, s1, w)
    assert torch.equal(d0[rows], d1[rows]) and d1[[1, 3, 5]].isnan().all() and w1.isnan().all()
    assert torch.equal(b0, b1)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_dropped_elements_are_zero_whatever_they_held(dtype):
    import torch
    g = G()
    rows, size = 6, 203
    f = factors(rows, size) != 0
    x = lu.matrix(np.where(f, 1.0, np.nan), dtype)
    y = g.dropout_forward(x, mask())
    assert np.array_equal(lu.values(y) != 0, f) and not y.isnan().any()
    h, y, _, _ = g.residual_norm_forward(x, torch.ones_like(x), mask=mask())
    assert not h.isnan().any() and not y.isnan().any() and np.array_equal(lu.values(h) != 1, f)
    x = lu.matrix(np.where(f, 1.0, np.inf), dtype)
    assert not g.dropout_backward(x, mask()).isinf().any()


def test_masks_differ_by_every_argument_and_counter():
    import torch
    g = G()
    x = torch.ones(50, 300, device="cuda")
    counter = torch.tensor([4], dtype=torch.int32, device="cuda")
    for m, k in ((mask(step=9), dict(step=9)), (mask(site=4), dict(site=4)),
                 (mask(counter=counter), dict(step=STEP + 4)),
                 (mask(step=0xFFFFFFFE, counter=counter), dict(step=2)),
                 (mask().at(step=1, site=2), dict(step=1, site=2))):
        assert np.array_equal(lu.values(g.dropout_forward(x, m)), factors(50, 300, **k))


def test_no_weights_or_one_of_them():
    import torch
    g, rng = G(), np.random.default_rng(8)
    x, dy = (lu.matrix(rng.standard_normal((20, 300)), "bf16") for _ in range(2))
    w, b = vectors(300, "bf16", rng)
    one, zero = np.ones(300), np.zeros(300)
    xv, dyv = lu.values(x), lu.values(dy)
    for ww, bb in ((None, None), (w, None), (None, b)):
        wv, bv = one if ww is None else lu.values(w), zero if bb is None else lu.values(b)
        y, mean, rstd = g.layer_norm_forward(x, ww, bb, EPS)
        mv, sv = lu.values(mean), lu.values(rstd)
        lu.check_norm(xv, lu.values(y), mv, sv, wv, bv, EPS, "bf16", "weights")
        dx, dw, db = g.layer_norm_backward(dy, x, mean, rstd, ww)
        assert (dw is None) == (ww is None) and (db is None) == (ww is None)
        lu.check_norm_gradient(lu.values(dx), None, None, dyv, xv, mv, sv, wv, "bf16", "bf16", "weights")
    for want in ((True, False), (False, True)):
        dx, dw, db = g.layer_norm_backward(dy, x, mean, rstd, w, weight_grad=want[0], bias_grad=want[1])
        assert (dw is not None, db is not None) == want
        lu.check_norm_gradient(None, lu.values(dw) if want[0] else None, lu.values(db) if want[1] else None, dyv, xv,
                               mv, sv, lu.values(w), "bf16", "bf16", "one gradient")
    buf = torch.full((300,), 0.5, dtype=torch.bfloat16, device="cuda")
    g.layer_norm_backward(dy, x, mean, rstd, w, dbias=buf, weight_grad=False, accumulate=True)
    lu.check_norm_gradient(None, None, lu.values(buf), dyv, xv, mv, sv, lu.values(w), "bf16", "bf16", "accumulate",
                           db0=0.5)


@pytest.mark.parametrize("size", [48, 768, 3001, 40000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place(size, dtype):
    import torch
    g, rng = G(), np.random.default_rng(size)
    mk = lambda: lu.matrix(rng.standard_normal((37, size)), dtype, "padded")  # noqa: E731
    x, r, dy, dh = mk(), mk(), mk(), mk()
    w, b = vectors(size, "f32", rng)
    h, y, mean, rstd = g.residual_norm_forward(x, r, w, b, EPS, mask())
    dx, dres, dw, db = g.residual_norm_backward(dy, dh, h, mean, rstd, w, mask())

    def _restride(t):
        buf = torch.zeros(t.shape[0], t.stride(0), dtype=t.dtype, device="cuda")
        return buf[:, :t.shape[1]].copy_(t)

    x2, r2 = _restride(x), _restride(r)
    h2, y2, m2, s2 = g.residual_norm_forward(x2, r2, w, b, EPS, mask(), out_h=r2, out=x2)
    assert h2 is r2 and y2 is x2 and torch.equal(h2, h) and torch.equal(y2, y) and torch.equal(m2, mean)
    for over in (("dy", "dh"), ("dh", "h"), ("h", "dy")):
        t = dict(dy=_restride(dy), dh=_restride(dh), h=_restride(h))
        dx2, dres2, dw2, db2 = g.residual_norm_backward(t["dy"], t["dh"], t["h"], mean, rstd, w, mask(),
                                                        out=t[over[0]], out_residual=t[over[1]])
        assert torch.equal(dx2, dx) and torch.equal(dres2, dres) and torch.equal(dw2, dw) and torch.equal(db2, db), over
    y1, _, _ = g.layer_norm_forward(x, w, b, EPS)
    x2 = _restride(x)
    assert torch.equal(g.layer_norm_forward(x2, w, b, EPS, out=x2)[0], y1) and torch.equal(x2, y1)
    x2 = _restride(x)
    y1 = g.dropout_forward(x, mask())
    assert torch.equal(g.dropout_forward(x2, mask(), out=x2), y1)
    # the columns beside a written slice stay
    buf = torch.full((37, 3 * size), 7.0, dtype=x.dtype, device="cuda")
    buf[:, :size] = x
    g.layer_norm_forward(buf[:, :size], w, b, EPS, out=buf[:, size:2 * size])
    assert torch.equal(buf[:, :size], x) and (buf[:, 2 * size:] == 7.0).all()
    assert torch.equal(buf[:, size:2 * size], g.layer_norm_forward(x, w, b, EPS)[0])


def test_nothing_beside_the_outputs_is_written():
    """Guard elements around every output, at ends inside a vector."""
    import torch
    g, rng = G(), np.random.default_rng(1)
    for size in (1, 3, 13, 70, 770, 2051, 9001, 40001):
        for dtype in ("f32", "bf16"):
            t = lu.torch_type(dtype)
            x, r, dy, dh = (lu.matrix(rng.standard_normal((5, size)), dtype) for _ in range(4))
            w, b = vectors(size, "f32", rng)

            def guarded(shape, dt):
                n = int(np.prod(shape))
                buf = torch.full((n + 32,), 7.0, dtype=dt, device="cuda")
                return buf, buf[16:16 + n].view(shape)

            outs = [guarded((5, size), t) for _ in range(6)] + [guarded((size,), torch.float32) for _ in range(2)]
            h, y, mean, rstd = g.residual_norm_forward(x, r, w, b, EPS, mask(), out_h=outs[0][1], out=outs[1][1])
            g.residual_norm_backward(dy, dh, h, mean, rstd, w, mask(), out=outs[2][1], out_residual=outs[3][1],
                                     dweight=outs[6][1], dbias=outs[7][1])
            g.dropout_forward(x, mask(), out=outs[4][1])
            g.layer_norm_forward(x, w, b, EPS, out=outs[5][1])
            for buf, _ in outs:
                assert (buf[:16] == 7).all() and (buf[-16:] == 7).all(), (size, dtype)


def test_no_rows():
    import torch
    g = G()
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    y, mean, rstd = g.layer_norm_forward(x, w, w)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = g.layer_norm_backward(x, x, mean, rstd, w)
    assert not dw.any() and not db.any()
    buf = [torch.full((64,), 3.0, device="cuda") for _ in range(2)]
    g.layer_norm_backward(x, x, mean, rstd, w, dweight=buf[0], dbias=buf[1], accumulate=True)
    assert (buf[0] == 3).all() and (buf[1] == 3).all()
    h, y, mean, rstd = g.residual_norm_forward(x, x, w, w, EPS, mask())
    g.residual_norm_backward(x, None, h, mean, rstd, w, mask())
    assert g.dropout_forward(torch.empty(3, 0, device="cuda"), mask()).shape == (3, 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_lie_past_4_gib(dtype):
    """Three rows 2^31 + 24 elements apart: offsets past 32 bits."""
    import torch
    g, rng = G(), np.random.default_rng(3)
    t, size, ld = lu.torch_type(dtype), 771, (1 << 31) + 24
    vals = [rng.standard_normal((3, size)) for _ in range(3)]
    small = [lu.matrix(v, dtype) for v in vals]
    buf = torch.empty(2 * ld + 4 * 1024, dtype=t, device="cuda")
    far = [buf.as_strided((3, size), (ld, 1), 1024 * i).copy_(s) for i, s in enumerate(small)]
    w, b = vectors(size, "f32", rng)
    a = g.residual_norm_forward(*small[:2], w, b, EPS, mask())
    out_h, out = far[1], buf.as_strided((3, size), (ld, 1), 1024 * 3)
    dy = far[2]
    c = g.residual_norm_forward(far[0], far[1], w, b, EPS, mask(), out_h=out_h, out=out)
    for p, q in zip(a, c):
        assert torch.equal(p, q)
    p = g.residual_norm_backward(small[2], a[1], a[0], a[2], a[3], w, mask())
    q = g.residual_norm_backward(dy, c[1], c[0], c[2], c[3], w, mask(), out=far[0], out_residual=dy)
    for u, v in zip(p, q):
        assert torch.equal(u, v)
    assert torch.equal(g.dropout_forward(small[0], mask()),
                       g.dropout_forward(far[0].copy_(small[0]), mask(), out=far[0]))


@pytest.mark.parametrize("rows,size,dtype", [(16384, 2048, "bf16"), (16400, 2047, "f16"), (9000, 2048, "f32"),
                                             (13000, 1537, "f32"), (300000, 64, "bf16"), (2300, 8192, "f32")])
def test_calls_that_stream(rows, size, dtype):
    """Calls that move more than the caches hold take other loads and stores:
    the same bits as calls on parts of the rows, the weights' gradients as in
    binary64 (any order: rows u of the absolute values each)."""
    import torch
    g = G()
    t = lu.torch_type(dtype)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x, r, dy, dh = (torch.randn(rows, size, generator=gen, device="cuda").to(t) for _ in range(4))
    w, b = vectors(size, "f32", np.random.default_rng(1))
    m = mask()
    f = g.dropout_forward(torch.ones(rows, size, device="cuda"), m)
    h, y, mean, rstd = g.residual_norm_forward(x, r, w, b, EPS, m)
    assert torch.equal(h, (r.float() + torch.where(f != 0, x.float() * f, 0)).to(t))
    dx, dres, dw, db = g.residual_norm_backward(dy, dh, h, mean, rstd, w, m)
    one, _, _, _ = g.residual_norm_backward(dy, dh, h, mean, rstd, w)
    assert torch.equal(one, dres)
    assert not dx[f == 0].any()
    some = slice(5, None, 97)
    lu.check_norm_gradient(lu.values(dx[some]), None, None, lu.values(dy[some]), lu.values(h[some]),
                           lu.values(mean[some]), lu.values(rstd[some]), lu.values(w), dtype, "f32", "streamed",
                           lu.values(dh[some]), lu.values(f[some]), lu.values(dres[some]))
    at = 0
    while at < rows:  # parts of the rows, none of them few
        to = rows if rows - at < 2 * (rows // 4) else at + rows // 4
        part = slice(at, to)
        py, pm, ps = g.layer_norm_forward(h[part], w, b, EPS)
        assert torch.equal(py, y[part]) and torch.equal(pm, mean[part]) and torch.equal(ps, rstd[part]), at
        pd, _, _, _ = g.residual_norm_backward(dy[part], dh[part], h[part], mean[part], rstd[part], w)
        assert torch.equal(pd, dres[part]), at
        at = to
    n = (h.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for got, terms in ((dw, dy.double() * n), (db, dy.double())):
        tol = (rows + 4) * lu.U * terms.abs().sum(0)
        assert ((got.double() - terms.sum(0)).abs() <= tol).all()
    big = g.dropout_forward(torch.cat([x, x, x]), m)
    assert torch.equal(big[:rows], g.dropout_forward(x, m))


@pytest.mark.parametrize("rows,size,dtype", [(4099, 768, "f32"), (20000, 64, "bf16"), (3000, 2048, "bf16"),
                                             (700, 5000, "f16"), (300, 20000, "f32")])
def test_the_same_bits_every_run(rows, size, dtype):
    import torch
    g, rng = G(), np.random.default_rng(4)
    x, r, dy, dh = (lu.matrix(rng.standard_normal((rows, size)), dtype) for _ in range(4))
    w, b = vectors(size, "f32", rng)
    first = None
    for _ in range(4):
        f = g.residual_norm_forward(x, r, w, b, EPS, mask())
        now = f + g.residual_norm_backward(dy, dh, f[0], f[2], f[3], w, mask())
        if first is None:
            first = now
        assert all(torch.equal(p, q) for p, q in zip(first, now))


def test_graph_replays_take_the_counter():
    """Captured passes against eager ones over several replays with eager
    work between them; the counter gives each replay its own mask."""
    import torch
    g, rng = G(), np.random.default_rng(5)
    x, r, dy, dh = (lu.matrix(rng.standard_normal((130, 770)), "bf16") for _ in range(4))
    w, b = vectors(770, "f32", rng)
    counter = torch.zeros(1, dtype=torch.int32, device="cuda")
    m = mask(counter=counter)

    def step():
        f = g.residual_norm_forward(x, r, w, b, EPS, m)
        return f + g.residual_norm_backward(dy, dh, f[0], f[2], f[3], w, m) + (g.dropout_forward(x, m),)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    seen = []
    for i in range(4):
        counter.fill_(i)
        x.copy_(lu.matrix(rng.standard_normal((130, 770)), "bf16"))
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), i
        seen.append(got[-1] != 0)
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_another_stream():
    """Calls on a given stream: outputs and workspaces belong to it, and the
    operands' memory is not given out again before it has run."""
    import torch
    g, rng = G(), np.random.default_rng(6)
    vals = [rng.standard_normal((2000, 1500)) for _ in range(4)]
    w, b = vectors(1500, "f32", rng)
    x, r, dy, dh = (lu.matrix(v, "bf16") for v in vals)
    f = g.residual_norm_forward(x, r, w, b, EPS, mask())
    want = f + g.residual_norm_backward(dy, dh, f[0], f[2], f[3], w, mask())
    side = torch.cuda.Stream()
    for _ in range(3):
        t = [lu.matrix(v, "bf16") for v in vals]
        side.wait_stream(torch.cuda.current_stream())
        f = g.residual_norm_forward(t[0], t[1], w, b, EPS, mask(), stream=side)
        b2 = g.residual_norm_backward(t[2], t[3], f[0], f[2], f[3], w, mask(), stream=side)
        del t
        junk = [torch.full((2000, 1500), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(p, q) for p, q in zip(want, f + b2))
        del junk


@pytest.mark.parametrize("dtype,wt", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16")])
def test_autograd_gives_the_passes(dtype, wt):
    import torch
    g, rng = G(), np.random.default_rng(7)
    x, r, dy, dh = (lu.matrix(rng.standard_normal((60, 200)), dtype).view(4, 15, 200) for _ in range(4))
    w, b = vectors(200, wt, rng)
    m = mask()
    h, y, mean, rstd = g.residual_norm_forward(x, r, w, b, EPS, m)
    want = g.residual_norm_backward(dy, dh, h, mean, rstd, w, m)
    leaf = [t.clone().requires_grad_() for t in (x, r, w, b)]
    h2, y2 = g.residual_norm(*leaf, EPS, m)
    assert torch.equal(h2, h) and torch.equal(y2, y)
    got = torch.autograd.grad([h2, y2], leaf, [dh, dy])
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    # y alone, h alone, some inputs alone
    want = g.residual_norm_backward(dy, None, h, mean, rstd, w, m)
    got = torch.autograd.grad(g.residual_norm(*leaf, EPS, m)[1], leaf, dy)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    got = torch.autograd.grad(g.residual_norm(*leaf, EPS, m)[0], leaf, dh, allow_unused=True)
    assert torch.equal(got[0], g.dropout_backward(dh, m)) and torch.equal(got[1], dh) and got[2] is None
    got = torch.autograd.grad(g.residual_norm(x, leaf[1], w, leaf[3], EPS, m)[1], (leaf[1], leaf[3]), dy)
    assert torch.equal(got[0], want[1]) and torch.equal(got[1], want[3])
    # the norm, with a broadcast gradient
    y, mean, rstd = g.layer_norm_forward(x, w, b, EPS)
    ones = torch.ones_like(x)
    want = g.layer_norm_backward(ones, x, mean, rstd, w)
    got = torch.autograd.grad(g.layer_norm(leaf[0], leaf[2], leaf[3], EPS).sum(), (leaf[0], leaf[2], leaf[3]))
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    got = torch.autograd.grad(g.dropout(leaf[0], m), leaf[0], dy.transpose(0, 1).contiguous().transpose(0, 1))
    assert torch.equal(got[0], g.dropout_backward(dy, m))
    # a residual shared by all rows gets the sum of its rows' gradients
    row = x[0, 0].clone().requires_grad_()
    h, _ = g.residual_norm(x, row.expand_as(x), w, b, EPS, m)
    got = torch.autograd.grad(h, row, dh)[0]
    lu.within(lu.values(got), lu.values(dh).sum((0, 1)), 61 * lu.U * np.abs(lu.values(dh)).sum((0, 1))
              + lu.HALF[dtype] * 61 * np.abs(lu.values(dh)).sum((0, 1)), "shared residual")
    with torch.no_grad():
        assert torch.equal(g.layer_norm(leaf[0], leaf[2], leaf[3], EPS), y)


def test_gradients_against_differences():
    """Central differences of sum(dh h + dy y) in binary32 storage: the
    function's binary64 oracle at the kernel's own inputs, step 1e-3 (third
    derivatives of order one: error 1e-6 of a gradient of order one)."""
    import torch
    g, rng = G(), np.random.default_rng(9)
    rows, size, eps = 3, 20, 1e-2
    x, r, dy, dh = (lu.matrix(rng.standard_normal((rows, size)), "f32") for _ in range(4))
    w, b = vectors(size, "f32", rng)
    f = factors(rows, size)
    leaf = [t.clone().requires_grad_() for t in (x, r, w, b)]
    h, y = g.residual_norm(*leaf, eps, mask())
    got = [lu.values(t) for t in torch.autograd.grad([h, y], leaf, [dh, dy])]
    args = [lu.values(t) for t in (x, r, w, b)]
    dyv, dhv = lu.values(dy), lu.values(dh)

    def value(x, r, w, b):
        h = r + x * f
        return float((dhv * h).sum() + (dyv * L.norm(h, w, b, eps)[0]).sum())

    for k, grad in enumerate(got):
        for i in np.ndindex(grad.shape):
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[k][i] += 1e-3
            lo[k][i] -= 1e-3
            diff = (value(*hi) - value(*lo)) / 2e-3
            assert abs(diff - grad[i]) < 1e-4 * max(1.0, abs(diff)), (k, i, diff, grad[i])


def test_gradients_reach_the_gradient_list():
    """dweight and dbias accumulate over microbatches in the tensors of a
    GradList, which clips them."""
    import torch
    g, rng = G(), np.random.default_rng(10)
    w, b = vectors(768, "f32", rng)
    dw, db = torch.zeros_like(w), torch.zeros_like(b)
    grads = g.GradList([dw, db])
    total = np.zeros((2, 768))
    for i in range(3):
        x, dy = (lu.matrix(rng.standard_normal((100, 768)), "bf16") for _ in range(2))
        y, mean, rstd = g.layer_norm_forward(x, w, b)
        g.layer_norm_backward(dy, x, mean, rstd, w, dweight=dw, dbias=db, accumulate=True)
        o = L.norm_gradient(lu.values(dy), lu.values(x), lu.values(mean), lu.values(rstd), lu.values(w))
        total += np.stack(o[1:])
    grads.clip_(1.0, avg_factor=1 / 3)
    _, res = grads.read()
    assert abs(res["norm"] - np.sqrt((total ** 2).sum()) / 3) < 1e-5 * res["norm"] and res["clipped"]
    assert abs(float(torch.cat([dw, db]).double().norm()) - 1.0) < 1e-5


def test_bad_tensors_are_refused():
    import torch
    g = G()
    x = torch.ones(6, 32, device="cuda")
    w, y = torch.ones(32, device="cuda"), torch.empty(6, 32, device="cuda")
    y0, mean, rstd = g.layer_norm_forward(x, w, w)
    v, ty = ValueError, TypeError
    for error, call in [
        (v, lambda: g.layer_norm_forward(x.cpu(), w, w)), (ty, lambda: g.layer_norm_forward(x.double(), w, w)),
        (v, lambda: g.layer_norm_forward(x.t(), torch.ones(6, device="cuda"))),
        (v, lambda: g.layer_norm_forward(x, w[:31], w)), (v, lambda: g.layer_norm_forward(x, w.cpu())),
        (ty, lambda: g.layer_norm_forward(x, w.half(), w)), (ty, lambda: g.layer_norm_forward(x, w.half(), w.half())),
        (v, lambda: g.layer_norm_forward(x, torch.ones(64, device="cuda")[::2])),
        (v, lambda: g.layer_norm_forward(x, w, w, out=y[:5])),
        (ty, lambda: g.layer_norm_forward(x, w, w, out=y.half())),
        (v, lambda: g.layer_norm_forward(torch.tensor(1.0, device="cuda"))),
        (g.GclipError, lambda: g.layer_norm_forward(x, w, w, 0.0)),
        (g.GclipError, lambda: g.layer_norm_forward(torch.ones(3, 0, device="cuda"))),
        (g.GclipError, lambda: g.layer_norm_forward(x, w, w, out=x[:1].expand(6, 32))),
        (g.GclipError, lambda: g.layer_norm_forward(x[:5], w, w, out=x[1:])),
        (v, lambda: g.residual_norm_forward(x, x[:5], w, w)), (ty, lambda: g.residual_norm_forward(x, x.half(), w, w)),
        (v, lambda: g.residual_norm_forward(x, x[:, :1], w, w)),
        (v, lambda: g.layer_norm_backward(x[:5], x, mean, rstd, w)),
        (v, lambda: g.layer_norm_backward(x, x, mean[:5], rstd, w)),
        (ty, lambda: g.layer_norm_backward(x, x, mean.double(), rstd, w)),
        (v, lambda: g.layer_norm_backward(x, x, mean, rstd, w, accumulate=True)),
        (ty, lambda: g.layer_norm_backward(x, x, mean, rstd, w, dweight=torch.ones(32, device="cuda").half())),
        (v, lambda: g.residual_norm_backward(x, x, x, mean, rstd, w, out=y, out_residual=torch.empty_like(y))),
        (v, lambda: g.DropoutMask(-0.1, 1)), (v, lambda: g.DropoutMask(float("nan"), 1)),
        (v, lambda: g.DropoutMask(0.1, -1)), (v, lambda: g.DropoutMask(0.1, 1 << 64)),
        (v, lambda: g.DropoutMask(0.1, 1, step=1 << 32)), (v, lambda: g.DropoutMask(0.1, 1, counter=w)),
        (g.GclipError, lambda: g.dropout_forward(x[:5], mask(), out=x[1:])),
    ]:
        with pytest.raises(error):
            call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_the_example_learns(dtype):
    """examples/residual_lm.py: the loss of a uniform guess falls by more than
    half."""
    import importlib.util
    import os

    import torch
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "residual_lm.py")
    spec = importlib.util.spec_from_file_location("residual_lm", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, norms = mod.train(steps=60, dtype=getattr(torch, dtype))
    assert abs(losses[0] - np.log(257)) < 0.5 and losses[-1] < 0.5 * losses[0], losses
    assert all(np.isfinite(norms))
