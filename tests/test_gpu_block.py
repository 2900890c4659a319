"""The block operators on the GPU against their binary64 oracle
(oracle/block.py), to the tolerances that tests/block_util.py derives; the
stored sum exactly."""
import numpy as np
import pytest

from oracle import block as B
from tests import block_util as bu
from tests import layers_util as lu
from tests.test_gpu_layers import factors, mask, stored_sum

pytestmark = pytest.mark.gpu
EPS = 1e-5
DTYPES = ["f32", "f16", "bf16"]
KINDS = ["silu", "gelu", "gelu_tanh", "relu"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need an MI355X")
    import global_l2_norm_amd  # noqa: F401  (fails loudly when libgclip.so is missing)


def G():
    import global_l2_norm_amd
    return global_l2_norm_amd


def bits(*ts):
    import torch
    flat = []
    for t in ts:
        if t is None:
            continue
        flat += [t.values, t.scales] if isinstance(t, G().Packed8) else [t]
    return b"".join(t.detach().contiguous().reshape(-1).view(torch.uint8).cpu().numpy().tobytes() for t in flat)


# ---------------------------------------------------------------- 8 bits
@pytest.mark.parametrize("dtype", DTYPES)
def test_the_conversion_rounds_to_nearest_even(dtype):
    """Every value of the format, the middles between two and their
    neighbours, in blocks whose scale is 1."""
    import torch
    v = B.E4M3[:127]
    mid = (v[1:] + v[:-1]) / 2
    v = np.concatenate([v, mid, np.nextafter(mid.astype(np.float32), np.float32(1e9)),
                        np.nextafter(mid.astype(np.float32), np.float32(-1))]).astype(np.float64)
    v = np.concatenate([v, -v])
    v = np.resize(v, -(-len(v) // 127) * 127).reshape(-1, 127)
    x = torch.from_numpy(np.concatenate([np.full((len(v), 1), 448.0), v], 1)).to(lu.torch_type(dtype))
    p = G().pack8(x.cuda())
    q, s, _ = bu.packed_values(p)
    assert (s == 1).all()
    assert np.array_equal(q, B.round_e4m3(x.double().numpy()))
    assert np.array_equal(lu.values(p.dequantize()), q)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [1, 2, 3, 7, 8, 9, 31, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 384, 768, 1000,
                                  1111, 2047, 2048, 2049, 4096, 4099, 8200, 16384, 33001, 40000])
def test_pack_and_unpack(size, dtype):
    import torch
    g = G()
    for rows, layout, mode in ((1, "plain", "block"), (5, "padded", "row"), (37, "shifted", "block"), (3, "one row", "row"),
                               (130, "padded", "block"), (41, "plain", "row")):
        what = f"{rows} x {size} {dtype} {layout} {mode}"
        print(what, flush=True)
        rng = np.random.default_rng([rows, size])
        x = lu.matrix(rng.standard_normal((rows, size)) * np.exp(2 * rng.standard_normal((rows, 1))), dtype, layout)
        p = g.pack8(x, mode)
        # rows of a block have one scale either way, which is then a block's
        bu.check_packed(p, lu.values(x), mode if size > 128 else "block", what)
        _, _, stands = bu.packed_values(p)
        for other in DTYPES:
            y = g.unpack8(p, lu.torch_type(other))
            want = lu.rounded(stands.astype(np.float32), other)  # the product in binary32, then the format
            assert np.array_equal(lu.values(y), want), what + " " + other
        out = lu.matrix(np.zeros((rows, size)), dtype, "padded")
        assert g.unpack8(p, out=out) is out
        assert np.array_equal(lu.values(out), lu.rounded(stands.astype(np.float32), dtype)), what
        assert bits(g.pack8(x, mode)) == bits(p)


@pytest.mark.parametrize("mode", bu.MODES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_what_is_not_finite_becomes_nan_and_spares_the_scale(dtype, mode):
    import torch
    rng = np.random.default_rng(3)
    v = rng.standard_normal((9, 300))
    v[0, :] = 0
    v[1, 5], v[2, 130], v[3, 299] = np.nan, np.inf, -np.inf
    v[4, :] = np.nan
    v[5, 128:256] = np.inf
    v[6] *= 2.0 ** -14
    if dtype != "f16":
        v[7] *= 2.0 ** -130  # below what a scale reaches
        v[8] *= 2.0 ** 126
    x = lu.matrix(v, dtype)
    p = G().pack8(x, mode)
    bu.check_packed(p, lu.values(x), mode, f"{dtype} {mode}")
    assert torch.isfinite(p.scales).all()
    back = lu.values(p.dequantize())
    assert np.array_equal(np.isnan(back), ~np.isfinite(v))


# ---------------------------------------------------------------- RMS norm
def run_rms(rows, size, dtype, wt, layout="plain", p=0.3, seed=0, scale=1.0, eps=EPS, forms=(None, "row", "block")):
    """Every pass of the norm at one shape."""
    import torch
    g, rng = G(), np.random.default_rng([rows, size, seed])
    what = f"{rows} x {size} {dtype} weights {wt} {layout}"
    print(what, flush=True)
    mk = lambda s=1.0: lu.matrix(s * rng.standard_normal((rows, size)), dtype, layout)  # noqa: E731
    x, r, dy, dh = mk(scale), mk(scale), mk(), mk()
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(size)).to(lu.torch_type(wt)).cuda()
    xv, rv, dyv, dhv, wv = (lu.values(t) for t in (x, r, dy, dh, w))
    f = factors(rows, size, p)
    mode_of = lambda form: form if form is None or size > 128 else "block"  # noqa: E731

    for form in forms:
        for keep in (False, True):
            y, rstd, kept = g.rms_norm_forward(x, w, eps, packed=form, keep=keep)
            bu.check_rms(xv, lu.values(y) if form is None else y, lu.values(rstd), wv, eps, dtype, f"{what} {form} {keep}",
                         mode_of(form))
            assert (kept is None) == (not keep)
    bu.check_packed(kept, xv, "block", what + " kept")
    y, none, _ = g.rms_norm_forward(x, None, eps, stats=False)
    assert none is None
    bu.check_rms(xv, lu.values(y), None, np.ones(size), eps, dtype, what + " no weight")
    sv = lu.values(rstd)
    for held, hv in ((x, xv), (kept, bu.packed_values(kept)[2]), (g.pack8(x, "row"), bu.packed_values(g.pack8(x, "row"))[2])):
        dx, dw = g.rms_norm_backward(dy, held, rstd, w)
        assert dw.dtype == w.dtype
        bu.check_rms_gradient(lu.values(dx), lu.values(dw), dyv, hv, sv, wv, dtype, wt, what)

    for mm, ff in ((mask(p), f), (None, np.ones((rows, size)))):
        form = forms[-1]
        h, y, rstd, kept = g.residual_rms_norm_forward(x, r, w, eps, mm, keep=True, packed=form)
        h1, y1, _, _ = g.residual_rms_norm_forward(x, r, w, eps, mm, stats=False)
        hv, sv = lu.values(h), lu.values(rstd)
        assert np.array_equal(hv, stored_sum(rv, xv, ff, dtype)) and bits(h) == bits(h1), what + " h"
        bu.check_rms(hv, y if form else lu.values(y), sv, wv, eps, dtype, what + " residual", mode_of(form))
        bu.check_rms(hv, lu.values(y1), None, wv, eps, dtype, what + " residual")
        bu.check_packed(kept, hv, "block", what + " residual kept")
        for held, nv in ((h, hv), (kept, bu.packed_values(kept)[2])):
            acc = torch.from_numpy(rng.standard_normal(size)).float().cuda()
            start = lu.values(acc)
            dx, dres, dw = g.residual_rms_norm_backward(dy, dh, held, rstd, w, mm, dweight=acc, accumulate=True)
            assert dw is acc and (mm is not None or dx is dres)
            bu.check_rms_gradient(lu.values(dx), lu.values(dw), dyv, nv, sv, wv, dtype, "f32", what + " residual", dhv, ff,
                                  lu.values(dres), start)


SIZES = [1, 2, 7, 8, 9, 31, 63, 64, 65, 120, 128, 129, 192, 250, 256, 257, 384, 511, 512, 520, 768, 769, 1000, 1024, 1111,
         1536, 2040, 2047, 2048, 2049, 4096, 4100, 5000, 8192, 8200, 12288, 16384, 16400, 24000, 33001, 70001]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", SIZES)
def test_rms_every_row_length(size, dtype):
    for rows, layout, wt in ((1, "plain", dtype), (5, "padded", "f32"), (3, "shifted", dtype)):
        run_rms(rows, size, dtype, wt, layout)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,size", [(2, 64), (15, 768), (17, 8), (255, 64), (257, 33), (1000, 17), (513, 768), (4099, 8),
                                       (2053, 128), (2100, 2048), (600, 5000), (520, 16384)])
def test_rms_every_number_of_rows(rows, size, dtype):
    run_rms(rows, size, dtype, "f32", "plain" if rows % 2 else "padded", seed=1)


@pytest.mark.parametrize("rows,size", [(100, 768), (128, 130), (128, 4097), (129, 4097), (127, 8193), (129, 40), (2, 8193),
                                       (256, 16384), (257, 16384), (512, 4096), (513, 4096), (512, 4097), (300, 12289),
                                       (256, 8193), (600, 8200)])
def test_rms_weight_gradients_of_few_rows(rows, size):
    """As many rows as one launch serves, and one more."""
    for dtype, wt in (("bf16", "bf16"), ("f32", "f32"), ("f16", "f32")):
        run_rms(rows, size, dtype, wt, "shifted" if rows % 2 else "plain", seed=4, forms=("row",))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [8, 16, 32, 64, 128, 192, 256, 384, 512, 768, 1024, 1536, 2048, 4096, 6144, 8192, 12288])
def test_rms_shapes_of_many_rows(shape, dtype):
    """Rows that fill a shape, pass it by one column or fall short of it by one,
    over more of them than the few rows' shapes take."""
    for size in (shape - 1, shape, shape + 1):
        if size >= 8:
            run_rms(521, size, dtype, dtype, "shifted" if size % 2 else "plain", seed=2, forms=(None, "block"))


@pytest.mark.parametrize("rows,size,dtype", [(13000, 1537, "f32"), (300001, 64, "bf16"), (2300, 8192, "f32"),
                                             (9001, 2048, "f16"), (40000, 768, "bf16"),
                                             (1200, 16383, "bf16"), (1000, 12000, "f32")])
def test_rms_streamed(rows, size, dtype):
    run_rms(rows, size, dtype, "f32", seed=3, forms=(None, "row"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [5, 8, 100, 771, 2500, 8192, 10001, 40000])
def test_rms_rows_that_overflow_among_many_that_do_not(size, dtype):
    """The squares of some rows leave binary32; the others keep their bits."""
    import torch
    g, rng = G(), np.random.default_rng(size)
    for rows in (7, 700):
        v = rng.standard_normal((rows, size))
        plain = lu.matrix(v, dtype)
        big = v.copy()
        big[3] *= 2.0 ** 120
        big[rows - 1] = 3e38 * np.sign(v[-1])
        x = lu.matrix(big, dtype)
        w = torch.from_numpy(1 + 0.3 * rng.standard_normal(size)).float().cuda()
        a, b = (g.rms_norm_forward(t, w, EPS, keep=True) for t in (plain, x))
        bu.check_rms(lu.values(x), lu.values(b[0]), lu.values(b[1]), lu.values(w), EPS, dtype, f"{rows} x {size}")
        same = [i for i in range(rows) if i not in (3, rows - 1)]
        assert bits(a[0][same]) == bits(b[0][same]) and bits(a[1][same]) == bits(b[1][same])
        for mode in bu.MODES:
            y = g.rms_norm_forward(x, w, EPS, packed=mode)[0]
            bu.check_rms(lu.values(x), y, None, lu.values(w), EPS, dtype, f"{rows} x {size} {mode}", mode if size > 128 else "block")


@pytest.mark.parametrize("dtype", DTYPES)
def test_rms_of_zeros_tiny_and_nonfinite_rows(dtype):
    import torch
    g, rng = G(), np.random.default_rng(5)
    for size in (5, 300, 4100, 20000):
        v = rng.standard_normal((6, size))
        v[0] = 0
        v[1] *= 2.0 ** -20
        v[2, size // 2] = np.nan
        v[3, 1] = np.inf
        x = lu.matrix(v, dtype)
        w = torch.full((size,), 0.5, device="cuda")
        xv = lu.values(x)
        for eps in (EPS, 2.0 ** -126):
            y, rstd, kept = g.rms_norm_forward(x, w, eps, keep=True)
            with np.errstate(invalid="ignore"):
                wr = B.rms(xv, eps)
                wy = xv * wr[:, None] * 0.5
            yv = lu.values(y)
            assert np.isnan(yv[2]).all() and np.isnan(yv[3, 1]) and (yv[3, 2:] == 0).all() and (yv[0] == 0).all()
            keep = [0, 1, 4, 5]
            lu.within(yv[keep], wy[keep], bu.stored(wy[keep], dtype, bu.REL_Y * np.abs(wy[keep])), f"{size} {eps}")
            bu.check_packed(kept, xv, "block", f"{size} kept")
            for mode in bu.MODES:
                p = g.rms_norm_forward(x, w, eps, packed=mode)[0]
                q, s, _ = bu.packed_values(p)
                assert np.isnan(q[2]).all() and np.isfinite(s).all()
                bu.check_packed(G().Packed8(p.values[keep].contiguous() if size % 8 == 0 else _aligned(p.values[keep]),
                                            p.scales[keep].contiguous()), wy[keep], mode if size > 128 else "block",
                                f"{size} {mode}", bu.REL_Y)


def _aligned(values):
    import torch
    rows, size = values.shape
    held = torch.zeros(rows, (size + 7) // 8 * 8, dtype=torch.uint8, device="cuda")
    held[:, :size] = values.view(torch.uint8)
    return held.view(torch.float8_e4m3fn)[:, :size]


def test_products_that_leave_binary32_do_not_spoil_a_rows_scale():
    """x * weight over- or underflows where y does not."""
    import torch
    rng = np.random.default_rng(6)
    for xs, ws in ((1e10, 1e30), (1e-20, 1e-20), (1e-25, 1e20)):
        for size in (64, 1000, 5000, 20000):
            v = rng.standard_normal((4, size)) * xs
            x, w = lu.matrix(v, "f32"), torch.from_numpy(rng.standard_normal(size) * ws).float().cuda()
            y = G().rms_norm_forward(x, w, 2.0 ** -126, packed="row")[0]
            bu.check_rms(lu.values(x), y, None, lu.values(w), 2.0 ** -126, "f32", f"{xs} {ws} {size}", "row" if size > 128 else "block")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [5, 100, 768, 2047, 8192, 12287, 16384, 40000])
def test_rms_in_place_and_between_guards(size, dtype):
    """Outputs over inputs give the bits of apart ones; nothing around an
    output changes."""
    import torch
    g, rng = G(), np.random.default_rng(size)
    rows = 9
    v = [rng.standard_normal((rows, size)) for _ in range(4)]
    fresh = lambda: [lu.matrix(t, dtype, "padded") for t in v]  # noqa: E731
    x, r, dy, dh = fresh()
    w = torch.ones(size, device="cuda")
    m = mask()
    h, y, rstd, kept = g.residual_rms_norm_forward(x, r, w, EPS, m, keep=True)
    y0 = g.rms_norm_forward(x, w, EPS)[0]
    x1, r1, dy1, dh1 = fresh()
    got = g.residual_rms_norm_forward(x1, r1, w, EPS, m, out_h=r1, out=x1)
    assert got[0] is r1 and got[1] is x1 and bits(r1) == bits(h) and bits(x1) == bits(y)
    x1 = fresh()[0]
    assert bits(g.rms_norm_forward(x1, w, EPS, out=x1)[0]) == bits(y0)
    for held in (h, kept):
        want = g.residual_rms_norm_backward(dy, dh, held, rstd, w, m)
        _, _, dy1, dh1 = fresh()
        got = g.residual_rms_norm_backward(dy1, dh1, held, rstd, w, m, out=dy1, out_residual=dh1)
        assert bits(*got) == bits(*want)
    guard = torch.full((rows + 2, size + 11), 7.0, dtype=lu.torch_type(dtype), device="cuda")
    g.rms_norm_forward(x, w, EPS, out=guard[1:-1, 3:3 + size])
    assert bits(guard[1:-1, 3:3 + size]) == bits(y0)
    guard[1:-1, 3:3 + size] = 7.0
    assert (guard == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,size", [(9, 768), (128, 768), (100, 8200), (128, 2047), (129, 2047), (128, 16384), (70, 20000),
                                       (256, 2048), (512, 4095), (257, 8200), (256, 12289)])
def test_rms_gradients_in_place_of_few_rows(rows, size, dtype):
    """The weight's gradient reads dy and x of all rows, which the rows' own
    results may be written over."""
    import torch
    g, rng = G(), np.random.default_rng([rows, size])
    v = [rng.standard_normal((rows, size)) for _ in range(3)]
    fresh = lambda: [lu.matrix(t, dtype, "padded") for t in v]  # noqa: E731
    x, dy, dh = fresh()
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(size)).float().cuda()
    m = mask()
    _, rstd, kept = g.rms_norm_forward(x, w, EPS, keep=True)
    for held in (x, kept):
        plain, step = g.rms_norm_backward(dy, held, rstd, w), g.residual_rms_norm_backward(dy, dh, held, rstd, w, m)
        for _ in range(3):
            x1, dy1, dh1 = fresh()
            x2 = x1 if held is x else held
            assert bits(*g.rms_norm_backward(dy1, x2, rstd, w, out=dy1)) == bits(*plain)
            x1, dy1, dh1 = fresh()
            x2 = x1 if held is x else held
            assert bits(*g.residual_rms_norm_backward(dy1, dh1, x2, rstd, w, m, out=x1, out_residual=dy1)) == bits(*step)
    for _ in range(3):
        x1, dy1, _ = fresh()
        assert bits(*g.rms_norm_backward(dy1, x1, rstd, w, out=x1)) == bits(*g.rms_norm_backward(dy, x, rstd, w))


@pytest.mark.parametrize("size", [5, 64, 129, 1000, 2048, 20001])
def test_values_in_8_bits_between_guards(size):
    """The C ABI's rows of values in a wider buffer: bytes outside of a row's
    groups of eight stay."""
    import torch
    from global_l2_norm_amd import _lib
    g, rows = G(), 7
    whole, ld = (size + 7) // 8 * 8, (size + 7) // 8 * 8 + 24
    buf = torch.full((rows + 2, ld), 0x55, dtype=torch.uint8, device="cuda")
    n = -(-size // 128)
    scales = torch.full((rows + 2, n), 7.0, device="cuda")
    x = lu.matrix(np.random.default_rng(1).standard_normal((rows, size)), "bf16")
    at = _lib.GclipPacked8(buf[1:, 8:].data_ptr(), ld, scales[1:].data_ptr(), 0, 0)
    st = torch.cuda.current_stream().cuda_stream
    y = torch.empty_like(x)
    none = _lib.GclipPacked8()
    want = g.pack8(x)
    calls = [lambda: g.gclip_pack(x.data_ptr(), size, at, rows, size, _lib.GCLIP_BF16, st),
             lambda: g.gclip_rmsnorm_forward(_lib.GclipRmsForward(rows, size, _lib.GCLIP_BF16, 0, EPS, x.data_ptr(), size, None, 0,
                                                                  None, None, 0, y.data_ptr(), size, none, at, None), st),
             lambda: g.gclip_activation_forward(_lib.GclipActivate(rows, size, _lib.GCLIP_BF16, 0, x.data_ptr(), size, None, 0, at,
                                                                   none, y.data_ptr(), size, None, 0, None, 0, None, 0), st)]
    for call in calls:
        buf.fill_(0x55)
        scales.fill_(7.0)
        call()
        assert bits(buf[1:-1, 8:8 + size]) == bits(want.values) and bits(scales[1:-1]) == bits(want.scales)
        buf[1:-1, 8:8 + whole] = 0x55
        scales[1:-1] = 7.0
        assert (buf == 0x55).all() and (scales == 7.0).all()


# ---------------------------------------------------------------- the activation
def run_activation(rows, size, dtype, kind, gated, layout="plain", seed=0, spread=3.0):
    import torch
    g, rng = G(), np.random.default_rng([rows, size, seed])
    what = f"{rows} x {size} {dtype} {kind} {'gated ' if gated else ''}{layout}"
    print(what, flush=True)
    mk = lambda s: lu.matrix(s * rng.standard_normal((rows, size)), dtype, layout)  # noqa: E731
    gate, up, dy = mk(spread), mk(1.0) if gated else None, mk(1.0)
    gv, dyv = lu.values(gate), lu.values(dy)
    uv = lu.values(up) if gated else np.ones_like(gv)

    def check_y(y, a, b, note):
        wy = B.act(kind, a)[0] * b
        tol = bu.act_tolerances(kind, a)[0] * np.abs(b) + 2 * lu.U * np.abs(wy)
        lu.within(lu.values(y), wy, bu.stored(wy, dtype, tol), what + note)

    y, no_gate, no_up = g.activation_forward(gate, up, kind)
    assert no_gate is None and no_up is None
    check_y(y, gv, uv, " y")
    y8, gate8, up8 = g.activation_forward(gate, up, kind, keep=True)
    assert bits(y8) == bits(y) and (up8 is None) == (not gated)
    bu.check_packed(gate8, gv, "block", what + " gate8")
    if gated:
        bu.check_packed(up8, uv, "block", what + " up8")
    for hg, hu, note in ((gate, up, ""), (gate8, up8, " kept")):
        a = gv if hg is gate else bu.packed_values(gate8)[2].astype(np.float32).astype(np.float64)
        b = np.ones_like(a) if not gated else uv if hu is up else bu.packed_values(up8)[2].astype(np.float32).astype(np.float64)
        dgate, dup, none = g.activation_backward(dy, hg, hu, kind)
        assert none is None
        dgate1, dup1, again = g.activation_backward(dy, hg, hu, kind, recompute=True)
        assert bits(dgate, dup) == bits(dgate1, dup1)
        check_y(again, a, b, note + " y again")
        ty, ts = bu.act_tolerances(kind, a)
        wy, ws = B.act(kind, a)
        want = dyv * b * ws
        # the derivative's own error, its product's roundings, and where its
        # terms cancel the result is smaller than they are
        tol = np.abs(dyv * b) * (ts + 3 * lu.U * np.abs(ws))
        lu.within(lu.values(dgate), want, bu.stored(want, dtype, tol), what + note + " dgate")
        if gated:
            want = dyv * wy
            lu.within(lu.values(dup), want, bu.stored(want, dtype, np.abs(dyv) * ty + 2 * lu.U * np.abs(want)), what + note + " dup")
        else:
            assert dup is None


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [1, 3, 7, 8, 9, 64, 100, 127, 128, 129, 255, 257, 1000, 1367, 2048, 5504, 8193, 33001])
def test_activation_every_row_length(size, dtype):
    for i, (rows, layout) in enumerate(((1, "plain"), (5, "padded"), (37, "shifted"))):
        for gated in (False, True):
            run_activation(rows, size, dtype, KINDS[(i + size) % 4], gated, layout)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
def test_activation_of_every_kind(kind, dtype):
    run_activation(64, 1024, dtype, kind, True, spread=6.0)
    run_activation(63, 1001, dtype, kind, False, "padded", spread=20.0)
    run_activation(1, 4096, dtype, kind, True, spread=0.01)


@pytest.mark.parametrize("dtype,rows,size", [("bf16", 20000, 2048), ("f32", 11001, 1801), ("f16", 650001, 63)])
@pytest.mark.parametrize("gated", [False, True])
def test_activation_streamed(dtype, rows, size, gated):
    """Calls that move enough to be streamed give the bits of the same rows in
    calls that are not."""
    import torch
    g = G()
    torch.manual_seed(rows)
    make = lambda: torch.randn(rows, size, device="cuda").to(lu.torch_type(dtype))  # noqa: E731
    gate, up, dy = make(), make() if gated else None, make()
    y, gate8, up8 = g.activation_forward(gate, up, keep=True)
    whole = [y, g.activation_forward(gate, up)[0], gate8.values.contiguous().view(torch.uint8), gate8.scales]
    for held, other in ((gate, up), (gate8, up8)):
        whole += [t for t in g.activation_backward(dy, held, other, recompute=True) if t is not None]
    for first in range(0, rows, -(-rows // 8)):
        at = slice(first, first + -(-rows // 8))
        u = up[at] if gated else None
        y, gate8, up8 = g.activation_forward(gate[at], u, keep=True)
        parts = [y, g.activation_forward(gate[at], u)[0], gate8.values.contiguous().view(torch.uint8), gate8.scales]
        for held, other in ((gate[at], u), (gate8, up8)):
            parts += [t for t in g.activation_backward(dy[at], held, other, recompute=True) if t is not None]
        assert all(torch.equal(w[at], p) for w, p in zip(whole, parts, strict=True))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_activation_far_out(kind, dtype):
    """Far from zero the activations are 0 and x, their slopes 0 and 1; NaNs
    stay."""
    import torch
    far = [30.0, 100.0, 1000.0, 60000.0] + ([1e10, 1e20, 1e30, 3e38] if dtype != "f16" else [])
    v = np.array([far + [-a for a in far] + [np.nan, 0.0]])
    x = lu.matrix(v, dtype)
    ones = torch.ones_like(x)
    y = lu.values(G().activation_forward(x, None, kind)[0])[0]
    s = lu.values(G().activation_backward(ones, x, None, kind)[0])[0]
    xv, n = lu.values(x)[0], len(far)
    assert np.array_equal(y[:n], xv[:n]) and (np.abs(y[n:2 * n]) <= 1e-10).all() and np.isnan(y[2 * n]) and y[2 * n + 1] == 0
    assert (s[:n] == 1).all() and (np.abs(s[n:2 * n]) <= 1e-10).all() and np.isnan(s[2 * n])
    assert s[2 * n + 1] == (0 if kind == "relu" else 0.5)


def test_activation_in_place_and_halves_of_one_matrix():
    import torch
    g, rng = G(), np.random.default_rng(9)
    for rows, size in ((65, 1000), (3, 77), (17, 5)):
        both = lu.matrix(rng.standard_normal((rows, 2 * size)), "bf16")
        gate, up = both[:, :size], both[:, size:]
        dy = lu.matrix(rng.standard_normal((rows, size)), "bf16")
        y, gate8, up8 = g.activation_forward(gate, up, keep=True)
        assert bits(y) == bits(g.activation_forward(gate.contiguous(), up.contiguous())[0])
        dgate, dup, _ = g.activation_backward(dy, gate, up)
        into = torch.full((rows, 2 * size + 3), 7.0, dtype=torch.bfloat16, device="cuda")
        g.activation_backward(dy, gate, up, out_gate=into[:, 1:1 + size], out_up=into[:, 1 + size:1 + 2 * size])
        assert bits(into[:, 1:1 + size], into[:, 1 + size:1 + 2 * size]) == bits(dgate, dup)
        assert (into[:, 0] == 7).all() and (into[:, 1 + 2 * size:] == 7).all()
        again = both.clone()
        g.activation_backward(dy, again[:, :size], again[:, size:], out_gate=again[:, :size], out_up=again[:, size:])
        assert bits(again) == bits(torch.cat((dgate, dup), 1))
        one = gate.contiguous()
        assert bits(g.activation_forward(one, up, out=one)[0]) == bits(y)


# ---------------------------------------------------------------- refusals
def test_refusals():
    import torch
    g = G()
    x, w, r = torch.ones(8, 256, device="cuda"), torch.ones(256, device="cuda"), torch.ones(8, device="cuda")
    p = g.pack8(x)
    other = g.pack8(torch.ones(8, 128, device="cuda"))
    bad = [(ValueError, lambda: g.rms_norm_forward(x, packed="rows")), (ValueError, lambda: g.rms_norm_forward(x, out=x, packed="row")),
           (ValueError, lambda: g.rms_norm_forward(x, w[:8])), (TypeError, lambda: g.rms_norm_forward(x, w.half())),
           (ValueError, lambda: g.rms_norm_forward(x.t())), (g.GclipError, lambda: g.rms_norm_forward(x, eps=0.0)),
           (ValueError, lambda: g.rms_norm_backward(x, other, r)), (ValueError, lambda: g.rms_norm_backward(x, x[:4], r)),
           (TypeError, lambda: g.rms_norm_backward(x, x, r.double())), (ValueError, lambda: g.rms_norm_backward(x, x, r[:3])),
           (ValueError, lambda: g.rms_norm_backward(x, x, r, accumulate=True, weight_grad=True)),
           (TypeError, lambda: g.rms_norm_backward(x, x.half(), r)), (ValueError, lambda: g.residual_rms_norm_forward(x, x[:4])),
           (ValueError, lambda: g.activation_forward(x, x[:4])), (ValueError, lambda: g.activation_forward(x, kind="tanh")),
           (TypeError, lambda: g.activation_backward(x, p, x)), (TypeError, lambda: g.activation_backward(x, x, p)),
           (ValueError, lambda: g.activation_backward(x, other)), (ValueError, lambda: g.activation_backward(x, x, out=x.clone())),
           (ValueError, lambda: g.activation_backward(x, x, out_up=x.clone())),
           (g.GclipError, lambda: g.activation_backward(x, x, x, out_gate=x.clone()[:, :256], out_up=x[:1].expand(8, 256))),
           (TypeError, lambda: g.unpack8(p, torch.float64)), (TypeError, lambda: g.unpack8(p, torch.float16, out=x)),
           (ValueError, lambda: g.unpack8(p, out=x[:4])), (ValueError, lambda: g.pack8(x[:, :0])),
           (g.GclipError, lambda: g.unpack8(p, out=x[:1].expand(8, 256)))]
    for error, call in bad:
        with pytest.raises(error):
            call()
    moved = g.pack8(x)
    moved.values.set_(torch.zeros(8, 256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn))
    with pytest.raises(ValueError, match="storage"):
        moved.dequantize()


def test_no_rows_and_no_columns():
    import torch
    g = G()
    x, w = torch.ones(0, 24, device="cuda"), torch.ones(24, device="cuda")
    y, rstd, kept = g.rms_norm_forward(x, w, packed="row", keep=True)
    assert y.shape == (0, 24) and rstd.shape == (0,) and kept.scales.shape == (0, 1)
    dx, dw = g.rms_norm_backward(x, kept, rstd, w)
    assert dx.shape == (0, 24) and (dw == 0).all()
    acc = torch.full((24,), 5.0, device="cuda")
    g.rms_norm_backward(x, x, rstd, w, dweight=acc, accumulate=True)
    assert (acc == 5).all()
    assert g.activation_forward(x, x, keep=True)[0].shape == (0, 24)
    assert g.activation_backward(x, x, x)[1].shape == (0, 24)
    assert g.unpack8(g.pack8(x)).shape == (0, 24)
    e = torch.ones(4, 0, device="cuda")
    assert g.activation_forward(e, e)[0].shape == (4, 0) and g.activation_backward(e, e, e)[0].shape == (4, 0)


def test_single_rows_without_other_dimensions():
    import torch
    g, x, w = G(), torch.randn(300, device="cuda"), torch.ones(300, device="cuda")
    m = x[None]
    for args in ({}, {"packed": "row", "keep": True}, {"packed": "block"}):
        a, b = g.rms_norm_forward(x, w, **args), g.rms_norm_forward(m, w, **args)
        assert bits(*a) == bits(*b) and a[1].shape == () and a[0].shape == (300,)
    y, rstd, kept = g.rms_norm_forward(x, w, keep=True)
    assert bits(*g.rms_norm_backward(x, kept, rstd, w)) == bits(*g.rms_norm_backward(m, g.pack8(m), rstd[None], w))
    assert bits(*g.activation_forward(x, w, keep=True)) == bits(*g.activation_forward(m, w[None], keep=True))
    assert bits(g.unpack8(g.pack8(x))) == bits(g.unpack8(g.pack8(m)))
    t = torch.tensor(7, device="cuda")
    a, b = (g.token_log_probs_forward(v, s, entropy=True, top=3) for v, s in ((x, t), (m, t[None])))
    assert bits(*a) == bits(*b) and a.logp.shape == () and a.top_ids.shape == (3,)
    v = x.clone().requires_grad_()
    g.token_log_probs(g.rms_norm(g.activation(v, checkpoint=True), w, checkpoint=True), t).logp.backward()
    assert torch.isfinite(v.grad).all()


# ---------------------------------------------------------------- as they are used
def test_large_matrices():
    """Rows and columns past 2^31 elements and 4 GiB."""
    import torch
    g = G()
    rows, size = 70001, 32768
    x = torch.empty(rows, size, dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 10000):
        x[i:i + 10000].normal_(generator=torch.Generator("cuda").manual_seed(i))
    last = x[-3:].clone()
    y, rstd, kept = g.rms_norm_forward(x, None, EPS, keep=True)
    a, ra, ka = g.rms_norm_forward(last, None, EPS, keep=True)
    assert bits(y[-3:]) == bits(a) and bits(rstd[-3:]) == bits(ra)
    assert bits(kept.values[-3:]) == bits(ka.values) and bits(kept.scales[-3:]) == bits(ka.scales)
    dx, _ = g.rms_norm_backward(x, kept, rstd, out=y)
    b, _ = g.rms_norm_backward(last, ka, ra)
    assert bits(dx[-3:]) == bits(b)
    back = g.unpack8(kept, out=y)
    assert bits(back[-3:]) == bits(g.unpack8(ka))
    del kept
    z, k8, _ = g.activation_forward(x, None, keep=True, out=y)
    c, kc, _ = g.activation_forward(last, None, keep=True)
    assert bits(z[-3:]) == bits(c) and bits(k8.values[-3:]) == bits(kc.values) and bits(k8.scales[-3:]) == bits(kc.scales)
    dgate, _, _ = g.activation_backward(x, k8, out_gate=y)
    assert bits(dgate[-3:]) == bits(g.activation_backward(last, kc)[0])


def test_one_row_of_everything():
    """The longest row that fits: columns past 2^31 bytes."""
    import torch
    g, size = G(), (1 << 30) + 1027
    x = torch.ones(1, size, dtype=torch.bfloat16, device="cuda")
    x[0, -2:] = torch.tensor([3.0, -448.0])
    y, rstd, kept = g.rms_norm_forward(x, None, EPS, keep=True)
    want = float(1 / np.sqrt((size - 2 + 9 + 448.0 ** 2) / size + EPS))
    assert abs(float(rstd) - want) <= bu.rstd_tolerance(want)
    assert float(kept.scales[0, -1]) == 1.0 and kept.values[0, -2:].float().tolist() == [3.0, -448.0]
    z, k8, _ = g.activation_forward(x, None, "relu", keep=True, out=y)
    assert z[0, -2:].tolist() == [3.0, 0.0] and bits(k8.values[0, -200:]) == bits(kept.values[0, -200:])


def test_the_same_bits_every_run():
    g, rng = G(), np.random.default_rng(11)
    import torch
    for rows, size in ((300, 1000), (3000, 768), (9, 20000)):
        x, r, dy, dh = (lu.matrix(rng.standard_normal((rows, size)), "bf16") for _ in range(4))
        w = torch.ones(size, device="cuda")
        runs = []
        for _ in range(3):
            f = g.residual_rms_norm_forward(x, r, w, EPS, mask(), packed="row", keep=True)
            b = g.residual_rms_norm_backward(dy, dh, f[3], f[2], w, mask())
            a = g.activation_forward(x, r, keep=True)
            c = g.activation_backward(dy, a[1], a[2], recompute=True)
            runs.append(bits(*f, *b, *a, *c))
        assert runs[0] == runs[1] == runs[2]


def test_captured_and_replayed():
    import torch
    g, rng = G(), np.random.default_rng(12)
    rows, size = 200, 1000
    x, r, dy, dh = (lu.matrix(rng.standard_normal((rows, size)), "bf16") for _ in range(4))
    w, acc = torch.ones(size, device="cuda"), torch.zeros(size, device="cuda")
    counter = torch.zeros(1, dtype=torch.int32, device="cuda")
    m = g.DropoutMask(0.3, 5, counter=counter)

    def step(acc):
        h, y, rstd, kept = g.residual_rms_norm_forward(x, r, w, EPS, m, keep=True)
        z, g8, u8 = g.activation_forward(y, h, keep=True)
        dgate, dup, _ = g.activation_backward(dy, g8, u8)
        return h, y, z, *g.residual_rms_norm_backward(dgate, dup, kept, rstd, w, m, dweight=acc, accumulate=True)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(acc)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(acc)
    acc.zero_()
    for i in range(4):
        x.mul_(0.75)
        eager = acc.clone()
        want = bits(*step(eager)[:-1], eager)
        graph.replay()
        torch.cuda.synchronize()
        assert bits(*out[:-1], acc) == want, i
        counter.add_(1)


def test_another_stream_and_two_at_once():
    import torch
    g, rng = G(), np.random.default_rng(13)
    xs = [lu.matrix(rng.standard_normal((4000, 2048)), "bf16") for _ in range(2)]
    w = torch.ones(2048, device="cuda")
    streams = [torch.cuda.Stream() for _ in xs]

    def passes(x, stream=None):
        y, rstd, kept = g.rms_norm_forward(x, w, EPS, keep=True, stream=stream)
        dx, dw = g.rms_norm_backward(y, kept, rstd, w, stream=stream)
        z, g8, u8 = g.activation_forward(y, dx, keep=True, stream=stream)
        d = g.activation_backward(z, g8, u8, stream=stream)
        return y, rstd, kept, dx, dw, z, g8, u8, *d, g.unpack8(g.pack8(d[0], "row", stream=stream), stream=stream)

    want = [bits(*passes(x)) for x in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [passes(x, s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        assert [bits(*t) for t in got] == want


@pytest.mark.parametrize("dtype", DTYPES)
def test_under_autograd(dtype):
    """The gradients are the passes'; kept in 8 bits they are those from the
    kept values, and nothing else is saved."""
    import torch
    g, rng = G(), np.random.default_rng(14)
    t = lu.torch_type(dtype)
    mk = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(t).cuda()  # noqa: E731
    x, r, w, dy, dh = mk(3, 5, 200), mk(3, 5, 200), mk(200), mk(3, 5, 200), mk(3, 5, 200)
    m = mask()
    for checkpoint in (False, True):
        leaves = [v.clone().requires_grad_() for v in (x, r, w)]
        saved = []
        with torch.autograd.graph.saved_tensors_hooks(lambda s: (saved.append(s), s)[1], lambda s: s):
            h, y = g.residual_rms_norm(*leaves, EPS, m, checkpoint=checkpoint)
        assert checkpoint != any(s.dtype == t and s.shape == x.shape for s in saved)
        torch.autograd.backward((h, y), (dh, dy))
        fh, fy, rstd, kept = g.residual_rms_norm_forward(x, r, w, EPS, m, keep=True)
        want = g.residual_rms_norm_backward(dy, dh, kept if checkpoint else fh, rstd, w, m)
        assert bits(h, y) == bits(fh, fy) and bits(*(v.grad for v in leaves)) == bits(*want)

        leaves = [v.clone().requires_grad_() for v in (x, w)]
        y = g.rms_norm(*leaves, EPS, checkpoint=checkpoint)
        y.backward(dy.transpose(0, 1).contiguous().transpose(0, 1))
        fy, rstd, kept = g.rms_norm_forward(x, w, EPS, keep=True)
        assert bits(y) == bits(fy)
        assert bits(*(v.grad for v in leaves)) == bits(*g.rms_norm_backward(dy, kept if checkpoint else x, rstd, w))

        for up in (r, None):
            leaves = [v.clone().requires_grad_() for v in (x, up) if v is not None]
            y = g.activation(*leaves, kind="gelu_tanh", checkpoint=checkpoint)
            y.backward(dy)
            fy, g8, u8 = g.activation_forward(x, up, "gelu_tanh", keep=True)
            want = g.activation_backward(dy, g8 if checkpoint else x, u8 if checkpoint else up, "gelu_tanh")
            assert bits(y) == bits(fy) and bits(*(v.grad for v in leaves)) == bits(*want[:2])
        # nothing is tracked
        with torch.no_grad():
            assert g.rms_norm(leaves[0], w).grad_fn is None and g.activation(leaves[0]).grad_fn is None
    # parts that are not asked for
    a = x.clone().requires_grad_()
    g.residual_rms_norm(a, r, w, EPS, m)[0].backward(dh)
    assert bits(a.grad) == bits(g.dropout_backward(dh, m))
    b = w.clone().requires_grad_()
    g.rms_norm(x, b, EPS).backward(dy)
    assert bits(b.grad) == bits(g.rms_norm_backward(dy, x, g.rms_norm_forward(x, w, EPS)[1], w)[1])
    with pytest.raises(RuntimeError):
        v = x.clone().requires_grad_()
        (first,) = torch.autograd.grad(g.activation(v).sum(), v, create_graph=True)
        first.sum().backward()


def test_saved_tensors_may_be_moved():
    """Hooks that move what autograd saves (to the host and back, or into
    memory of another layout) keep the gradients' bits."""
    import torch
    g = G()
    for size in (200, 203):
        x = torch.randn(6, 2 * size, device="cuda", dtype=torch.bfloat16)
        w = torch.ones(size, device="cuda")

        def step(hooks):
            v = x.clone().requires_grad_()
            with hooks:
                h, y = g.residual_rms_norm(v[:, :size], v[:, size:], w, checkpoint=True)
                z = g.activation(y, h, checkpoint=True)
                z = g.rms_norm(z, w, checkpoint=True)
                p = g.token_log_probs(z, torch.zeros(6, dtype=torch.int64, device="cuda"), entropy=True)
            (p.logp.sum() + p.entropy.sum()).backward()
            return bits(v.grad)
        import contextlib
        want = step(contextlib.nullcontext())
        assert step(torch.autograd.graph.save_on_cpu()) == want
        assert step(torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(memory_format=torch.contiguous_format), lambda t: t)) == want


def test_written_buffers_count_their_versions_up():
    import torch
    g = G()
    x = torch.randn(4, 64, device="cuda").requires_grad_()
    y = x.exp()  # saves its result
    g.rms_norm_forward(torch.ones(4, 64, device="cuda"), out=y.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.sum().backward()
