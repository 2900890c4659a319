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
