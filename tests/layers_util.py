"""Helpers of the layers' GPU tests: inputs in a storage format with layouts
a caller may have, their binary64 values, and how far results may be off.

Tolerances, with u = 2^-24 (half a step of binary32, in which everything is
computed) and half(T) half a step of the storage format T, to which results
are rounded once.  A sum of k terms in any order is off by at most
(k - 1) u times the sum of their absolute values.  The kernels add a row's
terms in chains of at most 32 in a lane, then by a tree of six levels over a
wave, then the sums of at most 16 waves: a path of at most 31 + 6 + 15 = 52
additions (rows of other lengths in binary64), for which 64 stands."""
import numpy as np

U = 2.0 ** -24
PATH = 64
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # torch.finfo(T).eps / 2
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half a step of the subnormals


def torch_type(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def matrix(values, dtype, layout="plain"):
    """A device tensor holding `values` in the format: `plain`, `padded`
    (rows further apart, beginning at any element), `shifted` (contiguous,
    off by one element), or `one row` (row 0 for all)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(values)).to(torch_type(dtype))
    rows, size = t.shape
    if layout == "padded":
        buf = torch.full((rows * (size + 5) + 3,), 3.0, dtype=t.dtype, device="cuda")
        out = buf[1:1 + rows * (size + 5)].view(rows, size + 5)[:, 2:2 + size]
        return out.copy_(t)
    if layout == "shifted":
        buf = torch.full((rows * size + 1,), 3.0, dtype=t.dtype, device="cuda")
        return buf[1:].view(rows, size).copy_(t)
    if layout == "one row":
        return t[:1].cuda().expand(rows, size)
    return t.cuda()


def values(t):
    return t.detach().double().cpu().numpy()


def rounded(t, dtype):
    """binary32 numpy values as the format's, exactly."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(t, dtype=np.float32)).to(torch_type(dtype)).double().numpy()


def within(got, want, tol, what):
    got, want, tol = np.broadcast_arrays(got, want, tol)
    nan = np.isnan(want)
    assert np.array_equal(nan, np.isnan(got)), f"{what}: NaN at other places"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: other infinities"
    ok = nan | inf
    with np.errstate(invalid="ignore"):
        off = np.where(ok, 0.0, np.abs(got - want))
        bad = ~(off <= np.where(ok, 1.0, tol))
    if bad.any():
        i = tuple(int(k) for k in np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} too far off, first at {i}: {got[i]!r} for "
                             f"{want[i]!r}, tolerance {tol[i]!r}")


def statistics_tolerance(x, mean, rstd):
    """Of mean (absolute) and rstd (absolute), and D, the error of the mean in
    standard deviations.  Sum: PATH u max|x| each.  Squares: PATH + 2 u, and
    the mean's error adds its square; half of that in rstd, and two operations
    more, one of them a root."""
    big = np.abs(x).max(1)
    dm = (PATH + 1) * U * big
    d = dm * rstd
    return dm, rstd * ((PATH + 10) / 2 * U + d * d), d


def check_norm(x, y, mean, rstd, w, b, eps, dtype, what):
    """y (and mean, rstd where kept) against the norm of the stored x."""
    from oracle import layers as L
    wy, wm, wr = L.norm(x, w, b, eps)
    dm, dr, d = statistics_tolerance(x, wm, wr)
    n = (x - wm[:, None]) * wr[:, None]
    # n: the mean's error, a rounding of x - mean, rstd's, a product
    dn = d[:, None] + np.abs(n) * (dr / wr + 2 * U)[:, None]
    tol = np.abs(w) * dn + 3 * U * (np.abs(n * w) + np.abs(b))
    tol = tol + HALF[dtype] * (np.abs(wy) + tol) + TINY[dtype]
    within(y, wy, tol, what + " y")
    if mean is not None:
        within(mean, wm, dm, what + " mean")
        within(rstd, wr, dr, what + " rstd")


def check_norm_gradient(dx, dw, db, dy, x, mean, rstd, w, dtype, gtype, what, dh=None, factor=None, dres=None,
                        dw0=0.0, db0=0.0):
    """Gradients against the formula from the given mean and rstd."""
    from oracle import layers as L
    wdx, wdw, wdb = L.norm_gradient(dy, x, mean, rstd, w)
    n = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    ag, agn = np.abs(g).mean(1)[:, None], np.abs(g * n).mean(1)[:, None]
    # three roundings a term and the sum's path; n is off by 2 u of itself
    tol = np.abs(rstd)[:, None] * (6 * U * (np.abs(g) + ag + np.abs(n) * agn) + PATH * U * (ag + np.abs(n) * agn))
    if dh is not None:
        wdx = wdx + dh
    tol = tol + U * np.abs(wdx)
    store = lambda v, t: t + HALF[dtype] * (np.abs(v) + t) + TINY[dtype]  # noqa: E731
    if dres is not None:
        within(dres, wdx, store(wdx, tol), what + " dresidual")
    if factor is not None:
        wdx, tol = wdx * factor, tol * factor + 2 * U * np.abs(wdx * factor)
    if dx is not None:
        within(dx, wdx, store(wdx, tol), what + " dx")
    rows = x.shape[0]
    for got, want, start, size_of in ((dw, wdw, dw0, np.abs(dy * n).sum(0)), (db, wdb, db0, np.abs(dy).sum(0))):
        if got is not None:
            want = want + start
            t = (rows + 4) * U * size_of + U * np.abs(want)
            within(got, want, t + HALF[gtype] * (np.abs(want) + t) + TINY[gtype], what + " weight gradients")
