"""Helpers of the GPU tests of the block operators and the log probabilities:
how far results may be off, by the roundings that they take.

u = 2^-24 is half a step of binary32, in which everything is computed; PATH
bounds the additions that a term of a row's sum goes through (layers_util)."""
import math

import numpy as np

from oracle import block as B
from tests.layers_util import HALF, PATH, TINY, U, within

MODES = ("block", "row")


def stored(v, dtype, tol):
    """Of v with an error of tol, rounded once to the format."""
    return tol + HALF[dtype] * (np.abs(v) + tol) + TINY[dtype]


def packed_values(p):
    """(values as stored, scales, what they stand for) of a Packed8, binary64."""
    q = p.values.double().cpu().numpy().reshape(-1, p.shape[-1])
    s = p.scales.double().cpu().numpy().reshape(q.shape[0], -1)
    mode = "row" if s.shape[1] == 1 else "block"
    return q, s, q * B.spread(s, q.shape[1], mode)


def check_packed(p, v, mode, what, rel=0.0):
    """p against v (each element known to `rel` of itself).  A scale is the
    largest magnitude times 1/448, two roundings; a value is v times the
    scale's reciprocal, two more, so it is within half a step of the format of
    v / scale (1 + 4 u + twice rel, the largest's and its own)."""
    q, s, _ = packed_values(p)
    want = B.scales(v, mode)
    assert s.shape == want.shape, what
    within(s, want, want * (rel + 2 * U), what + " scales")
    spread = B.spread(s, v.shape[1], mode)
    with np.errstate(invalid="ignore"):
        x = np.where(np.isfinite(v), v / spread, np.nan)
    tol = np.abs(x) * (2 * rel + 4 * U)
    # the step at the end of the error's range
    within(q, x, tol + B.e4m3_half_step(np.abs(x) + tol), what + " values")


def rstd_tolerance(rstd):
    """The squares' sum is off by PATH + 2 u of itself, the mean and eps add
    three more; half of that, and a root and a division."""
    return rstd * ((PATH + 5) / 2 + 3) * U


REL_Y = ((PATH + 5) / 2 + 5) * U  # rstd and two products


def check_rms(x, y, rstd, w, eps, dtype, what, mode=None):
    """y (a matrix, or a Packed8 with scales of `mode`) and rstd against the
    norm of the stored x."""
    wr = B.rms(x, eps)
    wy = x * wr[:, None] * w
    if mode:
        check_packed(y, wy, mode, what + " y8", REL_Y)
    else:
        within(y, wy, stored(wy, dtype, REL_Y * np.abs(wy)), what + " y")
    if rstd is not None:
        within(rstd, wr, rstd_tolerance(wr) + 2.0 ** -149, what + " rstd")


def check_rms_gradient(dx, dw, dy, x, rstd, w, dtype, gtype, what, dh=None, factor=None, dres=None, dw0=0.0):
    """Gradients against the formula from the given rstd and x."""
    wdx, wdw = B.rms_gradient(dy, x, rstd, w)
    n = x * rstd[:, None]
    g = dy * w
    agn = np.abs(g * n).mean(1)[:, None]
    # g, n and their product: three roundings a term, and the sum's path; then
    # the mean, c2, n c2, the difference; in 8 bits n has one more
    tol = np.abs(rstd)[:, None] * (4 * U * np.abs(g) + (PATH + 10) * U * np.abs(n) * agn)
    if dh is not None:
        wdx = wdx + dh
    tol = tol + 2 * U * np.abs(wdx)
    if dres is not None:
        within(dres, wdx, stored(wdx, dtype, tol), what + " dresidual")
    if factor is not None:
        wdx, tol = wdx * factor, tol * factor + 2 * U * np.abs(wdx * factor)
    if dx is not None:
        within(dx, wdx, stored(wdx, dtype, tol), what + " dx")
    if dw is not None:
        want = wdw + dw0
        t = (x.shape[0] + 5) * U * np.abs(dy * n).sum(0) + U * np.abs(want)
        within(dw, want, stored(want, gtype, t), what + " dweight")


def act_tolerances(kind, x):
    """(of act(x), of its derivative), absolute, before rounding to a format.

    e^-x is off by (1.5 |x| + 3) u of itself: the product with log2(e), its
    constant, the power; p = 1 / (1 + e) by that times 1 - p and 3 more, and y
    by one more.  The derivative's two terms have those of p, of 1 - p and of
    two or three products.  erfc is taken to be good to 16 u, and its
    argument's rounding (1.5 u of x / sqrt 2) moves it by up to x^2 + 1 times
    that; the density e^(-x^2 / 2) has (x^2 + 4) u.  Where e^-x passes 2^126 (and leaves
    binary32 at 2^128) p may be 0, which is up to 2^-126 off: `less` of a p.
    The tail of erfc and the density below 2^-126 may be 0 as well."""
    a = np.abs(x)
    less = 2.0 ** -126
    y, slope = B.act(kind, x)
    if kind == "relu":
        return np.zeros_like(x), np.zeros_like(x)
    if kind == "silu":
        r = (1.5 * a + 8) * U
        from scipy.special import expit
        return np.abs(y) * r + less * a, expit(x) * (1 + a * expit(-x)) * 3 * r + less * (1 + a)
    if kind == "gelu":
        from scipy.special import erfc
        r = (16 + 2 * (x * x + 1)) * U
        return np.abs(y) * r + less * a, (less * (1 + a) + 0.5 * erfc(-x / math.sqrt(2)) * r
                               + a * np.exp(-0.5 * x * x) / math.sqrt(2 * math.pi) * (x * x + 6) * U)
    from scipy.special import expit
    k = math.sqrt(2 / math.pi)
    t = 2 * k * (a + 0.044715 * a ** 3)
    r = (6 * t + 10) * U
    sign = np.sign(x)
    p, q = expit(sign * t), expit(-sign * t)
    du = 2 * k * (1 + 0.134145 * x * x)
    return np.abs(y) * r + less * a, p * (1 + a * du * q) * 3 * r + less * (1 + a * du)


def log_prob_tolerances(x, chain):
    """(of s, of log p but for its own rounding, of the entropy), absolute:
    e^d is off by (1.5 |d| + 3) u of itself, its sum by the `chain` of
    additions; d and what is multiplied by it by one u each."""
    m, s, z, p, h = B.log_probs(x)
    with np.errstate(invalid="ignore"):
        d = np.where(p > 0, m[:, None] - x, 0.0)
        first, second = (p * d).sum(1), (p * d * d).sum(1)
    ts = (chain + 4) * U + 1.5 * U * first + U * np.abs(s)
    th = (chain + 8) * U * (1 + 2 * first) + 2 * U * second + 2 * U * np.abs(s) + U * np.abs(h) + 2 * first * 2 * U * (1 + first)
    return ts, ts, th
