"""The operators of include/gclip_block.h and gclip_logprob.h in binary64 on
the CPU, from their definitions: numpy arrays [rows, size] in, binary64 out."""
import math

import numpy as np

from .pieces import by_rows, in_pieces, joined

BLOCK = 128
LEAST_SCALE = 2.0 ** -112


# ---------------------------------------------------------------- 8 bits
def e4m3_table():
    """The 256 values of the OCP 8-bit float with 4 exponent and 3 fraction
    bits: sign, exponent biased by 7, no infinity, NaN where all others are set."""
    out = np.empty(256)
    for b in range(256):
        sign, exponent, fraction = -1.0 if b >> 7 else 1.0, b >> 3 & 15, b & 7
        if exponent == 15 and fraction == 7:
            out[b] = math.nan
        elif exponent == 0:
            out[b] = sign * fraction * 2.0 ** -9
        else:
            out[b] = sign * (8 + fraction) * 2.0 ** (exponent - 10)
    return out


E4M3 = e4m3_table()


@by_rows(0)
def e4m3_half_step(v):
    """Half of the distance of the values around v."""
    a = np.maximum(np.abs(v), 2.0 ** -6)
    finite = np.isfinite(a)
    # a = f 2^e with f in [1/2, 1)
    return np.where(finite, np.ldexp(1.0, np.frexp(np.where(finite, a, 1.0))[1] - 5), 0.0)


def round_e4m3(v):
    """v to the nearest value, of two equally near ones the even one."""
    step = 2.0 * e4m3_half_step(v)
    return np.where(np.isfinite(v), np.round(v / np.where(step == 0, 1.0, step)) * step, np.nan)


def groups(v, mode):
    """The columns that share a scale, as slices."""
    size = v.shape[1]
    return [slice(0, size)] if mode == "row" else [slice(c, min(c + BLOCK, size)) for c in range(0, size, BLOCK)]


@by_rows(0)
def scales(v, mode):
    out = []
    for g in groups(v, mode):
        part = np.abs(v[:, g])
        out.append(np.maximum(np.where(np.isfinite(part), part, 0.0).max(1) / 448.0, LEAST_SCALE))
    return np.stack(out, 1)


def spread(s, size, mode):
    """The scales of a row's columns."""
    return np.broadcast_to(s, (s.shape[0], size)) if mode == "row" else np.repeat(s, BLOCK, 1)[:, :size]


# ---------------------------------------------------------------- RMS norm
@by_rows(0)
def rms(x, eps):
    """rstd"""
    return 1.0 / np.sqrt((x.astype(np.float64) ** 2).sum(1) / x.shape[1] + eps)


def rms_gradient(dy, x, rstd, weight):
    """(dx, dweight)"""
    def piece(i, j):
        n = x[i:j] * rstd[i:j, None]
        g = dy[i:j] * weight
        return rstd[i:j, None] * (g - n * ((g * n).sum(1, keepdims=True) / x.shape[1])), (dy[i:j] * n).sum(0)[None]
    dx, dw = joined(in_pieces(piece, *x.shape))
    return dx, dw.sum(0)


# ---------------------------------------------------------------- the activation
def _erfc(x):
    from scipy.special import erfc
    return erfc(x)


def _logistic(x):
    from scipy.special import expit
    return expit(x)


@by_rows(1)
def act(kind, x):
    """(act(x), its derivative)"""
    if kind == "relu":
        return np.where(x > 0, x, 0.0), np.where(x > 0, 1.0, 0.0)
    if kind == "silu":
        p = _logistic(x)
        return x * p, p * (1.0 + x * _logistic(-x))
    if kind == "gelu":
        c = 0.5 * _erfc(-x / math.sqrt(2.0))
        return x * c, c + x * np.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    k = math.sqrt(2.0 / math.pi)
    p = _logistic(2.0 * k * (x + 0.044715 * x ** 3))
    q = _logistic(-2.0 * k * (x + 0.044715 * x ** 3))
    return x * p, p + x * p * q * 2.0 * k * (1.0 + 3 * 0.044715 * x * x)


# ---------------------------------------------------------------- log probabilities
@by_rows(0)
def log_probs(x):
    """(m, s, log p, p, entropy); rows of nothing but -infinity: m, s and log p
    of -infinity, and an entropy of 0."""
    x = x.astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        m = np.where(np.isnan(x), -np.inf, x).max(1)
        r = np.where(np.isneginf(m), 0.0, m)[:, None]
        s = np.log(np.exp(x - r).sum(1))
        z = np.where(np.isneginf(x), -np.inf, x - r - s[:, None])
        z = np.where(np.isnan(s)[:, None], np.nan, z)
        p = np.exp(z)
        h = -np.where(p > 0, p * np.where(p > 0, z, 0.0), np.where(np.isnan(p), np.nan, 0.0)).sum(1)
    return m, s, z, p, h


@by_rows(0)
def top(x, k):
    """Columns of the k largest, NaNs above everything, of equal ones the
    lowest first."""
    out = np.empty((len(x), k), dtype=np.int64)
    for row, r in zip(x, out):
        # numpy's order has NaNs behind everything: the k-th from there
        least = np.partition(row, len(row) - k)[len(row) - k] if k else np.nan
        columns = np.flatnonzero(np.isnan(row) if np.isnan(least) else np.isnan(row) | (row >= least))
        v = row[columns]
        r[:] = columns[np.lexsort((columns, -np.where(np.isnan(v), np.inf, v), ~np.isnan(v)))[:k]]
    return out


@by_rows(0, 1, 2, 3, 4, 5, 6)
def log_probs_gradient(x, target, dlogp, dentropy, m, s, entropy, ignore=-100):
    """dlogits from the given m, s and entropy."""
    x = x.astype(np.float64)
    with np.errstate(invalid="ignore"):
        z = x - m[:, None] - s[:, None]
        p = np.exp(z)
        zero = np.zeros_like(p)
        d = -np.where(p == 0, zero, p * (dlogp[:, None] + dentropy[:, None] * (np.where(p == 0, 0.0, z) + entropy[:, None])))
    valid = (target >= 0) & (target < x.shape[1])
    d[np.flatnonzero(valid), target[valid]] += dlogp[valid]
    d[~valid] = np.nan
    d[np.isneginf(s)] = 0.0
    d[target == ignore] = 0.0
    return d
